// rope.cu — rotary positions with several axes, with an optional RMS norm.
//
// DSV's queries and keys are the tokens of a T x Hl x Wl video latent
// ([nl] 1: 3D attention over space and time).  A video transformer marks a
// token's place by rotating channel pairs of q and k: the head's channels are
// cut into one band per axis, and in a band of c channels for an axis with
// coordinate p
//   pair i: (x_2i, x_2i+1) -> rotation by p * theta^(-2i/c)
// (the frequencies and channel pairs of the sinusoidal embedding that
// workloads.posemb_3d adds); channels behind the bands pass through.  With a
// weight w the rotation's input is the row's RMS norm: x rsqrt(mean(x^2) + eps) w.
//
// Backward: g = R^T dy; without the norm dx = g.  With it, x^ = x r,
// r = rsqrt(mean(x^2) + eps):  dx = r (g w - x^ mean(g w x^)),
// dw = sum over all rows of g x^.
//
// Angles.  p theta^(-2i/c) in fp32 is off by p 2^-24 rad: 0.06 rad at p = 10^6.
// Here the frequency is a 64-bit fixed-point fraction of a turn and the product
// with the integer coordinate wraps modulo 2^64, which is modulo whole turns:
// the fraction is good to p 2^-54 turns (the frequency comes from fp64: 2^-54.8
// at worst over 48 thetas and all bands), whatever the coordinate's size or
// sign, for one integer multiplication.  Its top 32 bits go to sincospif as
// fp32, which rounds the fraction by up to 2^-26 turns: 9e-8 rad, as much as
// fp32 can say of an angle.
//
// HBM-bound: 4 bytes per element (read, write; 6 for the backward with norm)
// at ~7 fp32 operations each.  D/8 lanes hold a token's row, 16 bytes each;
// the four rotations of a lane serve the token's heads in turn, so that
// sincospif costs 4 per (token, 8 channels) and not per element; the rows of
// a few heads are loaded before any is worked on, and registers are held to 64
// a thread so that four CTAs share an SM (what counts is bytes in flight: at 80
// registers the backward with norm took 86 us instead of 64).  Measured (a
// call, share of the copy bandwidth): forward with norm, 1.0 GB: 170 us, 87 %;
// backward without norm, 1.5 GB: 222 us, 100 %; backward with norm, 0.3 GB: 64
// us, 70 % (the partial sums' kernel is 5 us of it).
#include <math.h>

#include "dsv_launch.h"

namespace dsv {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeBatch = 3;            // rows in flight per thread (2: 180 us on the stress queries, 3: 170, 4: 175)

struct RopeTable {
  uint64_t turn[64];                     // frequency of a channel pair, fraction of a turn * 2^64
  int8_t axis[64];                       // its axis, -1: not rotated
};

struct RopeArgs {
  const int32_t* pos;
  long long pos_batch;                   // elements between batches of pos (0: shared)
  int N, H, axes, chunk;                 // heads per CTA
  float eps;
};

struct Row8 {
  float v[8];
};
__device__ __forceinline__ Row8 unpack8(const uint4& q) {
  Row8 r;
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[2 * i] = __uint_as_float(w[i] << 16);
    r.v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  return r;
}
__device__ __forceinline__ uint4 pack8(const Row8& r) {
  return make_uint4(pack_bf16x2(r.v[0], r.v[1]), pack_bf16x2(r.v[2], r.v[3]), pack_bf16x2(r.v[4], r.v[5]),
                    pack_bf16x2(r.v[6], r.v[7]));
}

// Sum over the D/8 lanes of a row.
template <int D>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// cos and sin of this lane's four channel pairs at token (b, n)
struct Turns {
  float c[4], s[4];
  uint32_t rotated;                      // bit i: pair i is rotated
};
__device__ __forceinline__ Turns token_turns(const RopeTable& t, const int32_t* p, int pair0) {
  Turns z;
  z.rotated = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int a = t.axis[pair0 + i];
    z.c[i] = 1.f;
    z.s[i] = 0.f;
    if (a >= 0) {
      const uint64_t f = (uint64_t)(int64_t)p[a] * t.turn[pair0 + i];
      // signed top 32 bits: the angle in [-1/2, 1/2) turns = [-1, 1) half turns
      sincospif((float)(int32_t)(uint32_t)(f >> 32) * 4.656612873077393e-10f, &z.s[i], &z.c[i]);   // 2^-31
      z.rotated |= 1u << i;
    }
  }
  return z;
}
// dir = 1: rotation; dir = -1: its transpose.  A pair outside the bands is
// left alone (x * 1 - y * 0 would turn a non-finite y into NaN).
template <int DIR>
__device__ __forceinline__ void rotate(Row8& r, const Turns& t) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = r.v[2 * i], b = r.v[2 * i + 1], s = DIR * t.s[i];
    const bool rot = (t.rotated >> i) & 1u;
    r.v[2 * i] = rot ? a * t.c[i] - b * s : a;
    r.v[2 * i + 1] = rot ? a * s + b * t.c[i] : b;
  }
}

struct RopeView {
  const __nv_bfloat16* p;
  long long b, h, n;
};
struct RopeOut {
  __nv_bfloat16* p;
  long long b, h, n;
};

// x may be y (each 16-byte piece is read and written by one thread).
template <int D, bool NORM>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_fwd_kernel(RopeView x, RopeOut y, RopeArgs a,
                                                                const __grid_constant__ RopeTable table,
                                                                const float* __restrict__ weight) {
  constexpr int LPR = D / 8, TOK = kRopeThreads / LPR;
  __shared__ RopeTable tab;
  if (threadIdx.x < D / 2) {
    tab.turn[threadIdx.x] = table.turn[threadIdx.x];
    tab.axis[threadIdx.x] = table.axis[threadIdx.x];
  }
  __syncthreads();
  const int c = threadIdx.x % LPR;
  const int n = blockIdx.x * TOK + threadIdx.x / LPR;
  const int b = blockIdx.z, h0 = blockIdx.y * a.chunk, h1 = min(a.H, h0 + a.chunk);
  const bool live = n < a.N;
  Turns t = {};
  if (live) t = token_turns(tab, a.pos + b * a.pos_batch + (long long)n * a.axes, 4 * c);
  float w[8];
  if (NORM) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = weight[8 * c + i];
  }
  const __nv_bfloat16* xp = x.p + b * x.b + (long long)n * x.n + 8 * c;
  __nv_bfloat16* yp = y.p + b * y.b + (long long)n * y.n + 8 * c;
  for (int h = h0; h < h1; h += kRopeBatch) {
    uint4 q[kRopeBatch];
#pragma unroll
    for (int k = 0; k < kRopeBatch; ++k)
      q[k] = live && h + k < h1 ? __ldcs(reinterpret_cast<const uint4*>(xp + (h + k) * x.h)) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < kRopeBatch; ++k) {
      Row8 r = unpack8(q[k]);
      if (NORM) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(r.v[i], r.v[i], ss);
        const float rs = rsqrtf(row_sum<D>(ss) * (1.0f / D) + a.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) r.v[i] *= rs * w[i];
      }
      rotate<1>(r, t);
      if (live && h + k < h1) __stcs(reinterpret_cast<uint4*>(yp + (h + k) * y.h), pack8(r));
    }
  }
}

// dx may be dy or x.  With the norm, CTA i walks the token tiles i, i +
// gridDim.x, ... and writes its sum of g x^ to part[i]; rope_dw_kernel adds
// the parts in order, so dw does not depend on which CTA ran first.
template <int D, bool NORM>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_bwd_kernel(RopeView dy, RopeView x, RopeOut dx, RopeArgs a,
                                                                const __grid_constant__ RopeTable table,
                                                                const float* __restrict__ weight,
                                                                float* __restrict__ part, long long items,
                                                                int tiles, int chunks) {
  constexpr int LPR = D / 8, TOK = kRopeThreads / LPR;
  constexpr int BATCH = NORM ? 2 : 4;    // rows of both inputs in flight
  if (NORM) cudaTriggerProgrammaticLaunchCompletion();   // rope_dw_kernel may come to wait
  __shared__ RopeTable tab;
  __shared__ float red[TOK][D + 8];
  if (threadIdx.x < D / 2) {
    tab.turn[threadIdx.x] = table.turn[threadIdx.x];
    tab.axis[threadIdx.x] = table.axis[threadIdx.x];
  }
  __syncthreads();
  const int c = threadIdx.x % LPR, row = threadIdx.x / LPR;
  float w[8], dw[8] = {};
  if (NORM) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = weight[8 * c + i];
  }
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int tile = (int)(it % tiles);
    const int rest = (int)(it / tiles);
    const int b = rest / chunks, h0 = (rest - b * chunks) * a.chunk, h1 = min(a.H, h0 + a.chunk);
    const int n = tile * TOK + row;
    const bool live = n < a.N;
    Turns t = {};
    if (live) t = token_turns(tab, a.pos + b * a.pos_batch + (long long)n * a.axes, 4 * c);
    const __nv_bfloat16* gp = dy.p + b * dy.b + (long long)n * dy.n + 8 * c;
    const __nv_bfloat16* xp = NORM ? x.p + b * x.b + (long long)n * x.n + 8 * c : nullptr;
    __nv_bfloat16* op = dx.p + b * dx.b + (long long)n * dx.n + 8 * c;
    for (int h = h0; h < h1; h += BATCH) {
      uint4 qg[BATCH], qx[BATCH];
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        const bool in = live && h + k < h1;
        qg[k] = in ? __ldcs(reinterpret_cast<const uint4*>(gp + (h + k) * dy.h)) : make_uint4(0, 0, 0, 0);
        if (NORM) qx[k] = in ? __ldcs(reinterpret_cast<const uint4*>(xp + (h + k) * x.h)) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        Row8 g = unpack8(qg[k]);
        rotate<-1>(g, t);
        if (NORM) {
          Row8 v = unpack8(qx[k]);
          float ss = 0.f, dot = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            ss = fmaf(v.v[i], v.v[i], ss);
            dot = fmaf(g.v[i] * w[i], v.v[i], dot);
          }
          const float rs = rsqrtf(row_sum<D>(ss) * (1.0f / D) + a.eps);
          const float mean = row_sum<D>(dot) * rs * (1.0f / D);       // mean(g w x^)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float xh = v.v[i] * rs;
            dw[i] = fmaf(g.v[i], xh, dw[i]);                          // rows past the end are zero
            g.v[i] = rs * (g.v[i] * w[i] - xh * mean);
          }
        }
        if (live && h + k < h1) __stcs(reinterpret_cast<uint4*>(op + (h + k) * dx.h), pack8(g));
      }
    }
  }
  if (NORM) {
#pragma unroll
    for (int i = 0; i < 8; ++i) red[row][8 * c + i] = dw[i];
    __syncthreads();
    if (threadIdx.x < D) {
      float s = 0.f;
#pragma unroll
      for (int r = 0; r < TOK; ++r) s += red[r][threadIdx.x];
      part[(long long)blockIdx.x * D + threadIdx.x] = s;
    }
  }
}

// dw[channel] = sum of the parts: 8 channels per CTA, 128 interleaved runs of
// parts each, joined pairwise (a fixed order).
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float* __restrict__ part, int parts, int d,
                                                       float* __restrict__ dw) {
  __shared__ float red[128][8];
  const int c = blockIdx.x * 8 + threadIdx.x, y = threadIdx.y;
  float s = 0.f;
  cudaGridDependencySynchronize();
#pragma unroll 5
  for (int p = y; p < parts; p += 128) s += part[(long long)p * d + c];
  red[y][threadIdx.x] = s;
  __syncthreads();
  for (int o = 64; o > 0; o >>= 1) {
    if (y < o) red[y][threadIdx.x] += red[y + o][threadIdx.x];
    __syncthreads();
  }
  if (y == 0) dw[c] = red[0][threadIdx.x];
}

RopeTable rope_table(const dsv_rope& r) {
  RopeTable t;
  for (int i = 0; i < 64; ++i) {
    t.turn[i] = 0;
    t.axis[i] = -1;
  }
  const double lt = log(r.theta);
  int at = 0;
  for (int a = 0; a < r.axes; ++a)
    for (int i = 0; i < r.section[a] / 2; ++i, ++at) {
      // theta^(-2i/c) / (2 pi) turns, at most 1 / (2 pi) as theta >= 1; * 2^64
      t.turn[at] = (uint64_t)(exp(lt * (-2.0 * i / r.section[a])) * (0.15915494309189533577 * 18446744073709551616.0));
      t.axis[at] = (int8_t)a;
    }
  return t;
}

// Heads per CTA: as many as leave at least `per` CTAs per SM to run (the
// rotations are worked out once per CTA, so few heads make them dear).
int head_chunk(const dsv_rope& r, int tiles, int per = 4) {
  int hc = r.H;
  while (hc > 1 && (long long)tiles * r.B * ((r.H + hc - 1) / hc) < (long long)per * kPackedSMs) hc = (hc + 1) / 2;
  return hc;
}

template <int D>
cudaError_t fwd_t(const RopeView& x, const RopeOut& y, RopeArgs a, const RopeTable& t, const dsv_rope& r,
                  const float* weight, cudaStream_t st) {
  constexpr int TOK = kRopeThreads / (D / 8);
  const int tiles = (r.N + TOK - 1) / TOK;
  a.chunk = head_chunk(r, tiles);
  const dim3 grid((unsigned)tiles, (unsigned)((r.H + a.chunk - 1) / a.chunk), (unsigned)r.B);
  if (weight) rope_fwd_kernel<D, true><<<grid, kRopeThreads, 0, st>>>(x, y, a, t, weight);
  else rope_fwd_kernel<D, false><<<grid, kRopeThreads, 0, st>>>(x, y, a, t, weight);
  return cudaGetLastError();
}

template <int D>
cudaError_t bwd_t(const RopeView& dy, const RopeView& x, const RopeOut& dx, RopeArgs a, const RopeTable& t,
                  const dsv_rope& r, const float* weight, float* dw, float* part, cudaStream_t st) {
  constexpr int TOK = kRopeThreads / (D / 8);
  const int tiles = (r.N + TOK - 1) / TOK;
  a.chunk = head_chunk(r, tiles, weight ? 12 : 4);
  const int chunks = (r.H + a.chunk - 1) / a.chunk;
  const long long items = (long long)tiles * chunks * r.B;
  if (!weight) {
    rope_bwd_kernel<D, false><<<(unsigned)items, kRopeThreads, 0, st>>>(dy, x, dx, a, t, weight, part, items, tiles,
                                                                        chunks);
    return cudaGetLastError();
  }
  const int parts = (int)(items < kRopeParts ? items : kRopeParts);
  rope_bwd_kernel<D, true><<<(unsigned)parts, kRopeThreads, 0, st>>>(dy, x, dx, a, t, weight, part, items, tiles,
                                                                     chunks);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(D / 8);
  cfg.blockDim = dim3(8, 128);
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_dw_kernel, static_cast<const float*>(part), parts, D, dw);
}

RopeView view(const dsv_view& v) {
  return {static_cast<const __nv_bfloat16*>(v.ptr), v.batch_stride, v.head_stride, v.token_stride};
}
RopeOut out(const dsv_view& v) {
  return {static_cast<__nv_bfloat16*>(v.ptr), v.batch_stride, v.head_stride, v.token_stride};
}

}  // namespace

size_t rope_bwd_ws_bytes(const dsv_rope& r) { return (size_t)kRopeParts * r.d * sizeof(float); }

cudaError_t launch_rope_fwd(const dsv_view& x, const int32_t* pos, int64_t pos_batch, const dsv_rope& r,
                            const float* weight, float eps, const dsv_view& y, cudaStream_t st) {
  const RopeArgs a{pos, pos_batch, r.N, r.H, r.axes, 0, eps};
  const RopeTable t = rope_table(r);
  return r.d == 128 ? fwd_t<128>(view(x), out(y), a, t, r, weight, st) : fwd_t<64>(view(x), out(y), a, t, r, weight, st);
}

cudaError_t launch_rope_bwd(const dsv_view& dy, const dsv_view& x, const int32_t* pos, int64_t pos_batch,
                            const dsv_rope& r, const float* weight, float eps, const dsv_view& dx, float* dw, void* ws,
                            cudaStream_t st) {
  const RopeArgs a{pos, pos_batch, r.N, r.H, r.axes, 0, eps};
  const RopeTable t = rope_table(r);
  float* part = static_cast<float*>(ws);
  return r.d == 128 ? bwd_t<128>(view(dy), view(x), out(dx), a, t, r, weight, dw, part, st)
                    : bwd_t<64>(view(dy), view(x), out(dx), a, t, r, weight, dw, part, st);
}

}  // namespace dsv
