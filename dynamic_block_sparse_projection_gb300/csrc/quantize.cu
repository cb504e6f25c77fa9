// quantize.cu — rows to 8-bit floating point, a power-of-two scale for each
// block of 1 x 128 or 128 x 128 elements, and the transposed copy.
//
//   scale = 2^k with the least k for which the block's largest magnitude is at
//   most M 2^k (M = 448 for e4m3, 57344 for e5m2: both 1.75 times a power of
//   two),  q = round-to-nearest-even of x / scale.
// A power of two makes the division exact: q is the element rounded once, to
// half a step of the 8-bit type, and q * scale is exact in fp32.
// The gradient products of a projection sum over its rows, so they read the
// transposed matrix with blocks along the rows: both copies are made from one
// read of x.  A CTA holds a 128 x 128 tile in registers, 8 x 8 elements a
// thread as they are in memory, so both copies' block maxima are inside the CTA, and
// four CTAs an SM hide each other's loads, exchanges and stores.  HBM-bound: 61440 x
// 2048 bf16 with both copies, 0.5 GB, 80 us, 6.4 TB/s (94 % of the copy bandwidth); a
// weight of 6144 x 2048 in fp32, 75 MB, 16 us: two CTAs an SM (120 registers a
// thread) and 2.5 waves.  Rows off 16 bytes are read by the
// 16-byte words that hold them (30000 x 1001 with both copies: bf16 37 us, 48 one by one, fp32 42 and 60).
#include <cuda_fp8.h>

#include "dsv_launch.h"

namespace dsv {

namespace {

constexpr int kQThreads = 256, kTile = 128;

struct QuantArgs {
  const void* x;
  long long xs;
  int R, C;
  uint8_t* q;
  long long qs;
  float* scale;
  uint8_t* qt;             // [C, R], or null
  long long qts;
  float* scale_t;
};

// The exponent of a block's scale, from the bits of its largest magnitude;
// kBad for a block with an infinity or a NaN.  TOP: the exponent of the type's
// largest value.
constexpr int kBad = 1 << 20;
template <int TOP>
__device__ __forceinline__ int block_exponent(uint32_t amax) {
  const int k = max((int)((amax + 0x1FFFFFu) >> 23) - 127 - TOP, -126);      // past 1.75: one more
  return amax == 0u ? 0 : amax >= 0x7F800000u ? kBad : k;
}
// 2^k, NaN for kBad
__device__ __forceinline__ float power_of_two(int k) {
  return k >= kBad / 2 ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float((uint32_t)(127 + k) << 23);
}
__device__ __forceinline__ float inverse_of(int k) {
  return k >= kBad / 2 ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float((uint32_t)(127 - k) << 23);
}
template <bool E5>
__device__ __forceinline__ uint32_t fp8x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, E5 ? __NV_E5M2 : __NV_E4M3);
}
template <bool E5>
__device__ __forceinline__ uint32_t fp8x4(uint64_t a, uint64_t b) {
  float a0, a1, b0, b1;
  f2_unpack(a, a0, a1);
  f2_unpack(b, b0, b1);
  return fp8x2<E5>(a0, a1) | (fp8x2<E5>(b0, b1) << 16);
}

// n of the 8 bytes of v, at an address that is a multiple of 8.
__device__ __forceinline__ void store_bytes(uint8_t* p, uint2 v, int n) {
  if (n >= 8) {
    *reinterpret_cast<uint2*>(p) = v;
  } else {
    for (int j = 0; j < n; ++j) p[j] = (uint8_t)((j < 4 ? v.x : v.y) >> (8 * (j & 3)));
  }
}

// 8 columns of a row as they are in memory, and their magnitudes' maxima as
// ordered integers (NaN ranks above infinity, infinity above numbers): two
// columns to a word for bf16, one for fp32.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// W words from each of four rows, which need not lie on 16 bytes: by 16-byte loads of
// what holds them, all of them under way at once, moved into place.  The loads stay
// inside 12 bytes in front of the words and behind them.
template <int W, typename Row>
__device__ __forceinline__ void words_of_four(uintptr_t at, long long pitch, Row* row) {
  uint4 v[4][W / 4 + 1];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4* q = reinterpret_cast<const uint4*>((at + j * pitch) & ~(uintptr_t)15);
#pragma unroll
    for (int i = 0; i < W / 4 + 1; ++i) v[j][i] = __ldg(q + i);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uintptr_t p = at + j * pitch;
    uint32_t s[W + 4];
#pragma unroll
    for (int i = 0; i < W / 4 + 1; ++i) s[4 * i] = v[j][i].x, s[4 * i + 1] = v[j][i].y, s[4 * i + 2] = v[j][i].z, s[4 * i + 3] = v[j][i].w;
    const bool two = p & 8, one = p & 4;
#pragma unroll
    for (int i = 0; i < W + 2; ++i) s[i] = two ? s[i + 2] : s[i];
#pragma unroll
    for (int i = 0; i < W + 1; ++i) s[i] = one ? s[i + 1] : s[i];
#pragma unroll
    for (int i = 0; i < W; ++i) row[j].w[i] = __funnelshift_r(s[i], s[i + 1], (uint32_t)(p & 2) * 8u);
  }
}
template <typename X>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  static constexpr int W = 4;
  uint32_t w[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
  }
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int n) {     // the first n columns, zeros behind
    const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a = 2 * j < n ? __ldg(h + 2 * j) : 0u, b = 2 * j + 1 < n ? __ldg(h + 2 * j + 1) : 0u;
      w[j] = a | (b << 16);
    }
  }
  __device__ __forceinline__ uint32_t mag(int j) const { return w[j] & 0x7FFF7FFFu; }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max_u16x2(a, b); }
  // a word's maxima as fp32 bits: over both columns, of column c of them
  static __device__ __forceinline__ uint32_t whole(uint32_t m) { return max(m << 16, m & 0xFFFF0000u); }
  static __device__ __forceinline__ uint32_t part(uint32_t m, int c) { return c ? m & 0xFFFF0000u : m << 16; }
  // columns 2 j, 2 j + 1
  __device__ __forceinline__ uint64_t pair(int j) const {
    return f2_pack(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
  }
};
template <>
struct Raw<float> {
  static constexpr int W = 8;
  uint32_t w[8];
  __device__ __forceinline__ void load(const float* p) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p)), b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
  __device__ __forceinline__ void load(const float* p, int n) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = j < n ? __ldg(reinterpret_cast<const uint32_t*>(p) + j) : 0u;
  }
  __device__ __forceinline__ uint32_t mag(int j) const { return w[j] & 0x7FFFFFFFu; }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max(a, b); }
  static __device__ __forceinline__ uint32_t whole(uint32_t m) { return m; }
  static __device__ __forceinline__ uint32_t part(uint32_t m, int) { return m; }
  __device__ __forceinline__ uint64_t pair(int j) const {
    return f2_pack(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
  }
};

// Thread: rows 8 u .. 8 u + 7 and columns 8 l .. 8 l + 7 of the tile, u = tid / 16, l = tid % 16.
template <typename X, bool AL, bool E5, bool SQUARE, bool TRANS>
__global__ void __launch_bounds__(kQThreads, AL && sizeof(X) == 2 ? 4 : 2) quantize_kernel(QuantArgs a, int tiles_c) {
  using Row = Raw<X>;
  constexpr int TOP = E5 ? 15 : 8, W = Row::W, WARPS = kQThreads / 32;
  __shared__ uint32_t red[WARPS][16 * W];                 // maxima of a warp's 16 rows, a word of columns each
  __shared__ float inv_t[kTile];
  __shared__ uint2 turn[TRANS ? kTile * 16 : 1];          // [column][8 rows each], its units swapped by column / 8
  cudaTriggerProgrammaticLaunchCompletion();              // a product behind this may come to wait
  const int u = threadIdx.x >> 4, l = threadIdx.x & 15, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tc = (int)(blockIdx.x % tiles_c), tr = (int)(blockIdx.x / tiles_c);
  const int row0 = tr * kTile + 8 * u, col0 = tc * kTile + 8 * l;
  const X* x = static_cast<const X*>(a.x) + (long long)row0 * a.xs + col0;
  Row v[8];
  if (!AL && col0 >= 8 && a.C - col0 >= 16 && row0 + 7 < a.R) {          // 16 bytes of the row on either side
#pragma unroll
    for (int i = 0; i < 8; i += 4)
      words_of_four<W>(reinterpret_cast<uintptr_t>(x + i * a.xs), a.xs * (long long)sizeof(X), &v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (row0 + i < a.R && col0 < a.C) {
        if (AL) v[i].load(x + i * a.xs); else v[i].load(x + i * a.xs, a.C - col0);
      } else {
#pragma unroll
        for (int j = 0; j < W; ++j) v[i].w[j] = 0u;
      }
    }
  }
  float inv[8];
  if constexpr (SQUARE) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < W; ++j) m = Row::larger(m, v[i].mag(j));
    m = __reduce_max_sync(0xffffffffu, Row::whole(m));
    if (lane == 0) red[0][warp] = m;
    __syncthreads();
    m = 0u;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) m = max(m, red[0][w]);
    const int k = block_exponent<TOP>(m);
#pragma unroll
    for (int i = 0; i < 8; ++i) inv[i] = inverse_of(k);
    if (threadIdx.x == 0) {
      a.scale[(long long)tc * ((a.R + kTile - 1) / kTile) + tr] = power_of_two(k);
      if (TRANS) a.scale_t[(long long)tr * tiles_c + tc] = power_of_two(k);
    }
  } else {
    // maxima of 8 rows over 16 lanes: a lane gives away half of its rows at each of three steps
    uint32_t m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t t = v[i].mag(0);
#pragma unroll
      for (int j = 1; j < W; ++j) t = Row::larger(t, v[i].mag(j));
      m[i] = Row::whole(t);
    }
#pragma unroll
    for (int n = 4; n > 0; n >>= 1) {
      const bool up = lane & (2 * n);
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const uint32_t keep = up ? m[i + n] : m[i], give = up ? m[i] : m[i + n];
        m[i] = max(keep, __shfl_xor_sync(0xffffffffu, give, 2 * n));
      }
    }
    m[0] = max(m[0], __shfl_xor_sync(0xffffffffu, m[0], 1));
    const int k = block_exponent<TOP>(m[0]);              // of row l / 2
    if (!(l & 1) && row0 + (l >> 1) < a.R) a.scale[(long long)tc * a.R + row0 + (l >> 1)] = power_of_two(k);
    const float f = inverse_of(k);
#pragma unroll
    for (int i = 0; i < 8; ++i) inv[i] = __shfl_sync(0xffffffffu, f, (lane & 16) + 2 * i);
  }
  if constexpr (TRANS && !SQUARE) {
    uint32_t m[W];
#pragma unroll
    for (int j = 0; j < W; ++j) {
      m[j] = v[0].mag(j);
#pragma unroll
      for (int i = 1; i < 8; ++i) m[j] = Row::larger(m[j], v[i].mag(j));
      m[j] = Row::larger(m[j], __shfl_xor_sync(0xffffffffu, m[j], 16));
    }
    if (lane < 16) {
#pragma unroll
      for (int j = 0; j < W; j += 4) *reinterpret_cast<uint4*>(&red[warp][l * W + j]) = make_uint4(m[j], m[j + 1], m[j + 2], m[j + 3]);
    }
  }
  if (col0 < a.C) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t f = f2_pack(inv[i], inv[i]);
      const uint2 b = make_uint2(fp8x4<E5>(mul2(v[i].pair(0), f), mul2(v[i].pair(1), f)),
                                 fp8x4<E5>(mul2(v[i].pair(2), f), mul2(v[i].pair(3), f)));
      if (row0 + i < a.R) store_bytes(a.q + (long long)(row0 + i) * a.qs + col0, b, a.C - col0);
    }
  }
  if constexpr (TRANS) {
    if constexpr (!SQUARE) {
      __syncthreads();
      constexpr int PER = kTile / (16 * W);               // columns of a word
      if (threadIdx.x < kTile) {
        const int word = threadIdx.x / PER, c = threadIdx.x % PER, col = tc * kTile + (int)threadIdx.x;
        uint32_t m = red[0][word];
#pragma unroll
        for (int w = 1; w < WARPS; ++w) m = Row::larger(m, red[w][word]);
        const int k = block_exponent<TOP>(Row::part(m, c));
        inv_t[threadIdx.x] = inverse_of(k);
        if (col < a.C) a.scale_t[(long long)tr * a.C + col] = power_of_two(k);
      }
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint64_t f = f2_pack(inv[0], inv[0]);
      if constexpr (!SQUARE) f = *reinterpret_cast<const uint64_t*>(&inv_t[8 * l + 2 * j]);
      uint32_t lo[4], hi[4];                              // two rows of column 2 j, of column 2 j + 1
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float a0, a1, b0, b1;
        f2_unpack(mul2(v[2 * i].pair(j), f), a0, a1);
        f2_unpack(mul2(v[2 * i + 1].pair(j), f), b0, b1);
        lo[i] = fp8x2<E5>(a0, b0);
        hi[i] = fp8x2<E5>(a1, b1);
      }
      const int c = 8 * l + 2 * j;
      turn[c * 16 + (u ^ l)] = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
      turn[(c + 1) * 16 + (u ^ l)] = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
    }
    __syncthreads();
    const int r0 = tr * kTile + 8 * l;                    // this thread writes rows r0 .. r0 + 7 of column 16 k + u
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = 16 * k + u, col = tc * kTile + c;
      if (col < a.C && r0 < a.R) store_bytes(a.qt + (long long)col * a.qts + r0, turn[c * 16 + (l ^ (c >> 3))], a.R - r0);
    }
  }
}

template <typename X, bool AL, bool E5>
cudaError_t quant_t(const QuantArgs& a, int rows, cudaStream_t st) {
  const int tc = (a.C + kTile - 1) / kTile;
  const unsigned grid = (unsigned)((long long)tc * ((a.R + kTile - 1) / kTile));
  if (rows == 1) {
    if (a.qt) quantize_kernel<X, AL, E5, false, true><<<grid, kQThreads, 0, st>>>(a, tc);
    else quantize_kernel<X, AL, E5, false, false><<<grid, kQThreads, 0, st>>>(a, tc);
  } else {
    if (a.qt) quantize_kernel<X, AL, E5, true, true><<<grid, kQThreads, 0, st>>>(a, tc);
    else quantize_kernel<X, AL, E5, true, false><<<grid, kQThreads, 0, st>>>(a, tc);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize(const dsv_rows& x, int R, int C, int rows, const dsv_rows& q, float* scale,
                            const dsv_rows& qt, float* scale_t, cudaStream_t st) {
  QuantArgs a;
  a.x = x.ptr;
  a.xs = x.stride;
  a.R = R;
  a.C = C;
  a.q = static_cast<uint8_t*>(q.ptr);
  a.qs = q.stride;
  a.scale = scale;
  a.qt = static_cast<uint8_t*>(qt.ptr);
  a.qts = qt.stride;
  a.scale_t = scale_t;
  const int size = x.type == DSV_F32 ? 4 : 2;
  // 16-byte loads: 8 columns lie inside a row or behind it
  const bool al = C % 8 == 0 && (reinterpret_cast<uintptr_t>(x.ptr) & 15u) == 0 && (x.stride * size) % 16 == 0;
  const bool e5 = q.type == DSV_E5M2;
  if (x.type == DSV_F32) {
    if (al) return e5 ? quant_t<float, true, true>(a, rows, st) : quant_t<float, true, false>(a, rows, st);
    return e5 ? quant_t<float, false, true>(a, rows, st) : quant_t<float, false, false>(a, rows, st);
  }
  if (al) return e5 ? quant_t<__nv_bfloat16, true, true>(a, rows, st) : quant_t<__nv_bfloat16, true, false>(a, rows, st);
  return e5 ? quant_t<__nv_bfloat16, false, true>(a, rows, st) : quant_t<__nv_bfloat16, false, false>(a, rows, st);
}

}  // namespace dsv
