// norm_fwd.cu — layer norm of the rows of [T, C] (norm.cuh).
//
// HBM-bound: 4 bytes an element (bf16) at some 5 operations.  A row belongs to
// 2^LG neighbouring threads, 8 to 256; each holds up to 8 quads of 4 columns (to 16
// of the widest rows) in the registers they come in, so that the mean is taken out
// before the squares are summed and every element is read once, and 32 warps an SM
// hide each other's loads.  Quads, not the 8 columns of a 16-byte load: the fp32
// weight and bias of a warp's quads are then whole lines, not halves of lines.
// What bounds it is the number of instructions, so the place of every quad is known
// when the kernel is compiled (200 us with it worked out at run time).  Two clips of
// 61440 rows of 2048, 1.0 GB: 163 us, 91 % of the copy bandwidth; rings in shared
// memory as the backward has them, 16 warps an SM that wait for two exchanges of
// sums a row, took 219; 16384 rows of 5120: 64 us.
// Rows that do not lie on 4 elements (an odd width, an odd start) are read and
// written one element at a time, neighbouring threads on neighbouring columns.
#include "norm.cuh"

namespace dsv {

namespace {

template <typename X>
struct Quad;
template <>
struct Quad<__nv_bfloat16> {
  uint2 q;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { q = __ldcs(reinterpret_cast<const uint2*>(p)); }
  __device__ __forceinline__ void zero() { q = make_uint2(0u, 0u); }
  __device__ __forceinline__ void set(const __nv_bfloat16* e) {
    q.x = __bfloat16_as_ushort(e[0]) | (uint32_t)__bfloat16_as_ushort(e[1]) << 16;
    q.y = __bfloat16_as_ushort(e[2]) | (uint32_t)__bfloat16_as_ushort(e[3]) << 16;
  }
  __device__ __forceinline__ uint64_t lo() const { return f2_pack(__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xFFFF0000u)); }
  __device__ __forceinline__ uint64_t hi() const { return f2_pack(__uint_as_float(q.y << 16), __uint_as_float(q.y & 0xFFFF0000u)); }
};
template <>
struct Quad<float> {
  ulonglong2 q;
  __device__ __forceinline__ void load(const float* p) {
    const float4 v = __ldcs(reinterpret_cast<const float4*>(p));
    q.x = f2_pack(v.x, v.y);
    q.y = f2_pack(v.z, v.w);
  }
  __device__ __forceinline__ void zero() { q.x = q.y = 0ull; }
  __device__ __forceinline__ void set(const float* e) {
    q.x = f2_pack(e[0], e[1]);
    q.y = f2_pack(e[2], e[3]);
  }
  __device__ __forceinline__ uint64_t lo() const { return q.x; }
  __device__ __forceinline__ uint64_t hi() const { return q.y; }
};


// Only a thread's last two quads can lie behind the row.  x may be y: a row is
// read whole before any of it is written.
template <typename X, int LG, int NQ, bool WIDE>
__global__ void __launch_bounds__(kNormThreads, NQ <= 8 ? 4 : 2)
    norm_fwd_kernel(const X* x, long long xs, __nv_bfloat16* y, long long ys, const float* __restrict__ weight,
                    const float* __restrict__ bias, float* __restrict__ stats, NormArgs a, Ctl ctl) {
  constexpr int GW = 1 << LG, QUAD = WIDE ? 4 : 1, NEXT = WIDE ? 1 : GW;   // columns from a thread's first to the next's, of a quad's
  __shared__ float slot[2][kNormWarps];
  check_ptr(a, ctl);
  const int gl = threadIdx.x & (GW - 1), row = (int)blockIdx.x * (kNormThreads >> LG) + (threadIdx.x >> LG);
  const int left = a.C - QUAD * gl;               // columns from the thread's first
  const float inv_c = 1.0f / (float)a.C;
  auto in = [&](int i, int j) { return i < NQ - 2 || 4 * i * GW + j * NEXT < left; };      // column j of quad i
  Quad<X> v[NQ];
  const X* src = x + row * xs + QUAD * gl;
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    if (WIDE) {
      if (row < a.T && in(i, 0)) v[i].load(src + 4 * i * GW); else v[i].zero();
    } else {
      X e[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) e[j] = row < a.T && in(i, j) ? src[4 * i * GW + j * GW] : X(0.f);
      v[i].set(e);
    }
  }
  const int s = row < a.T ? seq_of(a, row) : -1;
  const uint64_t one = twice(1.0f);
  uint64_t t = 0ull, u = 0ull;
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    t = fma2(v[i].lo(), one, t);
    u = fma2(v[i].hi(), one, u);
  }
  const float mean = row_sum<GW>(both(t) + both(u), slot[0]) * inv_c;
  const uint64_t m2 = twice(-mean);
  t = u = 0ull;
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    uint64_t d = fma2(v[i].lo(), one, m2), e = fma2(v[i].hi(), one, m2);
    if (!WIDE && i >= NQ - 2) {                   // a cut quad
      float d0, d1, e0, e1;
      f2_unpack(d, d0, d1);
      f2_unpack(e, e0, e1);
      d = f2_pack(in(i, 0) ? d0 : 0.f, in(i, 1) ? d1 : 0.f);
      e = f2_pack(in(i, 2) ? e0 : 0.f, in(i, 3) ? e1 : 0.f);
    }
    if (!WIDE || in(i, 0)) {
      t = fma2(d, d, t);
      u = fma2(e, e, u);
    }
  }
  const float rstd = 1.0f / sqrtf(row_sum<GW>(both(t) + both(u), slot[1]) * inv_c + a.eps);
  if (s < 0) return;
  if (gl == 0) {
    stats[row] = mean;
    stats[(long long)a.T + row] = rstd;
  }
  const uint64_t r2 = twice(rstd), off = twice(-mean * rstd);            // x^ = x r - mu r
  __nv_bfloat16* out = y + row * ys + QUAD * gl;
  const float* w = weight + (long long)s * a.C + QUAD * gl;
  const float* b = bias + (long long)s * a.C + QUAD * gl;
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    uint64_t l = fma2(v[i].lo(), r2, off), h = fma2(v[i].hi(), r2, off);
    if (WIDE) {
      if (!in(i, 0)) continue;
      if (weight != nullptr) {
        const ulonglong2 f = __ldg(reinterpret_cast<const ulonglong2*>(w + 4 * i * GW));
        ulonglong2 o;
        o.x = o.y = 0ull;
        if (bias != nullptr) o = __ldg(reinterpret_cast<const ulonglong2*>(b + 4 * i * GW));
        l = fma2(l, f.x, o.x);
        h = fma2(h, f.y, o.y);
      }
    }
    float z[4];
    f2_unpack(l, z[0], z[1]);
    f2_unpack(h, z[2], z[3]);
    if (WIDE) {
      __stcs(reinterpret_cast<uint2*>(out + 4 * i * GW), make_uint2(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3])));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = 4 * i * GW + j * GW;
        if (in(i, j)) {
          if (weight != nullptr) z[j] = fmaf(z[j], __ldg(w + c), bias != nullptr ? __ldg(b + c) : 0.f);
          out[c] = __float2bfloat16_rn(z[j]);
        }
      }
    }
  }
}

template <typename X, int LG, int NQ>
cudaError_t fwd_quad(bool wide_rows, const dsv_rows& x, const NormArgs& a, const float* w, const float* b,
                     const dsv_rows& y, float* stats, const Ctl& ctl, cudaStream_t st) {
  auto kern = wide_rows ? norm_fwd_kernel<X, LG, NQ, true> : norm_fwd_kernel<X, LG, NQ, false>;
  kern<<<ceil_div(a.T, kNormThreads >> LG), kNormThreads, 0, st>>>(static_cast<const X*>(x.ptr), x.stride,
                                                                  static_cast<__nv_bfloat16*>(y.ptr), y.stride, w, b,
                                                                  stats, a, ctl);
  return cudaGetLastError();
}
// Threads of a row: the fewest that hold it in 8 quads each (10 of 128 threads), 8 to 256.
template <typename X>
cudaError_t fwd_pick(bool v, const dsv_rows& x, const NormArgs& a, const float* w, const float* b, const dsv_rows& y,
                     float* stats, const Ctl& ctl, cudaStream_t st) {
  const int quads = ceil_div(a.C, 4);
  int lg = 3;
  while (lg < 8 && quads > (lg == 7 ? 10 : 8) << lg) ++lg;        // 10: 5120 columns in 128 threads, 77 -> 69 us
  switch (100 * lg + ceil_div(ceil_div(quads, 1 << lg), 2) * 2) {
    case 302: return fwd_quad<X, 3, 2>(v, x, a, w, b, y, stats, ctl, st);
    case 304: return fwd_quad<X, 3, 4>(v, x, a, w, b, y, stats, ctl, st);
    case 306: return fwd_quad<X, 3, 6>(v, x, a, w, b, y, stats, ctl, st);
    case 308: return fwd_quad<X, 3, 8>(v, x, a, w, b, y, stats, ctl, st);
    case 406: return fwd_quad<X, 4, 6>(v, x, a, w, b, y, stats, ctl, st);
    case 408: return fwd_quad<X, 4, 8>(v, x, a, w, b, y, stats, ctl, st);
    case 506: return fwd_quad<X, 5, 6>(v, x, a, w, b, y, stats, ctl, st);
    case 508: return fwd_quad<X, 5, 8>(v, x, a, w, b, y, stats, ctl, st);
    case 606: return fwd_quad<X, 6, 6>(v, x, a, w, b, y, stats, ctl, st);
    case 608: return fwd_quad<X, 6, 8>(v, x, a, w, b, y, stats, ctl, st);
    case 706: return fwd_quad<X, 7, 6>(v, x, a, w, b, y, stats, ctl, st);
    case 708: return fwd_quad<X, 7, 8>(v, x, a, w, b, y, stats, ctl, st);
    case 710: return fwd_quad<X, 7, 10>(v, x, a, w, b, y, stats, ctl, st);
    case 806: return fwd_quad<X, 8, 6>(v, x, a, w, b, y, stats, ctl, st);
    case 808: return fwd_quad<X, 8, 8>(v, x, a, w, b, y, stats, ctl, st);
    case 810: return fwd_quad<X, 8, 10>(v, x, a, w, b, y, stats, ctl, st);
    case 812: return fwd_quad<X, 8, 12>(v, x, a, w, b, y, stats, ctl, st);
    case 814: return fwd_quad<X, 8, 14>(v, x, a, w, b, y, stats, ctl, st);
    case 816: return fwd_quad<X, 8, 16>(v, x, a, w, b, y, stats, ctl, st);
    default: return cudaErrorInvalidValue;         // no width gives another pair
  }
}

}  // namespace

cudaError_t launch_norm_fwd(const dsv_rows& x, const dsv_norm& p, const int32_t* ptr, const float* weight,
                            const float* bias, const dsv_rows& y, float* stats, const Ctl& ctl, cudaStream_t st) {
  const NormArgs a = norm_args(p, ptr);
  const bool v = p.C % 4 == 0 && aligned(x, 4) && aligned(y, 4) && wide(weight) && wide(bias);
  return x.type == DSV_F32 ? fwd_pick<float>(v, x, a, weight, bias, y, stats, ctl, st)
                           : fwd_pick<__nv_bfloat16>(v, x, a, weight, bias, y, stats, ctl, st);
}

}  // namespace dsv
