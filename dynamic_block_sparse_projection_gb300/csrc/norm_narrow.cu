// norm_narrow.cu — gradient of the layer norm (norm.cuh) for rows without 16-byte
// accesses: an odd width, an odd start.
//
// One element at a time, or two where all rows start on two elements and the width is
// even; neighbouring threads have neighbouring columns.  2^LG threads have a row, each
// K columns of it, and hold the next row's elements, as they are in memory, while
// they work on this one's.  40000 rows of 1001 (bf16): 71 us, 50 % of the copy bandwidth
// (107 without the next row in hand and a pair of columns to an instruction); 43076 of
// 2310: 201 us, 44 % (334 one element at a time).
#include "norm.cuh"

namespace dsv {

namespace {

__host__ __device__ constexpr int narrow_threads(int lg) { return lg > 8 ? 1 << lg : kNormThreads; }

// V neighbouring elements
template <typename T, int V>
struct alignas(sizeof(T) * V) Few {
  T v[V];
};

// Two sums over the GW threads of a row.
template <int GW>
__device__ __forceinline__ float2 row_sums(float s, float t, float2* parts) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    t += __shfl_xor_sync(0xffffffffu, t, o);
  }
  if constexpr (GW > 32) {
    constexpr int WARPS = GW / 32;
    const int warp = threadIdx.x >> 5, first = warp & ~(WARPS - 1);
    if ((threadIdx.x & 31) == 0) parts[warp] = make_float2(s, t);
    group_sync(threadIdx.x / GW, GW);
    s = parts[first].x, t = parts[first].y;
#pragma unroll
    for (int k = 1; k < WARPS; ++k) s += parts[first + k].x, t += parts[first + k].y;
  }
  return make_float2(s, t);
}

// A thread's K columns are K / V groups of V, GW V columns apart; those of the last
// four (of the last 16 of 32) can lie behind the row.  All arithmetic is on pairs of
// its columns in their order.  dx may be dy or x: a row is read before it is written.
template <typename X, int V, int LG, int K>
__global__ void __launch_bounds__(narrow_threads(LG), LG <= 8 ? 2 : 1)
    norm_bwd_narrow_kernel(const __nv_bfloat16* dy, long long dys, const X* x, long long xs,
                           const float* __restrict__ stats, const float* __restrict__ weight, X* dx, long long dxs,
                           float* parts, int R, NormArgs a, Ctl ctl) {
  constexpr int GW = 1 << LG, THREADS = narrow_threads(LG), GROUPS = THREADS / GW, NE = K / V;
  constexpr int SURE = (K <= 16 ? K - 4 : 16) / V;
  constexpr bool AHEAD = K <= 16;                 // registers for the weight and the next row
  using G = __nv_bfloat16;
  cudaTriggerProgrammaticLaunchCompletion();      // norm_sums_kernel may come to wait
  extern __shared__ float sums[];                 // 2 C floats
  __shared__ float2 slot[2][THREADS / 32];
  check_ptr(a, ctl);
  const int group = threadIdx.x >> LG, gl = threadIdx.x & (GW - 1), left = a.C - V * gl;
  const float inv_c = 1.0f / (float)a.C;
  auto in = [&](int e) { return e < SURE || e * GW * V < left; };
  auto column = [&](int i) { return (i / V * GW + gl) * V + i % V; };
  StreamArgs sa;
  sa.R = R;
  sa.unit = 1;
  sa.teams = GROUPS;
  Walk at(a, sa);
  int parity = 0;
  while (at.next_sequence(group)) {
    const float* w = weight + (long long)at.s * a.C;
    auto weights = [&](int p) {                   // of columns 2 p, 2 p + 1 of the thread's
      const float u = weight != nullptr && in(2 * p / V) ? __ldg(w + column(2 * p)) : 1.f;
      const float v = weight != nullptr && in((2 * p + 1) / V) ? __ldg(w + column(2 * p + 1)) : 1.f;
      return f2_pack(u, v);
    };
    uint64_t dw[K / 2], db[K / 2], wk[AHEAD ? K / 2 : 1];
#pragma unroll
    for (int p = 0; p < K / 2; ++p) {
      dw[p] = db[p] = 0ull;
      if constexpr (AHEAD) wk[p] = weights(p);
    }
    Few<X, V> nx[NE];
    Few<G, V> ng[NE];
    float mean, rstd;
    auto fetch = [&](int row) {
      if (row >= at.q) return;
      const X* px = x + row * xs + V * gl;
      const G* pg = dy + row * dys + V * gl;
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        if (in(e)) {
          nx[e] = *reinterpret_cast<const Few<X, V>*>(px + e * GW * V);
          ng[e] = *reinterpret_cast<const Few<G, V>*>(pg + e * GW * V);
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) nx[e].v[j] = X(0.f), ng[e].v[j] = G(0.f);
        }
      }
      mean = __ldg(stats + row);
      rstd = __ldg(stats + a.T + row);
    };
    if (AHEAD) fetch(at.r);
    for (; at.r < at.q; at.next_unit()) {
      if (!AHEAD) fetch(at.r);
      Few<X, V> cx[NE];
      Few<G, V> cg[NE];
#pragma unroll
      for (int e = 0; e < NE; ++e) cx[e] = nx[e], cg[e] = ng[e];
      const uint64_t off = twice(-mean), rs = twice(rstd);
      if (AHEAD) fetch(at.r + GROUPS);
      auto hat = [&](int p) {                     // x^ of a pair
        const uint64_t v = f2_pack(to_f32(cx[2 * p / V].v[2 * p % V]), to_f32(cx[(2 * p + 1) / V].v[(2 * p + 1) % V]));
        return mul2(add2(v, off), rs);
      };
      auto grad = [&](int p) {
        return f2_pack(to_f32(cg[2 * p / V].v[2 * p % V]), to_f32(cg[(2 * p + 1) / V].v[(2 * p + 1) % V]));
      };
      auto weight_of = [&](int p) {
        if constexpr (AHEAD) return wk[p]; else return weights(p);
      };
      uint64_t s1 = 0ull, s2 = 0ull;
#pragma unroll
      for (int p = 0; p < K / 2; ++p) {
        const uint64_t h = hat(p), g = grad(p), gw = mul2(g, weight_of(p));
        dw[p] = fma2(g, h, dw[p]);
        db[p] = add2(db[p], g);
        s1 = add2(s1, gw);
        s2 = fma2(gw, h, s2);
      }
      const float2 s = row_sums<GW>(both(s1), both(s2), slot[parity]);
      parity ^= 1;
      s1 = twice(-s.x * inv_c), s2 = twice(-s.y * inv_c);
      X* out = dx + at.r * dxs + V * gl;
      Few<X, V> o[NE];
#pragma unroll
      for (int p = 0; p < K / 2; ++p) {
        float u, v;
        f2_unpack(mul2(fma2(hat(p), s2, fma2(grad(p), weight_of(p), s1)), rs), u, v);
        put(&o[2 * p / V].v[2 * p % V], u);
        put(&o[(2 * p + 1) / V].v[(2 * p + 1) % V], v);
      }
#pragma unroll
      for (int e = 0; e < NE; ++e)
        if (in(e)) *reinterpret_cast<Few<X, V>*>(out + e * GW * V) = o[e];
    }
    if (parts == nullptr) continue;
    // the groups' sums, one behind the other
    float* out = parts + 2LL * a.C * ((long long)blockIdx.x + at.s);
    for (int k = 0; k < GROUPS; ++k) {
      if (group == k) {
        float* to = k == GROUPS - 1 ? out : sums;
#pragma unroll
        for (int p = 0; p < K / 2; ++p) {
          float u[2], v[2];
          f2_unpack(dw[p], u[0], u[1]);
          f2_unpack(db[p], v[0], v[1]);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int i = 2 * p + j, c = column(i);
            if (!in(i / V)) continue;
            to[c] = k > 0 ? sums[c] + u[j] : u[j];
            to[a.C + c] = k > 0 ? sums[a.C + c] + v[j] : v[j];
          }
        }
      }
      if (GROUPS > 1) cta_sync();
    }
  }
}

// Threads of a row (2^lg), the fewest that hold it in 16 columns each, to 512; columns of a thread.
struct Narrow {
  int lg, k;
};
Narrow narrow_of(int C) {
  Narrow n = {5, 32};
  while (16 << n.lg < C && n.lg < 9) ++n.lg;
  if (C <= 16 << n.lg) n.k = ceil_div(ceil_div(C, 1 << n.lg), 4) * 4;
  return n;
}

struct Call {
  const dsv_rows& dy;
  const dsv_rows& x;
  const float* stats;
  const float* weight;
  const dsv_rows& dx;
  float* parts;
  int T, R;
  NormArgs a;
  const Ctl& ctl;
  cudaStream_t st;
};
template <typename X, int V, int LG, int K>
cudaError_t narrow_t(const Call& c) {
  const int smem = LG < 8 ? 2 * c.a.C * (int)sizeof(float) : 0;       // at most 16 KB
  norm_bwd_narrow_kernel<X, V, LG, K><<<ceil_div(c.T, c.R), narrow_threads(LG), smem, c.st>>>(
      static_cast<const __nv_bfloat16*>(c.dy.ptr), c.dy.stride, static_cast<const X*>(c.x.ptr), c.x.stride, c.stats, c.weight,
      static_cast<X*>(c.dx.ptr), c.dx.stride, c.parts, c.R, c.a, c.ctl);
  return cudaGetLastError();
}
template <typename X, int V>
cudaError_t narrow_pick(const Narrow& n, const Call& c) {
  switch (100 * n.lg + n.k) {
    case 504: return narrow_t<X, V, 5, 4>(c);
    case 508: return narrow_t<X, V, 5, 8>(c);
    case 512: return narrow_t<X, V, 5, 12>(c);
    case 516: return narrow_t<X, V, 5, 16>(c);
    case 612: return narrow_t<X, V, 6, 12>(c);
    case 616: return narrow_t<X, V, 6, 16>(c);
    case 712: return narrow_t<X, V, 7, 12>(c);
    case 716: return narrow_t<X, V, 7, 16>(c);
    case 812: return narrow_t<X, V, 8, 12>(c);
    case 816: return narrow_t<X, V, 8, 16>(c);
    case 912: return narrow_t<X, V, 9, 12>(c);
    case 916: return narrow_t<X, V, 9, 16>(c);
    case 932: return narrow_t<X, V, 9, 32>(c);
    default: return cudaErrorInvalidValue;         // no width gives another pair
  }
}

}  // namespace

// Rows of a CTA: two CTAs an SM, whole groups' turns.
int norm_narrow_rows(const dsv_norm& p) {
  const int lg = narrow_of(p.C).lg, groups = narrow_threads(lg) >> lg;
  return ceil_div(ceil_div(p.T, 2 * kSMs), groups) * groups;
}

cudaError_t launch_norm_bwd_narrow(const dsv_rows& dy, const dsv_rows& x, const float* stats, const dsv_norm& p,
                                   const int32_t* ptr, const float* weight, const dsv_rows& dx, float* parts, const Ctl& ctl,
                                   cudaStream_t st) {
  const Narrow n = narrow_of(p.C);
  const Call c = {dy, x, stats, weight, dx, parts, p.T, norm_narrow_rows(p), norm_args(p, ptr), ctl, st};
  const bool two = p.C % 2 == 0 && aligned(x, 2) && aligned(dy, 2) && aligned(dx, 2);
  if (x.type == DSV_F32) return two ? narrow_pick<float, 2>(n, c) : narrow_pick<float, 1>(n, c);
  return two ? narrow_pick<__nv_bfloat16, 2>(n, c) : narrow_pick<__nv_bfloat16, 1>(n, c);
}

}  // namespace dsv
