// norm.cu — layer norm of the rows of [T, C], forward and backward, with one
// weight and bias or a row of them for each sequence of tokens.
//
// A video transformer's block normalises the residual stream before its
// attention and scales and shifts the result by vectors that come from the
// clip's conditioning, so the weight changes at clip borders.
//   forward   mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps),
//             y = (x - mu) r w_s + b_s
//   backward  x^ = (x - mu) r, g = dy w_s,
//             dx = r (g - mean(g) - x^ mean(g x^)),
//             dw_s = sum over the rows of s of dy x^,  db_s = sum of dy
// A row stays in the registers of the 1 to 8 warps that hold it, so the mean is
// taken out before the squares are summed (an offset of the row costs no
// digits) and every element is read once.  All sums are fp32 in a fixed order.
#include <math.h>

#include "dsv_launch.h"

namespace dsv {

namespace {

constexpr int kNormThreads = 256, kNormWarps = kNormThreads / 32;

struct NormArgs {
  int T, C, S;
  int even;                // rows of a sequence where there are no pointers
  int gw;                  // threads that hold a row: 32, 64, 128 or 256
  float eps;
  const int32_t* ptr;      // [S + 1], or null
};

// The sequence of a row, -1 for a row outside all of them.
__device__ __forceinline__ int seq_of(const NormArgs& a, int row) {
  if (a.ptr == nullptr) return a.S == 1 ? 0 : row / a.even;
  int lo = 0, hi = a.S;                          // the last s with ptr[s] <= row
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(a.ptr + mid) <= row) lo = mid; else hi = mid;
  }
  return (__ldg(a.ptr + lo) <= row && row < __ldg(a.ptr + lo + 1)) ? lo : -1;
}
__device__ __forceinline__ void check_ptr(const NormArgs& a, const Ctl& ctl) {
  if (a.ptr == nullptr || blockIdx.x != 0) return;
  for (int s = threadIdx.x; s < a.S; s += kNormThreads) {
    const int p = a.ptr[s], q = a.ptr[s + 1];
    if (p < 0 || q < p || q > a.T) set_error(ctl, DSV_ERR_BAD_INDEX, (unsigned int)s);
  }
}

// Columns of a thread: chunk i holds 8 of them.  With 16-byte accesses (AL) a
// chunk is 8 neighbours; without, neighbouring threads take neighbouring
// columns, so that 2- and 4-byte accesses stay coalesced.
template <bool AL>
__device__ __forceinline__ int column(int i, int j, int gw, int gl) {
  return AL ? 8 * (i * gw + gl) + j : (8 * i + j) * gw + gl;
}

template <bool AL>
__device__ __forceinline__ void load8(const __nv_bfloat16* row, int i, int gw, int gl, int C, float* v) {
  if constexpr (AL) {
    const int c = column<true>(i, 0, gw, gl);
    const uint4 q = c < C ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0, 0, 0, 0);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = column<false>(i, j, gw, gl);
      v[j] = c < C ? __bfloat162float(row[c]) : 0.f;
    }
  }
}
template <bool AL>
__device__ __forceinline__ void load8(const float* row, int i, int gw, int gl, int C, float* v) {
  if constexpr (AL) {
    const int c = column<true>(i, 0, gw, gl);
    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 p = c < C ? *reinterpret_cast<const float4*>(row + c) : z;
    const float4 q = c < C ? *reinterpret_cast<const float4*>(row + c + 4) : z;
    v[0] = p.x, v[1] = p.y, v[2] = p.z, v[3] = p.w, v[4] = q.x, v[5] = q.y, v[6] = q.z, v[7] = q.w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = column<false>(i, j, gw, gl);
      v[j] = c < C ? row[c] : 0.f;
    }
  }
}
template <bool AL>
__device__ __forceinline__ void store8(__nv_bfloat16* row, int i, int gw, int gl, int C, const float* v) {
  if constexpr (AL) {
    const int c = column<true>(i, 0, gw, gl);
    if (c < C)
      *reinterpret_cast<uint4*>(row + c) =
          make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = column<false>(i, j, gw, gl);
      if (c < C) row[c] = __float2bfloat16_rn(v[j]);
    }
  }
}
template <bool AL>
__device__ __forceinline__ void store8(float* row, int i, int gw, int gl, int C, const float* v) {
  if constexpr (AL) {
    const int c = column<true>(i, 0, gw, gl);
    if (c < C) {
      *reinterpret_cast<float4*>(row + c) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(row + c + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = column<false>(i, j, gw, gl);
      if (c < C) row[c] = v[j];
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Barrier of the warps that hold one row.
__device__ __forceinline__ void group_sync(int group, int gw) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(gw) : "memory");
}
// Sum over the threads of a row.  `slot` holds one value of each warp; it is
// free again once the group has met at a barrier after this one.
__device__ __forceinline__ float group_sum(float v, float* slot, int group, int gw) {
  v = warp_sum(v);
  if (gw == 32) return v;
  const int warp = threadIdx.x >> 5, n = gw >> 5, first = group * n;
  if ((threadIdx.x & 31) == 0) slot[warp] = v;
  group_sync(group, gw);
  float t = 0.f;
  for (int k = 0; k < n; ++k) t += slot[first + k];
  return t;
}

// x may be y (each element is read and written by one thread).
template <typename X, int CH, bool AL>
__global__ void __launch_bounds__(kNormThreads) norm_fwd_kernel(const X* x, long long xs, __nv_bfloat16* y, long long ys,
                                                                 const float* __restrict__ weight,
                                                                 const float* __restrict__ bias, float* __restrict__ stats,
                                                                 NormArgs a, Ctl ctl) {
  __shared__ float slot[2][kNormWarps];
  check_ptr(a, ctl);
  const int gw = a.gw, groups = kNormThreads / gw, group = threadIdx.x / gw, gl = threadIdx.x % gw;
  const float inv_c = 1.0f / (float)a.C;
  for (long long r = (long long)blockIdx.x * groups + group; r < a.T; r += (long long)gridDim.x * groups) {
    const int row = (int)r;
    float v[CH * 8];
#pragma unroll
    for (int i = 0; i < CH; ++i) load8<AL>(x + row * xs, i, gw, gl, a.C, v + 8 * i);
    const int s = seq_of(a, row);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < CH * 8; ++i) sum += v[i];
    const float mean = group_sum(sum, slot[0], group, gw) * inv_c;
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[8 * i + j] -= mean;
        sq += column<AL>(i, j, gw, gl) < a.C ? v[8 * i + j] * v[8 * i + j] : 0.f;
      }
    const float rstd = 1.0f / sqrtf(group_sum(sq, slot[1], group, gw) * inv_c + a.eps);
    if (s < 0) continue;
    if (gl == 0) {
      stats[row] = mean;
      stats[(long long)a.T + row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      float w[8], b[8];
      if (weight != nullptr) load8<AL>(weight + (long long)s * a.C, i, gw, gl, a.C, w);
      if (bias != nullptr) load8<AL>(bias + (long long)s * a.C, i, gw, gl, a.C, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float t = v[8 * i + j] * rstd;
        if (weight != nullptr) t *= w[j];
        if (bias != nullptr) t += b[j];
        v[8 * i + j] = t;
      }
      store8<AL>(y + row * ys, i, gw, gl, a.C, v + 8 * i);
    }
  }
}

// A CTA takes the rows [R blockIdx, R (blockIdx + 1)) and walks through the
// sequences in them; the sums of the part of sequence s that it holds go to
// slot blockIdx + s of the workspace (2 C floats: dw, db).  The next part has a
// later CTA or a later sequence, so no two parts share a slot.
// dx may be dy or x.
template <typename X, int CH, bool AL>
__global__ void __launch_bounds__(kNormThreads) norm_bwd_kernel(const __nv_bfloat16* dy, long long dys, const X* x,
                                                                 long long xs, const float* __restrict__ stats,
                                                                 const float* __restrict__ weight, X* dx, long long dxs,
                                                                 float* __restrict__ parts, int R, NormArgs a, Ctl ctl) {
  extern __shared__ float sums[];                 // 2 C floats
  __shared__ float slot[2][2][kNormWarps];
  check_ptr(a, ctl);
  const int gw = a.gw, groups = kNormThreads / gw, group = threadIdx.x / gw, gl = threadIdx.x % gw;
  const float inv_c = 1.0f / (float)a.C;
  const int row0 = (int)blockIdx.x * R, row1 = (long long)row0 + R < a.T ? row0 + R : a.T;
  int s = 0;
  if (a.ptr == nullptr) {
    s = a.S == 1 ? 0 : row0 / a.even;
  } else {                                        // the first sequence that ends behind row0
    int lo = 0, hi = a.S;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(a.ptr + mid + 1) > row0) hi = mid; else lo = mid + 1;
    }
    s = lo;
  }
  int parity = 0;
  for (; s < a.S; ++s) {
    int p = a.ptr == nullptr ? (a.S == 1 ? 0 : s * a.even) : __ldg(a.ptr + s);
    int q = a.ptr == nullptr ? (a.S == 1 ? a.T : (s + 1) * a.even) : __ldg(a.ptr + s + 1);
    if (p >= row1) break;
    p = max(p, row0);
    q = min(q, row1);
    if (q <= p) continue;
    float dw[CH * 8], db[CH * 8];
#pragma unroll
    for (int i = 0; i < CH * 8; ++i) dw[i] = db[i] = 0.f;
    for (int row = p + group; row < q; row += groups) {
      float h[CH * 8], g[CH * 8];
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        load8<AL>(x + row * xs, i, gw, gl, a.C, h + 8 * i);
        load8<AL>(dy + row * dys, i, gw, gl, a.C, g + 8 * i);
      }
      const float mean = __ldg(stats + row), rstd = __ldg(stats + (long long)a.T + row);
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        float w[8];
        if (weight != nullptr) load8<AL>(weight + (long long)s * a.C, i, gw, gl, a.C, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int k = 8 * i + j;
          const bool in = column<AL>(i, j, gw, gl) < a.C;
          h[k] = in ? (h[k] - mean) * rstd : 0.f;
          dw[k] += g[k] * h[k];
          db[k] += g[k];
          if (weight != nullptr) g[k] *= w[j];
          s1 += g[k];
          s2 += g[k] * h[k];
        }
      }
      s1 = warp_sum(s1);
      s2 = warp_sum(s2);
      if (gw > 32) {
        const int warp = threadIdx.x >> 5, n = gw >> 5, first = group * n;
        if ((threadIdx.x & 31) == 0) {
          slot[parity][0][warp] = s1;
          slot[parity][1][warp] = s2;
        }
        group_sync(group, gw);
        s1 = s2 = 0.f;
        for (int k = 0; k < n; ++k) {
          s1 += slot[parity][0][first + k];
          s2 += slot[parity][1][first + k];
        }
        parity ^= 1;
      }
      s1 *= inv_c;
      s2 *= inv_c;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[8 * i + j] = rstd * (g[8 * i + j] - s1 - h[8 * i + j] * s2);
        store8<AL>(dx + row * dxs, i, gw, gl, a.C, g + 8 * i);
      }
    }
    if (parts == nullptr) continue;
    // the groups' sums, one group after the other
    float* out = parts + 2LL * a.C * ((long long)blockIdx.x + s);
    for (int k = 0; k < groups - 1; ++k) {
      if (group == k) {
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int c = column<AL>(i, j, gw, gl);
            if (c < a.C) {
              sums[c] = k > 0 ? sums[c] + dw[8 * i + j] : dw[8 * i + j];
              sums[a.C + c] = k > 0 ? sums[a.C + c] + db[8 * i + j] : db[8 * i + j];
            }
          }
      }
      __syncthreads();
    }
    if (group == groups - 1) {
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int c = column<AL>(i, j, gw, gl);
          if (c < a.C) {
            out[c] = groups > 1 ? sums[c] + dw[8 * i + j] : dw[8 * i + j];
            out[a.C + c] = groups > 1 ? sums[a.C + c] + db[8 * i + j] : db[8 * i + j];
          }
        }
    }
    __syncthreads();
  }
}

// dw_s, db_s: the parts of sequence s, in the order of their rows.  A CTA takes
// 32 columns; its warps take every eighth part.
__global__ void __launch_bounds__(kNormThreads) norm_sums_kernel(const float* __restrict__ parts, int R,
                                                                  float* __restrict__ dweight, float* __restrict__ dbias,
                                                                  NormArgs a) {
  __shared__ float sum[kNormWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c2 = (int)blockIdx.x * 32 + lane, s = (int)blockIdx.y;       // column of dw, then of db
  int p = a.ptr == nullptr ? (a.S == 1 ? 0 : s * a.even) : a.ptr[s];
  int q = a.ptr == nullptr ? (a.S == 1 ? a.T : (s + 1) * a.even) : a.ptr[s + 1];
  p = max(p, 0);
  q = min(q, a.T);
  float t = 0.f;
  if (p < q && c2 < 2 * a.C) {
    const int last = (q - 1) / R;
    for (int k = p / R + warp; k <= last; k += kNormWarps) t += parts[2LL * a.C * (k + s) + c2];
  }
  sum[warp][lane] = t;
  __syncthreads();
  if (warp == 0 && c2 < 2 * a.C) {
    t = 0.f;
#pragma unroll
    for (int k = 0; k < kNormWarps; ++k) t += sum[k][lane];
    float* out = c2 < a.C ? dweight + (long long)s * a.C + c2 : dbias + (long long)s * a.C + (c2 - a.C);
    *out = t;
  }
}

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

// Chunks a thread holds and threads a row takes.
void shape_of(int C, int* ch, int* gw) {
  const int chunks = ceil_div(C, 8);
  *gw = 32;
  while (*gw < kNormThreads && chunks > 4 * *gw) *gw *= 2;
  *ch = 1;
  while (*ch * *gw < chunks) *ch *= 2;
}
NormArgs norm_args(const dsv_norm& p, const int32_t* ptr) {
  NormArgs a;
  a.T = p.T;
  a.C = p.C;
  a.S = p.S;
  a.even = p.S > 0 ? p.T / p.S : 0;
  a.eps = p.eps;
  a.ptr = ptr;
  return a;
}
bool wide(const dsv_rows& v, int size) {
  return (reinterpret_cast<uintptr_t>(v.ptr) & 15u) == 0 && (v.stride * size) % 16 == 0;
}
bool wide(const float* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
int size_of(int type) { return type == DSV_F32 ? 4 : 2; }

// Rows of a CTA of the backward: as many CTAs as fill the SMs four times.
constexpr int kNormBwdCtas = 4 * 152;
int bwd_rows(const dsv_norm& p) {
  int ch, gw;
  shape_of(p.C, &ch, &gw);
  const int groups = kNormThreads / gw, r = ceil_div(p.T, kNormBwdCtas);
  return ceil_div(r, groups) * groups;
}

template <typename X, int CH, bool AL>
cudaError_t fwd_t(const dsv_rows& x, const NormArgs& a, const float* w, const float* b, const dsv_rows& y, float* stats,
                  const Ctl& ctl, cudaStream_t st) {
  const int groups = kNormThreads / a.gw, grid = min(ceil_div(a.T, groups), 152 * 8);
  norm_fwd_kernel<X, CH, AL><<<grid, kNormThreads, 0, st>>>(static_cast<const X*>(x.ptr), x.stride,
                                                           static_cast<__nv_bfloat16*>(y.ptr), y.stride, w, b, stats, a, ctl);
  return cudaGetLastError();
}
template <typename X, int CH, bool AL>
cudaError_t bwd_t(const dsv_rows& dy, const dsv_rows& x, const float* stats, const NormArgs& a, const float* w,
                  const dsv_rows& dx, float* parts, int R, const Ctl& ctl, cudaStream_t st) {
  const int smem = 2 * a.C * (int)sizeof(float);
  auto kern = norm_bwd_kernel<X, CH, AL>;
  const int groups = kNormThreads / a.gw;
  cudaError_t e;
  if (groups > 1 && smem > 40 * 1024 &&
      (e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
    return e;
  kern<<<ceil_div(a.T, R), kNormThreads, groups > 1 ? smem : 0, st>>>(
      static_cast<const __nv_bfloat16*>(dy.ptr), dy.stride, static_cast<const X*>(x.ptr), x.stride, stats, w,
      static_cast<X*>(dx.ptr), dx.stride, parts, R, a, ctl);
  return cudaGetLastError();
}
// The instance for a call's type, width and alignment.
#define NORM_PICK(fn, type, ch, al, ...)                                                               \
  (type == DSV_F32                                                                                      \
       ? (al ? (ch == 1 ? fn<float, 1, true>(__VA_ARGS__) : ch == 2 ? fn<float, 2, true>(__VA_ARGS__)   \
                : ch == 4 ? fn<float, 4, true>(__VA_ARGS__) : fn<float, 8, true>(__VA_ARGS__))          \
             : (ch == 1 ? fn<float, 1, false>(__VA_ARGS__) : ch == 2 ? fn<float, 2, false>(__VA_ARGS__) \
                : ch == 4 ? fn<float, 4, false>(__VA_ARGS__) : fn<float, 8, false>(__VA_ARGS__)))       \
       : (al ? (ch == 1 ? fn<__nv_bfloat16, 1, true>(__VA_ARGS__)                                       \
                : ch == 2 ? fn<__nv_bfloat16, 2, true>(__VA_ARGS__)                                     \
                : ch == 4 ? fn<__nv_bfloat16, 4, true>(__VA_ARGS__) : fn<__nv_bfloat16, 8, true>(__VA_ARGS__)) \
             : (ch == 1 ? fn<__nv_bfloat16, 1, false>(__VA_ARGS__)                                      \
                : ch == 2 ? fn<__nv_bfloat16, 2, false>(__VA_ARGS__)                                    \
                : ch == 4 ? fn<__nv_bfloat16, 4, false>(__VA_ARGS__) : fn<__nv_bfloat16, 8, false>(__VA_ARGS__))))

}  // namespace

cudaError_t launch_norm_fwd(const dsv_rows& x, const dsv_norm& p, const int32_t* ptr, const float* weight,
                            const float* bias, const dsv_rows& y, float* stats, const Ctl& ctl, cudaStream_t st) {
  NormArgs a = norm_args(p, ptr);
  int ch;
  shape_of(p.C, &ch, &a.gw);
  const bool al = p.C % 8 == 0 && wide(x, size_of(x.type)) && wide(y, 2) && wide(weight) && wide(bias);
  return NORM_PICK(fwd_t, x.type, ch, al, x, a, weight, bias, y, stats, ctl, st);
}

size_t norm_bwd_ws_bytes(const dsv_norm& p) {
  const int R = bwd_rows(p);
  return ((size_t)ceil_div(p.T, R) + p.S) * 2 * p.C * sizeof(float);
}

cudaError_t launch_norm_bwd(const dsv_rows& dy, const dsv_rows& x, const float* stats, const dsv_norm& p,
                            const int32_t* ptr, const float* weight, const dsv_rows& dx, float* dweight, float* dbias,
                            void* ws, const Ctl& ctl, cudaStream_t st) {
  NormArgs a = norm_args(p, ptr);
  int ch;
  shape_of(p.C, &ch, &a.gw);
  const int R = bwd_rows(p);
  const bool al = p.C % 8 == 0 && wide(x, size_of(x.type)) && wide(dy, 2) && wide(dx, size_of(dx.type)) && wide(weight);
  float* parts = dweight != nullptr ? static_cast<float*>(ws) : nullptr;
  cudaError_t e = NORM_PICK(bwd_t, x.type, ch, al, dy, x, stats, a, weight, dx, parts, R, ctl, st);
  if (e != cudaSuccess || parts == nullptr) return e;
  norm_sums_kernel<<<dim3(ceil_div(2LL * p.C, 32), p.S), kNormThreads, 0, st>>>(parts, R, dweight, dbias, a);
  return cudaGetLastError();
}

}  // namespace dsv
