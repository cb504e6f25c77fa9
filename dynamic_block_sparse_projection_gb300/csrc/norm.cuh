// norm.cuh — what the layer norm's kernels share (the way through the rows: the two of the backward).
//
// A video transformer's block normalises the residual stream before its
// attention and scales and shifts the result by vectors that come from the
// clip's conditioning, so the weight changes at clip borders.
//   forward   mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps),
//             y = (x - mu) r w_s + b_s
//   backward  x^ = (x - mu) r, g = dy w_s,
//             dx = r (g - mean(g) - x^ mean(g x^)),
//             dw_s = sum over the rows of s of dy x^,  db_s = sum of dy
// All sums are fp32 in a fixed order.
#pragma once

#include <math.h>

#include "dsv_launch.h"

namespace dsv {
namespace {

constexpr int kNormThreads = 256, kNormWarps = kNormThreads / 32;
constexpr int kSMs = 152;

struct NormArgs {
  int T, C, S;
  int even;                // rows of a sequence where there are no pointers
  int gw;                  // threads that hold a row (streamed backward)
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
  for (int s = threadIdx.x; s < a.S; s += blockDim.x) {
    const int p = a.ptr[s], q = a.ptr[s + 1];
    if (p < 0 || q < p || q > a.T) set_error(ctl, DSV_ERR_BAD_INDEX, (unsigned int)s);
  }
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Barrier of the warps that hold one row.
__device__ __forceinline__ void group_sync(int group, int gw) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(gw) : "memory");
}
// Sum over the GW threads of a row, by way of `parts` (one value of each warp),
// which is free again once the group has met at a barrier after this one.
template <int GW>
__device__ __forceinline__ float row_sum(float v, float* parts) {
#pragma unroll
  for (int o = (GW < 32 ? GW : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (GW > 32) {
    constexpr int WARPS = GW / 32;
    const int warp = threadIdx.x >> 5, first = warp & ~(WARPS - 1);
    if ((threadIdx.x & 31) == 0) parts[warp] = v;
    group_sync(threadIdx.x / GW, GW);
    v = parts[first];
#pragma unroll
    for (int k = 1; k < WARPS; ++k) v += parts[first + k];
  }
  return v;
}
__device__ __forceinline__ uint64_t twice(float v) { return f2_pack(v, v); }
__device__ __forceinline__ float both(uint64_t v) {
  float a, b;
  f2_unpack(v, a, b);
  return a + b;
}

// How a CTA of the backward goes through its rows.
struct StreamArgs {
  int R;                   // rows of a CTA
  int unit, teams, slots;  // rows that a team works on at once; teams; slots of a team's ring
  int one;                 // the rows of x (bit 0) and dy (bit 1) follow each other without gaps
  int sums;                // room in shared memory for sums: none, a team's, all teams'
};

// A team's way through the CTA's rows: the parts of the sequences in them, and in each the team's units.
struct Walk {
  const NormArgs& a;
  const StreamArgs& sa;
  int row0, row1, s, p, q, r;              // sequence, its rows here, the unit's first row
  int slot;
  uint32_t phase;
  __device__ Walk(const NormArgs& args, const StreamArgs& stream)
      : a(args), sa(stream), s(-1), p(0), q(0), r(0), slot(-1), phase(0) {
    row0 = (int)blockIdx.x * sa.R;
    row1 = (int)min((long long)row0 + sa.R, (long long)a.T);
    if (a.ptr == nullptr) {
      if (a.S > 1) s = row0 / a.even - 1;
    } else {                                      // the first sequence that ends behind row0
      int lo = 0, hi = a.S;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.ptr + mid + 1) > row0) hi = mid; else lo = mid + 1;
      }
      s = lo - 1;
    }
  }
  // the next sequence with rows here, and the team's first unit in it
  __device__ bool next_sequence(int team) {
    while (++s < a.S) {
      p = a.ptr == nullptr ? (a.S == 1 ? 0 : s * a.even) : __ldg(a.ptr + s);
      q = a.ptr == nullptr ? (a.S == 1 ? a.T : (s + 1) * a.even) : __ldg(a.ptr + s + 1);
      if (p >= row1) return false;
      p = max(p, row0);
      q = min(q, row1);
      r = p + team * sa.unit;
      if (p < q) return true;
    }
    return false;
  }
  __device__ void next_unit() { r += sa.teams * sa.unit; }
  __device__ void take_slot() {
    if (++slot == sa.slots) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

__device__ __forceinline__ void cta_sync() { asm volatile("bar.sync 0;" ::: "memory"); }

inline int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }
inline NormArgs norm_args(const dsv_norm& p, const int32_t* ptr) {
  NormArgs a;
  a.T = p.T;
  a.C = p.C;
  a.S = p.S;
  a.even = p.S > 0 ? p.T / p.S : 0;
  a.gw = 0;
  a.eps = p.eps;
  a.ptr = ptr;
  return a;
}
inline int size_of(int type) { return type == DSV_F32 ? 4 : 2; }
// Every row starts at a multiple of n elements.
inline bool aligned(const dsv_rows& v, int n) {
  return reinterpret_cast<uintptr_t>(v.ptr) % (n * size_of(v.type)) == 0 && v.stride % n == 0;
}
inline bool wide(const float* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace dsv
