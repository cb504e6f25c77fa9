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
constexpr int kSMs = 152;
constexpr int kStreamBytes = 220 * 1024, kFwdChunks = 8, kBwdChunks = 4;

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
  for (int s = threadIdx.x; s < a.S; s += blockDim.x) {
    const int p = a.ptr[s], q = a.ptr[s + 1];
    if (p < 0 || q < p || q > a.T) set_error(ctl, DSV_ERR_BAD_INDEX, (unsigned int)s);
  }
}

// ---------------------------------------------------------------------------
// Rows without 16-byte accesses (an odd width, an odd start): one element at a
// time, neighbouring threads on neighbouring columns
// ---------------------------------------------------------------------------
__device__ __forceinline__ int column(int i, int j, int gw, int gl) { return (8 * i + j) * gw + gl; }

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
template <typename X>
__device__ __forceinline__ void load8(const X* row, int i, int gw, int gl, int C, float* v) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int c = column(i, j, gw, gl);
    v[j] = c < C ? to_f32(row[c]) : 0.f;
  }
}
template <typename X>
__device__ __forceinline__ void store8(X* row, int i, int gw, int gl, int C, const float* v) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int c = column(i, j, gw, gl);
    if (c < C) put(row + c, v[j]);
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
template <typename X, int CH>
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
    for (int i = 0; i < CH; ++i) load8(x + row * xs, i, gw, gl, a.C, v + 8 * i);
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
        sq += column(i, j, gw, gl) < a.C ? v[8 * i + j] * v[8 * i + j] : 0.f;
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
      if (weight != nullptr) load8(weight + (long long)s * a.C, i, gw, gl, a.C, w);
      if (bias != nullptr) load8(bias + (long long)s * a.C, i, gw, gl, a.C, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float t = v[8 * i + j] * rstd;
        if (weight != nullptr) t *= w[j];
        if (bias != nullptr) t += b[j];
        v[8 * i + j] = t;
      }
      store8(y + row * ys, i, gw, gl, a.C, v + 8 * i);
    }
  }
}

// A CTA takes the rows [R blockIdx, R (blockIdx + 1)) and walks through the
// sequences in them; the sums of the part of sequence s that it holds go to
// slot blockIdx + s of the workspace (2 C floats: dw, db).  The next part has a
// later CTA or a later sequence, so no two parts share a slot.
// dx may be dy or x.
template <typename X, int CH>
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
        load8(x + row * xs, i, gw, gl, a.C, h + 8 * i);
        load8(dy + row * dys, i, gw, gl, a.C, g + 8 * i);
      }
      const float mean = __ldg(stats + row), rstd = __ldg(stats + (long long)a.T + row);
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        float w[8];
        if (weight != nullptr) load8(weight + (long long)s * a.C, i, gw, gl, a.C, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int k = 8 * i + j;
          const bool in = column(i, j, gw, gl) < a.C;
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
        store8(dx + row * dxs, i, gw, gl, a.C, g + 8 * i);
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
            const int c = column(i, j, gw, gl);
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
          const int c = column(i, j, gw, gl);
          if (c < a.C) {
            out[c] = groups > 1 ? sums[c] + dw[8 * i + j] : dw[8 * i + j];
            out[a.C + c] = groups > 1 ? sums[a.C + c] + db[8 * i + j] : db[8 * i + j];
          }
        }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Rows with 16-byte accesses: streamed through shared memory
// ---------------------------------------------------------------------------
// A row belongs to `gw` neighbouring threads, 2 to 512 of them, CH chunks of 8
// columns each: wide rows take several warps, narrow ones a part of one, so
// that the exchange of sums and the rest of a row's fixed cost (some 150
// instructions) are spread over at least 32 columns a thread.  The warps that
// share a row, or the one warp that holds several, are a team.  Every team has
// a ring of slots that its first warp fills by bulk copies, so that bytes in
// flight cost no registers and no team waits for another.  A CTA, one an SM,
// takes neighbouring rows: the weight and bias of a sequence are brought into
// shared memory once for all of its rows there, and a thread keeps the sums of
// dweight and dbias of its columns in registers.
constexpr int kTeamThreads = 512, kTeamWarps = kTeamThreads / 32, kMaxSlots = 8;

struct StreamArgs {
  int R;                   // rows of a CTA
  int unit, teams, slots;  // rows that a team works on at once; teams; slots of a team's ring
  int one;                 // the rows of x (bit 0) and dy (bit 1) follow each other without gaps
  int local, sums;         // weight and bias, and the teams' joined sums, in shared memory
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

// 8 columns as four pairs of fp32
__device__ __forceinline__ void pairs8(const __nv_bfloat16* p, uint64_t* v) {
  const uint4 q = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = f2_pack(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
}
__device__ __forceinline__ void pairs8(const float* p, uint64_t* v) {
  const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(p), b = *reinterpret_cast<const ulonglong2*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}
__device__ __forceinline__ void store_pairs8(__nv_bfloat16* p, const uint64_t* v) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a, b;
    f2_unpack(v[j], a, b);
    w[j] = pack_bf16x2(a, b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_pairs8(float* p, const uint64_t* v) {
  *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(v[0], v[1]);
  *reinterpret_cast<ulonglong2*>(p + 4) = make_ulonglong2(v[2], v[3]);
}
__device__ __forceinline__ uint64_t twice(float v) { return f2_pack(v, v); }
__device__ __forceinline__ float both(uint64_t v) {
  float a, b;
  f2_unpack(v, a, b);
  return a + b;
}
// A vector of fp32 columns in shared memory: the first halves of all chunks,
// then the second halves, so that neighbouring threads read neighbouring 16 bytes.
__device__ __forceinline__ void local8(const float* p, int chunk, int chunks, uint64_t* v) {
  const ulonglong2 a = reinterpret_cast<const ulonglong2*>(p)[chunk], b = reinterpret_cast<const ulonglong2*>(p)[chunks + chunk];
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}
__device__ __forceinline__ void make_local(float* to, const float* from, int chunks) {
  for (int k = threadIdx.x; k < 2 * chunks; k += kTeamThreads)
    reinterpret_cast<float4*>(to)[(k & 1) * chunks + (k >> 1)] = reinterpret_cast<const float4*>(from)[k];
}
__device__ __forceinline__ void cta_sync() { asm volatile("bar.sync 0;" ::: "memory"); }

// Sums of N values over the threads of a row, N = 1, 2 or 4.  Over whole
// warps, a lane gives away half of its values at each of the first steps, so
// that four values cost 6 shuffles and not 20.
template <int N>
__device__ __forceinline__ void group_sums(float* v, float (*slot)[4], int group, int gw) {
  const int lane = threadIdx.x & 31;
  if (gw < 32) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
      if (o < gw) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
      }
    return;
  }
  float t;
  if constexpr (N == 4) {
    const bool up = lane & 16;
    const float k0 = up ? v[2] : v[0], k1 = up ? v[3] : v[1], g0 = up ? v[0] : v[2], g1 = up ? v[1] : v[3];
    const float a = k0 + __shfl_xor_sync(0xffffffffu, g0, 16), b = k1 + __shfl_xor_sync(0xffffffffu, g1, 16);
    const bool up2 = lane & 8;
    t = (up2 ? b : a) + __shfl_xor_sync(0xffffffffu, up2 ? a : b, 8);
  } else if constexpr (N == 2) {
    const bool up = lane & 16;
    t = (up ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[1], 16);
    t += __shfl_xor_sync(0xffffffffu, t, 8);
  } else {
    t = v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
    t += __shfl_xor_sync(0xffffffffu, t, 8);
  }
  t += __shfl_xor_sync(0xffffffffu, t, 4);
  t += __shfl_xor_sync(0xffffffffu, t, 2);
  t += __shfl_xor_sync(0xffffffffu, t, 1);
  constexpr int SPAN = 32 / N;                    // value i sits in lanes i SPAN ..
  if (gw == 32) {
    if constexpr (N == 1) {
      v[0] = t;
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, t, i * SPAN);
    }
    return;
  }
  const int warp = threadIdx.x >> 5, n = gw >> 5, first = group * n;
  if (lane % SPAN == 0) slot[warp][lane / SPAN] = t;
  group_sync(group, gw);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = slot[first][i] + slot[first + 1][i];
  for (int k = 2; k < n; k += 2) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += slot[first + k][i] + slot[first + k + 1][i];
  }
}

// A team's first warp brings in its rows, unit by unit.
template <typename X, bool BWD>
struct Loader {
  const X* x;
  long long xs;
  const __nv_bfloat16* dy;
  long long dys;
  uint8_t* ring;                                  // the team's
  uint64_t* full;
  Walk at;
  int team;
  bool more;
  uint32_t xb, yb, issued;
  __device__ Loader(const X* x_, long long xs_, const __nv_bfloat16* dy_, long long dys_, uint8_t* ring_, uint64_t* full_,
                    const NormArgs& a, const StreamArgs& sa, int team_)
      : x(x_), xs(xs_), dy(dy_), dys(dys_), ring(ring_), full(full_), at(a, sa), team(team_), issued(0) {
    xb = (uint32_t)a.C * sizeof(X);
    yb = BWD ? (uint32_t)a.C * 2u : 0u;
    more = at.next_sequence(team);
    skip();
  }
  __device__ void skip() {
    while (more && at.r >= at.q) more = at.next_sequence(team);
  }
  // the next unit, into a slot that is free
  __device__ void load() {
    if (!more) return;
    const StreamArgs& sa = at.sa;
    const int lane = threadIdx.x & 31;
    at.take_slot();
    const int rows = min(sa.unit, at.q - at.r);
    uint64_t* bar = full + at.slot;
    uint8_t* dst = ring + (size_t)at.slot * sa.unit * (xb + yb);
    uint8_t* dst2 = dst + (size_t)sa.unit * xb;
    if (lane == 0) {
      mbar_arrive_expect_tx(bar, (uint32_t)rows * (xb + yb));
      if (sa.one & 1) bulk_load(dst, x + at.r * xs, (uint32_t)rows * xb, bar);
      if (BWD && (sa.one & 2)) bulk_load(dst2, dy + at.r * dys, (uint32_t)rows * yb, bar);
    }
    __syncwarp();
    if (!(sa.one & 1) && lane < rows) bulk_load(dst + lane * xb, x + (at.r + lane) * xs, xb, bar);
    if (BWD && !(sa.one & 2) && lane < rows) bulk_load(dst2 + lane * yb, dy + (at.r + lane) * dys, yb, bar);
    ++issued;
    at.next_unit();
    skip();
  }
  // every copy must land before the CTA exits; `used` of them were waited for
  __device__ void drain(uint32_t used, const Ctl& ctl) {
    Walk d(at.a, at.sa);
    for (uint32_t i = 0; i < issued; ++i) {
      d.take_slot();
      if (i >= used) mbar_wait_warp(full + d.slot, d.phase, nullptr, ctl, KID_NORM << 8 | 2);
    }
  }
};

// What the streamed kernels begin with: the barriers, and the thread's place.
struct Place {
  int gw, team, first, gl, lane;                  // threads of a row; team; is this its first warp; thread in the row; lane
  int sub;                                        // row of the unit
  __device__ Place(const NormArgs& a) {
    gw = a.gw;
    lane = threadIdx.x & 31;
    team = gw > 32 ? threadIdx.x / gw : threadIdx.x >> 5;
    first = (int)threadIdx.x - team * max(gw, 32) < 32;
    gl = threadIdx.x % gw;
    sub = gw < 32 ? lane / gw : 0;
  }
};
__device__ __forceinline__ void stream_begin(uint64_t* full, int n, int* abort_word) {
  for (int i = threadIdx.x; i < n; i += kTeamThreads) mbar_init(&full[i], 1);
  if (threadIdx.x == 0) *abort_word = 0;
  fence_mbar_init();
  __syncthreads();
}

// CH chunks of 8 columns a thread; only the last can lie behind the row.
// x may be y: a row is read whole before any of it is written.
template <typename X, int CH>
__global__ void __launch_bounds__(kTeamThreads, 1)
    norm_fwd_stream_kernel(const X* x, long long xs, __nv_bfloat16* y, long long ys, const float* __restrict__ weight,
                           const float* __restrict__ bias, float* __restrict__ stats, NormArgs a, StreamArgs sa, Ctl ctl) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kTeamWarps * kMaxSlots];
  __shared__ float slot[2][kTeamWarps][4];
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  stream_begin(full, sa.teams * sa.slots, &abort_word);
  const Place me(a);
  const uint32_t unit_bytes = (uint32_t)sa.unit * a.C * sizeof(X);
  uint8_t* mine = ring + (size_t)me.team * sa.slots * unit_bytes;
  uint64_t* bar = full + me.team * sa.slots;
  Loader<X, false> in(x, xs, nullptr, 0, mine, bar, a, sa, me.team);
  if (me.first)
    for (int i = 0; i < sa.slots; ++i) in.load();
  check_ptr(a, ctl);
  const int chunks = a.C >> 3, gw = me.gw, gl = me.gl;
  const bool last = (CH - 1) * gw + gl < chunks;
  const float inv_c = 1.0f / (float)a.C;
  float* lw = reinterpret_cast<float*>(ring + (size_t)sa.teams * sa.slots * unit_bytes);
  float* lb = lw + a.C;
  Walk at(a, sa);
  bool ok = true;                                 // a failed wait: the loops go on, past the barriers, and write nothing
  uint32_t used = 0;
  while (at.next_sequence(me.team)) {
    const float* w = weight == nullptr ? nullptr : weight + (long long)at.s * a.C;
    const float* b = bias == nullptr ? nullptr : bias + (long long)at.s * a.C;
    if (sa.local && w != nullptr) {
      cta_sync();                                 // the last sequence's have been read
      make_local(lw, w, chunks);
      if (b != nullptr) make_local(lb, b, chunks);
      cta_sync();
    }
    for (; at.r < at.q; at.next_unit()) {
      at.take_slot();
      const int row = at.r + me.sub;
      const bool has = row < at.q;
      if (ok) ok = mbar_wait_warp(&bar[at.slot], at.phase, abort_flag, ctl, KID_NORM << 8 | 3);
      used += ok ? 1u : 0u;
      const X* src = reinterpret_cast<const X*>(mine + (size_t)at.slot * unit_bytes) + (size_t)me.sub * a.C + 8 * gl;
      uint64_t v[CH][4];
      uint64_t t = 0ull;
      if (has) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          if (i < CH - 1 || last) {
            pairs8(src + 8 * i * gw, v[i]);
            t = add2(t, add2(add2(v[i][0], v[i][1]), add2(v[i][2], v[i][3])));
          }
        }
      }
      float mean = both(t);
      group_sums<1>(&mean, slot[0], me.team, gw);
      __syncwarp();
      if (me.first && ok) in.load();              // the team has its rows in registers
      mean *= inv_c;
      const uint64_t m2 = twice(-mean);
      t = 0ull;
      if (has) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          if (i < CH - 1 || last) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              v[i][j] = add2(v[i][j], m2);
              t = fma2(v[i][j], v[i][j], t);
            }
          }
        }
      }
      float sq = both(t);
      group_sums<1>(&sq, slot[1], me.team, gw);
      if (has && ok) {
        const float rstd = 1.0f / sqrtf(sq * inv_c + a.eps);
        if (gl == 0) {
          stats[row] = mean;
          stats[(long long)a.T + row] = rstd;
        }
        const uint64_t r2 = twice(rstd);
        __nv_bfloat16* out = y + row * ys + 8 * gl;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          if (i < CH - 1 || last) {
            uint64_t wv[4], bv[4];
            if (w != nullptr) {
              if (sa.local) local8(lw, i * gw + gl, chunks, wv); else pairs8(w + 8 * (i * gw + gl), wv);
            }
            if (b != nullptr) {
              if (sa.local) local8(lb, i * gw + gl, chunks, bv); else pairs8(b + 8 * (i * gw + gl), bv);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              v[i][j] = mul2(v[i][j], r2);
              if (b != nullptr) v[i][j] = fma2(v[i][j], wv[j], bv[j]); else if (w != nullptr) v[i][j] = mul2(v[i][j], wv[j]);
            }
            store_pairs8(out + 8 * i * gw, v[i]);
          }
        }
      }
    }
  }
  if (me.first && used < in.issued) in.drain(used, ctl);
}

// The sums of the part of sequence s that a CTA holds go to slot blockIdx + s of
// the workspace (2 C floats: dw, db).  The next part has a later CTA or a later
// sequence, so no two parts share a slot.  dx may be x or dy.
template <typename X, int CH>
__global__ void __launch_bounds__(kTeamThreads, 1)
    norm_bwd_stream_kernel(const __nv_bfloat16* dy, long long dys, const X* x, long long xs,
                           const float* __restrict__ stats, const float* __restrict__ weight, X* dx, long long dxs,
                           float* parts, NormArgs a, StreamArgs sa, Ctl ctl) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kTeamWarps * kMaxSlots];
  __shared__ float slot[2][kTeamWarps][4];
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  stream_begin(full, sa.teams * sa.slots, &abort_word);
  const Place me(a);
  const uint32_t xbytes = (uint32_t)sa.unit * a.C * sizeof(X), unit_bytes = xbytes + (uint32_t)sa.unit * a.C * 2u;
  uint8_t* mine = ring + (size_t)me.team * sa.slots * unit_bytes;
  uint64_t* bar = full + me.team * sa.slots;
  Loader<X, true> in(x, xs, dy, dys, mine, bar, a, sa, me.team);
  if (me.first)
    for (int i = 0; i < sa.slots; ++i) in.load();
  check_ptr(a, ctl);
  const int chunks = a.C >> 3, gw = me.gw, gl = me.gl;
  const bool last = (CH - 1) * gw + gl < chunks;
  const float inv_c = 1.0f / (float)a.C;
  float* lw = reinterpret_cast<float*>(ring + (size_t)sa.teams * sa.slots * unit_bytes);
  float* near = lw + (sa.local ? a.C : 0);        // 2 C floats
  Walk at(a, sa);
  bool ok = true, behind = false;                 // behind: the team's last unit still holds its slot
  uint32_t used = 0;
  int parity = 0;
  while (at.next_sequence(me.team)) {
    const float* w = weight == nullptr ? nullptr : weight + (long long)at.s * a.C;
    if (sa.local && w != nullptr) {
      cta_sync();
      make_local(lw, w, chunks);
      cta_sync();
    }
    uint64_t dw[CH][4], db[CH][4];
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) dw[i][j] = db[i][j] = 0ull;
    float mean = 0.f, rstd = 0.f;
    if (at.r + me.sub < at.q) {
      mean = __ldg(stats + at.r + me.sub);
      rstd = __ldg(stats + (long long)a.T + at.r + me.sub);
    }
    for (; at.r < at.q; at.next_unit()) {
      at.take_slot();
      const int row = at.r + me.sub;
      const bool has = row < at.q;
      const uint64_t rs = twice(rstd), off = twice(-mean);       // x^ = (x + off) r
      const int next = row + sa.teams * sa.unit;
      if (next < at.q) {
        mean = __ldg(stats + next);
        rstd = __ldg(stats + (long long)a.T + next);
      }
      if (ok) ok = mbar_wait_warp(&bar[at.slot], at.phase, abort_flag, ctl, KID_NORM << 8 | 3);
      used += ok ? 1u : 0u;
      const X* px = reinterpret_cast<const X*>(mine + (size_t)at.slot * unit_bytes) + (size_t)me.sub * a.C + 8 * gl;
      const __nv_bfloat16* pg =
          reinterpret_cast<const __nv_bfloat16*>(mine + (size_t)at.slot * unit_bytes + xbytes) + (size_t)me.sub * a.C + 8 * gl;
      auto weights = [&](int i, uint64_t* v) {
        if (w == nullptr) {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = twice(1.0f);
        } else if (sa.local) {
          local8(lw, i * gw + gl, chunks, v);
        } else {
          pairs8(w + 8 * (i * gw + gl), v);
        }
      };
      uint64_t s1 = 0ull, s2 = 0ull;
      if (has) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          if (i < CH - 1 || last) {
            uint64_t wv[4], h[4], g[4];
            weights(i, wv);
            pairs8(px + 8 * i * gw, h);
            pairs8(pg + 8 * i * gw, g);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint64_t xh = mul2(add2(h[j], off), rs);
              dw[i][j] = fma2(g[j], xh, dw[i][j]);
              db[i][j] = add2(db[i][j], g[j]);
              const uint64_t gw2 = mul2(g[j], wv[j]);
              s1 = add2(s1, gw2);
              s2 = fma2(gw2, xh, s2);
            }
          }
        }
      }
      float s[2] = {both(s1), both(s2)};
      group_sums<2>(s, slot[parity], me.team, gw);
      parity ^= 1;
      // several warps: all have met, so all are done with the unit before this one
      if (gw > 32 && me.first && ok && behind) in.load();
      behind = true;
      if (has && ok) {
        s1 = twice(-s[0] * inv_c), s2 = twice(-s[1] * inv_c);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          if (i < CH - 1 || last) {
            uint64_t wv[4], h[4], g[4];
            weights(i, wv);
            pairs8(px + 8 * i * gw, h);
            pairs8(pg + 8 * i * gw, g);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint64_t xh = mul2(add2(h[j], off), rs);
              g[j] = mul2(fma2(xh, s2, fma2(g[j], wv[j], s1)), rs);
            }
            store_pairs8(dx + row * dxs + 8 * (i * gw + gl), g);
          }
        }
      }
      __syncwarp();
      if (gw <= 32 && ok) in.load();
    }
    if (parts == nullptr) continue;
    // the teams' sums, one behind the other: inside a warp by shuffles, then through memory
    float* out = parts + 2LL * a.C * ((long long)blockIdx.x + at.s);
    float* held = sa.sums ? near : out;
    for (int o = gw; o < 32; o <<= 1) {
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          dw[i][j] = add2(dw[i][j], __shfl_xor_sync(0xffffffffu, dw[i][j], o));
          db[i][j] = add2(db[i][j], __shfl_xor_sync(0xffffffffu, db[i][j], o));
        }
    }
    const int turns = min(sa.teams, (at.q - at.p + sa.unit - 1) / sa.unit);
    for (int k = 0; k < turns; ++k) {
      if (me.team == k && me.sub == 0) {
        float* to = k == turns - 1 ? out : held;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          if (i < CH - 1 || last) {
            const int c = 8 * (i * gw + gl);
            if (k > 0) {
              uint64_t t[4], u[4];
              pairs8(held + c, t);
              pairs8(held + a.C + c, u);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                dw[i][j] = add2(t[j], dw[i][j]);
                db[i][j] = add2(u[j], db[i][j]);
              }
            }
            store_pairs8(to + c, dw[i]);
            store_pairs8(to + a.C + c, db[i]);
          }
        }
      }
      if (turns > 1) cta_sync();
    }
  }
  if (me.first && used < in.issued) in.drain(used, ctl);
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
    const long long step = 2LL * a.C;
    const float* at = parts + step * s + c2;
    int k = p / R + warp;
    for (; k + 3 * kNormWarps <= last; k += 4 * kNormWarps) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __ldg(at + step * (k + i * kNormWarps));
#pragma unroll
      for (int i = 0; i < 4; ++i) t += v[i];
    }
    for (; k <= last; k += kNormWarps) t += __ldg(at + step * k);
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

// Streamed rows: threads of a row, chunks of a thread, teams and slots.
struct Stream {
  int gw, ch, smem;
  StreamArgs a;
};
Stream stream_of(const dsv_norm& p, int xsize, bool bwd) {
  Stream s;
  const int chunks = p.C / 8;
  // the forward keeps a row of up to 8 chunks in registers, the backward two sums of up to 4
  const int most = bwd ? kBwdChunks : kFwdChunks;
  s.gw = 2;
  while (s.gw < 32 && chunks > 4 * s.gw) s.gw *= 2;
  while (s.gw < kTeamThreads && chunks > most * s.gw) s.gw *= 2;
  s.a.sums = bwd && p.C <= 2048 ? 1 : 0;
  const int sums = s.a.sums ? 8 * p.C : 0, vectors = (bwd ? 4 : 8) * p.C;
  int unit;
  for (;; s.gw *= 2) {                             // two slots a team, or fewer and larger teams
    s.a.unit = s.gw < 32 ? 32 / s.gw : 1;
    s.a.teams = kTeamThreads / max(s.gw, 32);
    unit = s.a.unit * p.C * (xsize + (bwd ? 2 : 0));
    if (2 * s.a.teams * unit + sums <= kStreamBytes || s.gw == kTeamThreads) break;
  }
  s.ch = max(1, ceil_div(chunks, s.gw));
  s.a.local = 2 * s.a.teams * unit + sums + vectors <= kStreamBytes ? 1 : 0;
  const int more = (s.a.local ? vectors : 0) + sums;
  s.a.slots = min(kMaxSlots, (kStreamBytes - more) / (s.a.teams * unit));
  s.smem = s.a.slots * s.a.teams * unit + more;
  s.a.R = max(ceil_div(p.T, kSMs), s.a.unit);
  s.a.one = 0;
  return s;
}
// Rows of a CTA of the backward with narrow accesses.
int narrow_rows(const dsv_norm& p) {
  int ch, gw;
  shape_of(p.C, &ch, &gw);
  const int groups = kNormThreads / gw, r = ceil_div(p.T, 2 * kSMs);
  return ceil_div(r, groups) * groups;
}

template <typename X, int CH>
cudaError_t fwd_stream(const dsv_rows& x, const NormArgs& a, const Stream& s, const float* w, const float* b,
                       const dsv_rows& y, float* stats, const Ctl& ctl, cudaStream_t st) {
  auto kern = norm_fwd_stream_kernel<X, CH>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, s.smem);
  if (e != cudaSuccess) return e;
  kern<<<ceil_div(a.T, s.a.R), kTeamThreads, s.smem, st>>>(static_cast<const X*>(x.ptr), x.stride,
                                                             static_cast<__nv_bfloat16*>(y.ptr), y.stride, w, b, stats, a,
                                                             s.a, ctl);
  return cudaGetLastError();
}
template <typename X, int CH>
cudaError_t bwd_stream(const dsv_rows& dy, const dsv_rows& x, const float* stats, const NormArgs& a, const Stream& s,
                       const float* w, const dsv_rows& dx, float* parts, const Ctl& ctl, cudaStream_t st) {
  auto kern = norm_bwd_stream_kernel<X, CH>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, s.smem);
  if (e != cudaSuccess) return e;
  kern<<<ceil_div(a.T, s.a.R), kTeamThreads, s.smem, st>>>(
      static_cast<const __nv_bfloat16*>(dy.ptr), dy.stride, static_cast<const X*>(x.ptr), x.stride, stats, w,
      static_cast<X*>(dx.ptr), dx.stride, parts, a, s.a, ctl);
  return cudaGetLastError();
}
template <typename X>
cudaError_t fwd_pick(const dsv_rows& x, const NormArgs& a, const Stream& s, const float* w, const float* b,
                     const dsv_rows& y, float* stats, const Ctl& ctl, cudaStream_t st) {
  switch (s.ch) {
    case 1: return fwd_stream<X, 1>(x, a, s, w, b, y, stats, ctl, st);
    case 2: return fwd_stream<X, 2>(x, a, s, w, b, y, stats, ctl, st);
    case 3: return fwd_stream<X, 3>(x, a, s, w, b, y, stats, ctl, st);
    case 4: return fwd_stream<X, 4>(x, a, s, w, b, y, stats, ctl, st);
    case 5: return fwd_stream<X, 5>(x, a, s, w, b, y, stats, ctl, st);
    case 6: return fwd_stream<X, 6>(x, a, s, w, b, y, stats, ctl, st);
    case 7: return fwd_stream<X, 7>(x, a, s, w, b, y, stats, ctl, st);
    default: return fwd_stream<X, 8>(x, a, s, w, b, y, stats, ctl, st);
  }
}
template <typename X>
cudaError_t bwd_pick(const dsv_rows& dy, const dsv_rows& x, const float* stats, const NormArgs& a, const Stream& s,
                     const float* w, const dsv_rows& dx, float* parts, const Ctl& ctl, cudaStream_t st) {
  switch (s.ch) {
    case 1: return bwd_stream<X, 1>(dy, x, stats, a, s, w, dx, parts, ctl, st);
    case 2: return bwd_stream<X, 2>(dy, x, stats, a, s, w, dx, parts, ctl, st);
    case 3: return bwd_stream<X, 3>(dy, x, stats, a, s, w, dx, parts, ctl, st);
    default: return bwd_stream<X, 4>(dy, x, stats, a, s, w, dx, parts, ctl, st);
  }
}

template <typename X, int CH>
cudaError_t fwd_narrow(const dsv_rows& x, const NormArgs& a, const float* w, const float* b, const dsv_rows& y,
                       float* stats, const Ctl& ctl, cudaStream_t st) {
  const int groups = kNormThreads / a.gw, grid = min(ceil_div(a.T, groups), kSMs * 8);
  norm_fwd_kernel<X, CH><<<grid, kNormThreads, 0, st>>>(static_cast<const X*>(x.ptr), x.stride,
                                                       static_cast<__nv_bfloat16*>(y.ptr), y.stride, w, b, stats, a, ctl);
  return cudaGetLastError();
}
template <typename X, int CH>
cudaError_t bwd_narrow(const dsv_rows& dy, const dsv_rows& x, const float* stats, const NormArgs& a, const float* w,
                       const dsv_rows& dx, float* parts, int R, const Ctl& ctl, cudaStream_t st) {
  const int groups = kNormThreads / a.gw, smem = groups > 1 ? 2 * a.C * (int)sizeof(float) : 0;
  auto kern = norm_bwd_kernel<X, CH>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<ceil_div(a.T, R), kNormThreads, smem, st>>>(
      static_cast<const __nv_bfloat16*>(dy.ptr), dy.stride, static_cast<const X*>(x.ptr), x.stride, stats, w,
      static_cast<X*>(dx.ptr), dx.stride, parts, R, a, ctl);
  return cudaGetLastError();
}
#define NARROW_PICK(fn, type, ch, ...)                                                               \
  (type == DSV_F32 ? (ch == 1 ? fn<float, 1>(__VA_ARGS__) : ch == 2 ? fn<float, 2>(__VA_ARGS__)      \
                      : ch == 4 ? fn<float, 4>(__VA_ARGS__) : fn<float, 8>(__VA_ARGS__))             \
                   : (ch == 1 ? fn<__nv_bfloat16, 1>(__VA_ARGS__) : ch == 2 ? fn<__nv_bfloat16, 2>(__VA_ARGS__) \
                      : ch == 4 ? fn<__nv_bfloat16, 4>(__VA_ARGS__) : fn<__nv_bfloat16, 8>(__VA_ARGS__)))

}  // namespace

cudaError_t launch_norm_fwd(const dsv_rows& x, const dsv_norm& p, const int32_t* ptr, const float* weight,
                            const float* bias, const dsv_rows& y, float* stats, const Ctl& ctl, cudaStream_t st) {
  NormArgs a = norm_args(p, ptr);
  if (p.C % 8 == 0 && wide(x, size_of(x.type)) && wide(y, 2) && wide(weight) && wide(bias)) {
    Stream s = stream_of(p, size_of(x.type), false);
    a.gw = s.gw;
    s.a.one = x.stride == p.C ? 1 : 0;
    return x.type == DSV_F32 ? fwd_pick<float>(x, a, s, weight, bias, y, stats, ctl, st)
                             : fwd_pick<__nv_bfloat16>(x, a, s, weight, bias, y, stats, ctl, st);
  }
  int ch;
  shape_of(p.C, &ch, &a.gw);
  return NARROW_PICK(fwd_narrow, x.type, ch, x, a, weight, bias, y, stats, ctl, st);
}

// The call's alignment is not known here: room for either way.
size_t norm_bwd_ws_bytes(const dsv_norm& p) {
  const int R = min(narrow_rows(p), min(stream_of(p, 2, true).a.R, stream_of(p, 4, true).a.R));
  return ((size_t)ceil_div(p.T, R) + p.S) * 2 * p.C * sizeof(float);
}

cudaError_t launch_norm_bwd(const dsv_rows& dy, const dsv_rows& x, const float* stats, const dsv_norm& p,
                            const int32_t* ptr, const float* weight, const dsv_rows& dx, float* dweight, float* dbias,
                            void* ws, const Ctl& ctl, cudaStream_t st) {
  NormArgs a = norm_args(p, ptr);
  float* parts = dweight != nullptr ? static_cast<float*>(ws) : nullptr;
  cudaError_t e;
  int R;
  if (p.C % 8 == 0 && wide(x, size_of(x.type)) && wide(dy, 2) && wide(dx, size_of(dx.type)) && wide(weight)) {
    Stream s = stream_of(p, size_of(x.type), true);
    a.gw = s.gw;
    s.a.one = (x.stride == p.C ? 1 : 0) | (dy.stride == p.C ? 2 : 0);
    R = s.a.R;
    e = x.type == DSV_F32 ? bwd_pick<float>(dy, x, stats, a, s, weight, dx, parts, ctl, st)
                          : bwd_pick<__nv_bfloat16>(dy, x, stats, a, s, weight, dx, parts, ctl, st);
  } else {
    int ch;
    shape_of(p.C, &ch, &a.gw);
    R = narrow_rows(p);
    e = NARROW_PICK(bwd_narrow, x.type, ch, dy, x, stats, a, weight, dx, parts, R, ctl, st);
  }
  if (e != cudaSuccess || parts == nullptr) return e;
  norm_sums_kernel<<<dim3(ceil_div(2LL * p.C, 32), p.S), kNormThreads, 0, st>>>(parts, R, dweight, dbias, a);
  return cudaGetLastError();
}

}  // namespace dsv
