// norm_bwd.cu — gradient of the layer norm (norm.cuh): dx, and the sums of dweight
// and dbias over the rows of each sequence.
//
// HBM-bound: 6 bytes an element (bf16) at some 10 operations.  A CTA takes
// neighbouring rows and keeps the sums of dweight and dbias of its columns in
// registers as long as a sequence lasts; the parts of all CTAs are added by a small
// second kernel in the order of their rows.
#include "norm.cuh"

namespace dsv {

namespace {

// ---------------------------------------------------------------------------
// Rows with 16-byte accesses: streamed through shared memory
// ---------------------------------------------------------------------------
// A row belongs to `gw` neighbouring threads, 2 to 512 of them, CH chunks of 8
// columns each.  The warps that share a row, or the one warp that holds several,
// are a team, which works on two rows (of a thread) at once where two slots of them fit: an
// exchange of sums, a wait and the rest of the fixed cost (some 200 instructions)
// serve both.  Every team has a ring of slots that its first warp fills by bulk
// copies, so that bytes in flight cost no registers and no team waits for another.
// One CTA an SM; a thread keeps the weight of its columns in registers too (in
// shared memory, with 4 chunks a thread and a row at a time: 330 us and not 246).
// Measured: 122880 rows of 2048, 1.5 GB, 244 us, 91 % of the copy bandwidth; 16384
// rows of 5120 105 us, 71 %; 16384 of 8192 142 us, 84 %.
constexpr int kStreamBytes = 220 * 1024;       // of shared memory
constexpr int kTeamThreads = 512, kTeamWarps = kTeamThreads / 32, kMaxSlots = 8;

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
  float4 u = *reinterpret_cast<const float4*>(slot[first]);
  for (int k = 1; k < n; ++k) {
    const float4 q = *reinterpret_cast<const float4*>(slot[first + k]);
    u.x += q.x, u.y += q.y;
    if constexpr (N == 4) u.z += q.z, u.w += q.w;
  }
  v[0] = u.x;
  if constexpr (N >= 2) v[1] = u.y;
  if constexpr (N == 4) v[2] = u.z, v[3] = u.w;
}

// A team's first warp brings in its rows, unit by unit.
template <typename X>
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
    yb = (uint32_t)a.C * 2u;
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
      if (sa.one & 2) bulk_load(dst2, dy + at.r * dys, (uint32_t)rows * yb, bar);
    }
    __syncwarp();
    if (!(sa.one & 1) && lane < rows) bulk_load(dst + lane * xb, x + (at.r + lane) * xs, xb, bar);
    if (!(sa.one & 2) && lane < rows) bulk_load(dst2 + lane * yb, dy + (at.r + lane) * dys, yb, bar);
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

// What the kernel begins with: the barriers, and the thread's place.
struct Place {
  int gw, team, gl, lane;                         // threads of a row; team; thread in the row; lane
  int sub;                                        // its first row of the unit
  bool first, idle;                               // is this the team's first warp; in no team
  __device__ Place(const NormArgs& a, const StreamArgs& sa, int rows) {
    gw = a.gw;
    lane = threadIdx.x & 31;
    team = gw > 32 ? threadIdx.x / gw : threadIdx.x >> 5;
    idle = team >= sa.teams;
    first = !idle && (int)threadIdx.x - team * max(gw, 32) < 32;
    gl = threadIdx.x % gw;
    sub = gw < 32 ? lane / gw * rows : 0;
  }
};
__device__ __forceinline__ void stream_begin(uint64_t* full, int n, int* abort_word) {
  for (int i = threadIdx.x; i < n; i += kTeamThreads) mbar_init(&full[i], 1);
  if (threadIdx.x == 0) *abort_word = 0;
  fence_mbar_init();
  __syncthreads();
}

// The weight of a thread's columns, in registers where they are few.
template <int CH>
struct Columns {
  static constexpr bool KEEP = CH <= 3;
  uint64_t v[KEEP ? CH : 1][4];
  const float* from;
  float none;
  // p: the vector of the sequence, at the thread's first chunk, or null: `value` in all columns
  __device__ __forceinline__ void set(const float* p, float value, int gw, bool last) {
    from = p;
    none = value;
    if constexpr (KEEP) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j] = twice(value);
        if (p != nullptr && (i < CH - 1 || last)) pairs8(p + 8 * i * gw, v[i]);
      }
    }
  }
  __device__ __forceinline__ void get(int i, int gw, uint64_t* to) const {
    if constexpr (KEEP) {
#pragma unroll
      for (int j = 0; j < 4; ++j) to[j] = v[i][j];
    } else if (from != nullptr) {
      pairs8(from + 8 * i * gw, to);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) to[j] = twice(none);
    }
  }
};

// CH chunks of 8 columns a thread, of which only the last can lie behind the row;
// ROWS rows of a team at once.
// The sums of the part of sequence s that a CTA holds go to slot blockIdx + s of
// the workspace (2 C floats: dw, db).  The next part has a later CTA or a later
// sequence, so no two parts share a slot.  dx may be x or dy.
template <typename X, int CH, int ROWS>
__global__ void __launch_bounds__(kTeamThreads, 1)
    norm_bwd_stream_kernel(const __nv_bfloat16* dy, long long dys, const X* x, long long xs,
                           const float* __restrict__ stats, const float* __restrict__ weight, X* dx, long long dxs,
                           float* parts, NormArgs a, StreamArgs sa, Ctl ctl) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kTeamWarps * kMaxSlots];
  __shared__ __align__(16) float slot[2][kTeamWarps][4];
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  cudaTriggerProgrammaticLaunchCompletion();      // norm_sums_kernel may come to wait
  stream_begin(full, sa.teams * sa.slots, &abort_word);
  const Place me(a, sa, ROWS);
  const uint32_t xbytes = (uint32_t)sa.unit * a.C * sizeof(X), unit_bytes = xbytes + (uint32_t)sa.unit * a.C * 2u;
  uint8_t* mine = ring + (size_t)me.team * sa.slots * unit_bytes;
  uint64_t* bar = full + me.team * sa.slots;
  Loader<X> in(x, xs, dy, dys, mine, bar, a, sa, me.team);
  if (me.first)
    for (int i = 0; i < sa.slots; ++i) in.load();
  check_ptr(a, ctl);
  const int chunks = a.C >> 3, gw = me.gw, gl = me.gl;
  const bool last = (CH - 1) * gw + gl < chunks;
  const float inv_c = 1.0f / (float)a.C;
  float* near = reinterpret_cast<float*>(ring + (size_t)sa.teams * sa.slots * unit_bytes);       // 2 C floats
  Walk at(a, sa);
  bool ok = true, behind = false;                 // behind: the team's last unit still holds its slot
  uint32_t used = 0;
  int parity = 0;
  while (at.next_sequence(me.team)) {
    Columns<CH> w;
    w.set(weight == nullptr ? nullptr : weight + (long long)at.s * a.C + 8 * gl, 1.0f, gw, last);
    uint64_t dw[CH][4], db[CH][4];
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) dw[i][j] = db[i][j] = 0ull;
    float mean[ROWS], rstd[ROWS];
    auto load_stats = [&](int row) {                // rows behind the end: the last one's
#pragma unroll
      for (int k = 0; k < ROWS; ++k) {
        const int i = min(row + k, at.q - 1);
        mean[k] = __ldg(stats + i);
        rstd[k] = __ldg(stats + a.T + i);
      }
    };
    if (me.idle) at.r = at.q;
    load_stats(at.r + me.sub);
    for (; at.r < at.q; at.next_unit()) {
      at.take_slot();
      const int row = at.r + me.sub, rows = at.q - row;          // rows <= 0: none here
      uint64_t rs[ROWS], off[ROWS];                               // x^ = (x + off) r
#pragma unroll
      for (int k = 0; k < ROWS; ++k) rs[k] = twice(rstd[k]), off[k] = twice(-mean[k]);
      load_stats(row + sa.teams * sa.unit);
      if (ok) ok = mbar_wait_warp(&bar[at.slot], at.phase, abort_flag, ctl, KID_NORM << 8 | 3);
      used += ok ? 1u : 0u;
      const X* px = reinterpret_cast<const X*>(mine + (size_t)at.slot * unit_bytes) + (size_t)me.sub * a.C + 8 * gl;
      const __nv_bfloat16* pg =
          reinterpret_cast<const __nv_bfloat16*>(mine + (size_t)at.slot * unit_bytes + xbytes) + (size_t)me.sub * a.C + 8 * gl;
      uint64_t s1[ROWS], s2[ROWS];
#pragma unroll
      for (int k = 0; k < ROWS; ++k) s1[k] = s2[k] = 0ull;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        if (i < CH - 1 || last) {
          uint64_t wv[4];
          w.get(i, gw, wv);
#pragma unroll
          for (int k = 0; k < ROWS; ++k) {
            if (k < rows) {
              uint64_t h[4], g[4];
              pairs8(px + k * a.C + 8 * i * gw, h);
              pairs8(pg + k * a.C + 8 * i * gw, g);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint64_t xh = mul2(add2(h[j], off[k]), rs[k]);
                dw[i][j] = fma2(g[j], xh, dw[i][j]);
                db[i][j] = add2(db[i][j], g[j]);
                const uint64_t gw2 = mul2(g[j], wv[j]);
                s1[k] = add2(s1[k], gw2);
                s2[k] = fma2(gw2, xh, s2[k]);
              }
            }
          }
        }
      }
      float s[2 * ROWS];
#pragma unroll
      for (int k = 0; k < ROWS; ++k) s[2 * k] = both(s1[k]), s[2 * k + 1] = both(s2[k]);
      group_sums<2 * ROWS>(s, slot[parity], me.team, gw);
      parity ^= 1;
      // several warps: all have met, so all are done with the unit before this one
      if (gw > 32 && me.first && ok && behind) in.load();
      behind = true;
      if (ok) {
#pragma unroll
        for (int k = 0; k < ROWS; ++k) s1[k] = twice(-s[2 * k] * inv_c), s2[k] = twice(-s[2 * k + 1] * inv_c);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          if (i < CH - 1 || last) {
            uint64_t wv[4];
            w.get(i, gw, wv);
#pragma unroll
            for (int k = 0; k < ROWS; ++k) {
              if (k < rows) {
                uint64_t h[4], g[4];
                pairs8(px + k * a.C + 8 * i * gw, h);
                pairs8(pg + k * a.C + 8 * i * gw, g);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const uint64_t xh = mul2(add2(h[j], off[k]), rs[k]);
                  g[j] = mul2(fma2(xh, s2[k], fma2(g[j], wv[j], s1[k])), rs[k]);
                }
                store_pairs8(dx + (row + k) * dxs + 8 * (i * gw + gl), g);
              }
            }
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
    if (CH <= 2 && sa.sums > 1 && turns > 1) {
      // few columns: all teams at once (6 sequences of 22620 rows of 360: 42 us with 16 turns, 35 so)
      if (me.team < turns && me.sub == 0) {
        float* to = near + 2 * a.C * me.team;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          if (i < CH - 1 || last) {
            store_pairs8(to + 8 * (i * gw + gl), dw[i]);
            store_pairs8(to + a.C + 8 * (i * gw + gl), db[i]);
          }
        }
      }
      cta_sync();
      for (int c = threadIdx.x; c < 2 * a.C; c += kTeamThreads) {
        float t = near[c];
        for (int k = 1; k < turns; ++k) t += near[2 * a.C * k + c];
        out[c] = t;
      }
      cta_sync();
      continue;
    }
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

// dw_s, db_s: the parts of sequence s, in the order of their rows.  WARPS warps
// share 32 columns and take every WARPS-th part; with many sequences of few parts
// each, a warp has its columns to itself (the gradient of 2000 sequences of 30 rows of
// 1024: 232 -> 126 us a call).
template <int WARPS>
__global__ void __launch_bounds__(kNormThreads) norm_sums_kernel(const float* parts, int R, float* dweight, float* dbias,
                                                                 NormArgs a) {
  __shared__ float sum[WARPS > 1 ? WARPS : 1][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, turn = warp % WARPS;
  const int c2 = ((int)blockIdx.x * (kNormWarps / WARPS) + warp / WARPS) * 32 + lane, s = (int)blockIdx.y;   // of dw, then of db
  int p = a.ptr == nullptr ? (a.S == 1 ? 0 : s * a.even) : a.ptr[s];
  int q = a.ptr == nullptr ? (a.S == 1 ? a.T : (s + 1) * a.even) : a.ptr[s + 1];
  p = max(p, 0);
  q = min(q, a.T);
  float t = 0.f;
  cudaGridDependencySynchronize();
  if (p < q && c2 < 2 * a.C) {
    const int last = (q - 1) / R;
    const long long step = 2LL * a.C;
    const float* at = parts + step * s + c2;
    int k = p / R + turn;
    constexpr int N = WARPS > 1 ? 20 : 4;            // 152 parts of one CTA an SM: 19 a warp
    for (; k <= last; k += N * WARPS) {
      float v[N];
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = k + i * WARPS <= last ? __ldcg(at + step * (k + i * WARPS)) : 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) t += v[i];
    }
  }
  if constexpr (WARPS > 1) {
    sum[warp][lane] = t;
    __syncthreads();
    t = 0.f;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) t += sum[k][lane];
  }
  if (turn == 0 && c2 < 2 * a.C) {
    float* out = c2 < a.C ? dweight + (long long)s * a.C + c2 : dbias + (long long)s * a.C + (c2 - a.C);
    *out = t;
  }
}

// Streamed rows: threads of a row, chunks of a thread, teams and slots.
struct Stream {
  int gw, ch, rows, smem;
  StreamArgs a;
};
Stream stream_of(const dsv_norm& p, int xsize) {
  Stream s;
  const int chunks = p.C / 8;
  // all teams' sums leave room for two slots of two rows up to 512 columns
  s.a.sums = p.C <= 512 ? 2 : p.C <= 2048 ? 1 : 0;
  const int row = p.C * (xsize + 2), sums = s.a.sums == 2 ? 8 * p.C * kTeamWarps : s.a.sums ? 8 * p.C : 0;
  if (chunks <= 64) {                              // part of a warp, two chunks a thread
    s.gw = 2;
    while (chunks > 2 * s.gw) s.gw *= 2;
    s.ch = ceil_div(chunks, s.gw);
    s.rows = 2;
  } else {
    // Whole warps: a row of 1, 2 or 3 chunks a thread takes a team a time of 10, 16 or 28,
    // and a quarter more where shared memory has no room for two rows at once.  Measured,
    // 1, 2 and 3 chunks: rows of 1160 (17154, fp32) 48.4, 47.8, 52 us, of 2048 (122880) 314,
    // 246, 263, of 640 (30000, fp32) 45.7, 47.8, 52, of 5120 (16384) -, 119, 108.
    s.rows = 2;
    s.gw = 0;
    const int cost[4] = {10, 16, 28, 0};
    int best = 0;
    for (int ch = 1; ch <= 4; ++ch) {
      const int gw = ceil_div(ceil_div(chunks, ch), 32) * 32, teams = kTeamThreads / gw;
      if (teams == 0 || (ch == 4 && s.gw != 0)) continue;
      const bool two = 4 * teams * row + sums <= kStreamBytes;
      const int speed = ch == 4 ? 1 : teams * (two ? 5000 : 4000) / cost[ch - 1];
      if (speed > best) best = speed, s.gw = gw, s.ch = ceil_div(chunks, gw);
    }
  }
  for (;;) {                                       // two slots a team, or one row at once, or fewer teams
    s.a.unit = s.gw < 32 ? 32 / s.gw * s.rows : s.rows;
    s.a.teams = kTeamThreads / max(s.gw, 32);
    if (2 * s.a.teams * s.a.unit * row + sums <= kStreamBytes) break;
    if (s.rows == 2) {
      s.rows = 1;
    } else if (s.gw < 32) {
      s.gw *= 2;
    } else {
      s.gw = kTeamThreads / (s.a.teams - 1) / 32 * 32;
    }
    s.ch = ceil_div(chunks, s.gw);
  }
  s.a.slots = min(kMaxSlots, (kStreamBytes - sums) / (s.a.teams * s.a.unit * row));
  s.smem = s.a.slots * s.a.teams * s.a.unit * row + sums;
  s.a.R = max(ceil_div(p.T, kSMs), s.a.unit);
  s.a.one = 0;
  return s;
}

template <typename X, int CH, int ROWS>
cudaError_t bwd_stream(const dsv_rows& dy, const dsv_rows& x, const float* stats, const NormArgs& a, const Stream& s,
                       const float* w, const dsv_rows& dx, float* parts, const Ctl& ctl, cudaStream_t st) {
  auto kern = norm_bwd_stream_kernel<X, CH, ROWS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, s.smem);
  if (e != cudaSuccess) return e;
  kern<<<ceil_div(a.T, s.a.R), kTeamThreads, s.smem, st>>>(
      static_cast<const __nv_bfloat16*>(dy.ptr), dy.stride, static_cast<const X*>(x.ptr), x.stride, stats, w,
      static_cast<X*>(dx.ptr), dx.stride, parts, a, s.a, ctl);
  return cudaGetLastError();
}
template <typename X>
cudaError_t bwd_pick(const dsv_rows& dy, const dsv_rows& x, const float* stats, const NormArgs& a, const Stream& s,
                     const float* w, const dsv_rows& dx, float* parts, const Ctl& ctl, cudaStream_t st) {
  switch (10 * s.ch + s.rows) {
    case 12: return bwd_stream<X, 1, 2>(dy, x, stats, a, s, w, dx, parts, ctl, st);
    case 22: return bwd_stream<X, 2, 2>(dy, x, stats, a, s, w, dx, parts, ctl, st);
    case 32: return bwd_stream<X, 3, 2>(dy, x, stats, a, s, w, dx, parts, ctl, st);
    case 41: return bwd_stream<X, 4, 1>(dy, x, stats, a, s, w, dx, parts, ctl, st);
  }
  if constexpr (sizeof(X) == 4) {                // what only one type's rows get
    if (s.ch == 2) return bwd_stream<X, 2, 1>(dy, x, stats, a, s, w, dx, parts, ctl, st);
    if (s.ch == 3) return bwd_stream<X, 3, 1>(dy, x, stats, a, s, w, dx, parts, ctl, st);
  } else {
    if (s.ch == 4) return bwd_stream<X, 4, 2>(dy, x, stats, a, s, w, dx, parts, ctl, st);
  }
  return cudaErrorInvalidValue;                  // no width gives another pair
}

}  // namespace

// The call's alignment is not known here: room for either way.
size_t norm_bwd_ws_bytes(const dsv_norm& p) {
  const int R = min(norm_narrow_rows(p), min(stream_of(p, 2).a.R, stream_of(p, 4).a.R));
  return ((size_t)ceil_div(p.T, R) + p.S) * 2 * p.C * sizeof(float);
}

cudaError_t launch_norm_bwd(const dsv_rows& dy, const dsv_rows& x, const float* stats, const dsv_norm& p,
                            const int32_t* ptr, const float* weight, const dsv_rows& dx, float* dweight, float* dbias,
                            void* ws, const Ctl& ctl, cudaStream_t st) {
  NormArgs a = norm_args(p, ptr);
  float* parts = dweight != nullptr ? static_cast<float*>(ws) : nullptr;
  cudaError_t e;
  int R;
  // 16 bytes: 8 elements of bf16, 4 of fp32
  auto lies = [](const dsv_rows& v) { return aligned(v, 16 / size_of(v.type)); };
  if (p.C % 8 == 0 && lies(x) && lies(dy) && lies(dx) && wide(weight)) {
    Stream s = stream_of(p, size_of(x.type));
    a.gw = s.gw;
    s.a.one = (x.stride == p.C ? 1 : 0) | (dy.stride == p.C ? 2 : 0);
    R = s.a.R;
    e = x.type == DSV_F32 ? bwd_pick<float>(dy, x, stats, a, s, weight, dx, parts, ctl, st)
                          : bwd_pick<__nv_bfloat16>(dy, x, stats, a, s, weight, dx, parts, ctl, st);
  } else {
    R = norm_narrow_rows(p);
    e = launch_norm_bwd_narrow(dy, x, stats, p, a.ptr, weight, dx, parts, ctl, st);
  }
  if (e != cudaSuccess || parts == nullptr) return e;
  // it comes as the rows' CTAs leave room, and waits for them
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  const bool few = ceil_div(p.T, R) <= 3LL * p.S;            // parts of a sequence: at most 4 on average
  cfg.gridDim = dim3(ceil_div(2LL * p.C, few ? 32 * kNormWarps : 32), p.S);
  cfg.blockDim = dim3(kNormThreads);
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few ? norm_sums_kernel<1> : norm_sums_kernel<kNormWarps>,
                            static_cast<const float*>(parts), R, dweight, dbias, a);
}

}  // namespace dsv
