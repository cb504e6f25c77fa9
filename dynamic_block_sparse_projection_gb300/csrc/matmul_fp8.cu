// matmul_fp8.cu — products of 8-bit floating-point matrices with a scale for
// each block of 128 along the summed dimension.
//
//   C[m, n] = sum over kb of sa[kb, m] sb[kb, n] (sum over k in block kb of a[m, k] b[n, k])
//
// a [M, K] and b [N, K] are e4m3 or e5m2 with K contiguous; a scale belongs to
// one row, or to 128 rows.  The tensor cores sum a block's 128 products (exact
// products, fp32 sums) into tensor memory; eight warps read each block's sums,
// scale them and add them up in fp32 registers, while the next block's
// products run into the other half of the tensor memory.
#include <math.h>

#include <type_traits>

#include "dsv_launch.h"

namespace dsv {

namespace {

constexpr int kSMs = 152;
constexpr int kPairs = 76;                 // pairs of SMs
constexpr int kKb = 128;                   // elements and bytes of a block along K: one swizzle row
constexpr int kStoreBytes = 8 * 4096;      // on C's way out, 4 KB a warp

enum : unsigned int { W_EMPTY = 1, W_FULL = 2, W_FREE = 3, W_SUMS = 4, W_DRAIN = 5 };

struct MmArgs {
  int M, N, kbs;                           // rows of C, columns, blocks of K
  int tm, tn, group;                       // tiles; columns of tiles that are worked on together
  const float* sa;
  const float* sb;
  long long sa_ld, sb_ld;                  // scales of a block of K
  int sa_shift, sb_shift;                  // 0: a scale for each row, 7: for 128 rows
  void* c;
  long long ldc;
  int split, vec;                          // small tiles: CTAs that share the blocks of K; rows of C on 4 values
  int accumulate, tma;                     // tma: C takes tensor copies (2: of every chunk, 1: not of a cut one)
  uint32_t idesc;
};

// kind::f8f6f4, one elected lane of a converged warp
__device__ __forceinline__ void mma_f8_w(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b32 r;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor: fp32 sums (bits 4-5), A's type (7-9) and B's (10-12): 0 e4m3, 1 e5m2; N>>3, M>>4.
uint32_t idesc_f8(int M, int N, bool a_e5, bool b_e5) {
  return (1u << 4) | ((a_e5 ? 1u : 0u) << 7) | ((b_e5 ? 1u : 0u) << 10) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// Waits for the loads from tensor memory; the registers pass through, so that no
// use of them can be moved ahead of the wait.
__device__ __forceinline__ void tmem_ld_wait16(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_ld_wait32(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
// Tensor memory -> registers, 16 lanes x 32 columns: r[4 i], r[4 i + 1] are columns 8 i + 2 (lane % 4) and the
// next of row lane / 4, and r[4 i + 2], r[4 i + 3] those of row lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_rows16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// 4 bytes to shared memory beside what the thread does (zero where !in).
__device__ __forceinline__ void copy4(float* dst, const float* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 4 : 0) : "memory");
}
// N registers that a wait before this has covered.
template <int N>
__device__ __forceinline__ void tmem_pass(uint32_t* r) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i])::"memory");
}

// A warp's part of C: 32 rows from `row0` and 128 columns from `col`, by way of 4 KB of shared memory: 32 rows of 128 bytes, the
// 16-byte units of a row swapped by the row, as tensor copies with the 128-byte
// swizzle have them.  The tensor copy out runs beside the next tile; where C's
// rows do not lie on 16 bytes, or are added to, the warp writes them itself.
// (A lane that stores its row itself takes 32 lines an instruction: 13 % of a
// product with K = 2048.)  acc: the pairs of a lane's own row in their order; or
// (SPREAD) [32 columns][16 rows][8 columns][8 rows] as tmem_ld_rows16 gives them.
template <bool F32, bool ADD, bool SPREAD>
__device__ __forceinline__ void store_rows(const MmArgs& g, const CUtensorMap* tmC, uint8_t* stage, int row0, int col,
                                           const uint64_t* acc) {
  using C = typename std::conditional<F32, float, __nv_bfloat16>::type;
  constexpr int COLS = F32 ? 32 : 64;                    // columns of a chunk
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c0 = 0; c0 < 128; c0 += COLS) {
    // the last chunk has left shared memory
    if (g.tma && lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
    if constexpr (SPREAD) {
#pragma unroll
      for (int i = 0; i < COLS / 2; ++i) {                 // 8 columns and 8 rows a step
        const int c = c0 + i / 4 * 8, h = i / 2 % 2, k = i % 2;
        float x, y;
        f2_unpack(acc[c / 32 * 16 + h * 8 + c / 8 % 4 * 2 + k], x, y);
        const int row = lane / 4 + 16 * h + 8 * k, at = (c - c0 + 2 * (lane & 3)) * (F32 ? 4 : 2);
        uint8_t* to = stage + row * 128 + (((at >> 4) ^ (row & 7)) << 4) + (at & 15);
        if constexpr (F32) *reinterpret_cast<float2*>(to) = make_float2(x, y);
        else *reinterpret_cast<uint32_t*>(to) = pack_bf16x2(x, y);
      }
    } else {
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        uint32_t w[4];
        if constexpr (F32) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float x, y;
            f2_unpack(acc[c0 / 2 + 2 * u + i], x, y);
            w[2 * i] = __float_as_uint(x);
            w[2 * i + 1] = __float_as_uint(y);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float x, y;
            f2_unpack(acc[c0 / 2 + 4 * u + i], x, y);
            w[i] = pack_bf16x2(x, y);
          }
        }
        *reinterpret_cast<uint4*>(stage + lane * 128 + ((u ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    if (row0 >= g.M || col + c0 >= g.N) continue;
    // a copy that the end of the rows cuts writes up to the next 16 bytes
    if (g.tma == 2 || (g.tma == 1 && col + c0 + COLS <= g.N)) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                         reinterpret_cast<uint64_t>(tmC)),
                     "r"(col + c0), "r"(row0), "r"(smem_u32(stage))
                     : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
    } else if (ADD && g.vec) {
      // added to rows on 16 bytes: a lane has unit lane % 8 of every fourth row (64 us at
      // 6144 x 2048 x 2048, 38 without adding; value by value 10 more; these kernels spill 116 bytes a thread)
      if constexpr (ADD) {
        const int c = col + c0 + 4 * (lane & 7), n = g.N - c, rows = g.M - row0 - lane / 8;
        float* out = static_cast<float*>(g.c) + (long long)(row0 + lane / 8) * g.ldc + c;
        float4 was[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (4 * j < rows && n >= 4) was[j] = *reinterpret_cast<const float4*>(out + 4LL * j * g.ldc);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (4 * j >= rows || n <= 0) continue;
          const int i = 4 * j + lane / 8;
          const float4 x = *reinterpret_cast<const float4*>(stage + i * 128 + (((lane & 7) ^ (i & 7)) << 4));
          float* to = out + 4LL * j * g.ldc;
          if (n >= 4) {
            *reinterpret_cast<float4*>(to) = make_float4(was[j].x + x.x, was[j].y + x.y, was[j].z + x.z, was[j].w + x.w);
          } else {
            to[0] += x.x;
            if (n > 1) to[1] += x.y;
            if (n > 2) to[2] += x.z;
          }
        }
      }
    } else {
      __syncwarp();
      // eight rows at a time, so that their reads do not wait for one another (one by one:
      // 40 us and not 35 at 30000 x 1001 x 200)
      constexpr int WORDS = COLS / 32;
      const int rows = min(32, g.M - row0);
      for (int i0 = 0; i0 < rows; i0 += 8) {
        C v[8][WORDS];
        C* out = static_cast<C*>(g.c) + (long long)(row0 + i0) * g.ldc + col + c0 + lane;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < WORDS; ++j) {
            const int at = (32 * j + lane) * (int)sizeof(C);
            v[i][j] = *reinterpret_cast<const C*>(stage + (i0 + i) * 128 + (((at >> 4) ^ i) << 4) + (at & 15));
          }
        if constexpr (ADD) {
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = i0 + i < rows && col + c0 + lane < g.N ? out[i * g.ldc] : 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i][0] = o[i] + v[i][0];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < WORDS; ++j)
            if (i0 + i < rows && col + c0 + 32 * j + lane < g.N) out[i * g.ldc + 32 * j] = v[i][j];
      }
    }
  }
}
// Every copy out must be done before the CTA exits.
__device__ __forceinline__ void stores_done(const MmArgs& g) {
  if (g.tma && (threadIdx.x & 31) == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// ---------------------------------------------------------------------------
// Small products: a tile of 128 x BN, its blocks of K split over a cluster
// ---------------------------------------------------------------------------
// Where tiles are too few for the SMs, or one side is short (single tokens: the
// weight's rows then take the tile's 128 and the tokens its columns, SWAP).  The
// CTAs of a cluster take a run of the blocks of K each; then each adds up a part of
// the tile, out of all CTAs' shared memory in their order, and writes it.  One token x
// [12288, 2048], 25 MB, 8.0 us in a graph, of which 4 begin and end it; 640 x 1160 x 40000 with
// a scale for each column 64 us, split in five (twice that unsplit).
constexpr int kSmallThreads = 320;         // 8 warps that scale, then the copying and the issuing warp
constexpr int kCopyWarp = 8, kIssueWarp = 9;

// DUAL: two CTAs an SM, where there are more of them than SMs (BN = 32).
template <int BN, bool DUAL>
struct SmallTraits {
  static constexpr int P_BYTES = 128 * kKb, Q_BYTES = BN * kKb, STAGE = P_BYTES + Q_BYTES;
  static constexpr int STAGES = BN == 128 ? 5 : BN == 64 ? 7 : DUAL ? 4 : 9;
  static constexpr int AHEAD = DUAL ? 12 : 16;             // blocks whose scales are under way: a first read of memory's time
  static constexpr int BUFS = BN == 128 ? 4 : 8;
  static constexpr int TMEM = BUFS * BN;
  static constexpr int SMEM_USED = STAGES * STAGE + AHEAD * 2 * 256 * 4 + 1024;
  // two CTAs an SM, and none beside a kernel that takes all of its tensor memory (105 KB are used)
  static constexpr int SMEM = DUAL ? 110 * 1024 : SMEM_USED;
  static_assert(SMEM_USED <= SMEM && !fits_beside_owner(SMEM), "beside a kernel that takes all tensor memory");
  static_assert(!DUAL || (2 * (SMEM + kCtaSmem + 512) <= kSmSmem && 2 * TMEM <= 512), "two CTAs an SM (512: the barriers)");
  static_assert(STAGES * STAGE >= 128 * BN * 4, "the tile's sums take the stages' place");
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cta_meets() { asm volatile("bar.sync 0;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 16 bytes of shared memory of the cluster's CTA `rank`, at this CTA's address `at`.
__device__ __forceinline__ float4 cluster_load(uint32_t at, uint32_t rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [a];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(at), "r"(rank)
      : "memory");
  return v;
}
// Four neighbouring values of C from (row, col), those inside it.
template <bool F32>
__device__ __forceinline__ void store4(const MmArgs& g, int rows, int cols, int row, int col, float4 v) {
  if (row >= rows || col >= cols) return;
  const float x[4] = {v.x, v.y, v.z, v.w};
  const long long at = (long long)row * g.ldc + col;
  if constexpr (F32) {
    float* out = static_cast<float*>(g.c) + at;
    if (g.vec && col + 4 <= cols) {
      float4 o = v;
      if (g.accumulate) {
        o = *reinterpret_cast<const float4*>(out);
        o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
      }
      *reinterpret_cast<float4*>(out) = o;
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col + i < cols) out[i] = g.accumulate ? out[i] + x[i] : x[i];
  } else {
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(g.c) + at;
    if (g.vec && col + 4 <= cols) {
      *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col + i < cols) out[i] = __float2bfloat16_rn(x[i]);
  }
}

// g is that of the tile's rows (M, sa: b's with SWAP) and columns (N, sb).
// COLV: a scale for each column; else one for 128 of them.
template <int BN, bool DUAL, bool SWAP, bool COLV, bool F32>
__global__ void __launch_bounds__(kSmallThreads, DUAL ? 2 : 1)
    matmul_small_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ, MmArgs g, Ctl ctl) {
  using T = SmallTraits<BN, DUAL>;
  constexpr int NST = T::STAGES, NB = T::BUFS, HALF = BN / 2, AHEAD = T::AHEAD;
  extern __shared__ uint8_t raw[];
  uint8_t* ring = smem_align1024(raw);
  __shared__ uint64_t full[NST], empty[NST], sums[NB], freed[NB], drain;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  float* scales = reinterpret_cast<float*>(ring + NST * T::STAGE);     // [slot][rows', columns'][thread]
  volatile int* abort_flag = &abort_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned int kid = KID_MATMUL << 8;
  const int rank = g.split > 1 ? (int)cluster_rank() : 0, tile = (int)blockIdx.x / g.split;
  const int row0 = (tile % g.tm) * 128, col0 = (tile / g.tm) * BN;
  const int kb0 = (int)((long long)g.kbs * rank / g.split), kbs = (int)((long long)g.kbs * (rank + 1) / g.split) - kb0;
  // The first copies are under way while the tensor memory is allotted: every warp
  // does what it can before it meets the others.
  uint32_t tmem = 0;
  auto begin = [&] {
    tc_fence_before();
    cta_meets();
    tc_fence_after();
    tmem = *reinterpret_cast<volatile uint32_t*>(&tmem_slot);
  };
  bool ok = true;

  if (warp == kCopyWarp) {
    int n = 0;
    auto load = [&](int s) {
      mbar_arrive_expect_tx(&full[s], T::STAGE);
      tma_load_2d(ring + s * T::STAGE, &tmP, &full[s], (kb0 + n) * kKb, row0);
      tma_load_2d(ring + s * T::STAGE + T::P_BYTES, &tmQ, &full[s], (kb0 + n) * kKb, col0);
    };
    if (lane == 0) {
      for (int i = 0; i < NST; ++i) {
        mbar_init(&full[i], 1);
        mbar_init(&empty[i], 1);
      }
      for (int i = 0; i < NB; ++i) {
        mbar_init(&sums[i], 1);
        mbar_init(&freed[i], 8);
      }
      mbar_init(&drain, 1);
      abort_word = 0;
      fence_mbar_init();
      cudaGridDependencySynchronize();
      for (; n < kbs && n < NST; ++n) load(n);
    }
    __syncwarp();
    begin();
    if (lane == 0) {
      for (; n < kbs; ++n) {
        if (!mbar_wait(&empty[n % NST], (uint32_t)(n / NST - 1) & 1u, abort_flag, ctl, kid | W_EMPTY)) break;
        load(n % NST);
      }
      // every copy this thread started must land before the CTA exits
      for (int i = n > NST ? n - NST : 0; i < n; ++i)
        mbar_wait(&full[i % NST], (uint32_t)(i / NST) & 1u, nullptr, ctl, kid | W_DRAIN);
    }
  } else if (warp == kIssueWarp) {
    tmem_alloc(&tmem_slot, T::TMEM);
    tmem_relinquish();
    cudaTriggerProgrammaticLaunchCompletion();
    begin();
    const uint64_t p0 = sdesc_sw128(smem_u32(ring), 16, 1024);
    const uint64_t q0 = sdesc_sw128(smem_u32(ring + T::P_BYTES), 16, 1024);
    // a wait costs 200 clocks even where there is nothing to wait for: the next block's
    // barriers are tested ahead, beside the issuing of this one's products
    uint32_t here = 0, room = 1;
    for (int n = 0; n < kbs; ++n) {
      const int s = n % NST, buf = n % NB;
      ok = mbar_wait_warp_tested(&full[s], (uint32_t)(n / NST) & 1u, here, abort_flag, ctl, kid | W_FULL);
      if (ok && n >= NB)
        ok = mbar_wait_warp_tested(&freed[buf], (uint32_t)(n / NB - 1) & 1u, room, abort_flag, ctl, kid | W_FREE);
      if (!ok) break;
      here = mbar_test(&full[(n + 1) % NST], (uint32_t)((n + 1) / NST) & 1u);
      room = n + 1 >= NB ? mbar_test(&freed[(n + 1) % NB], (uint32_t)((n + 1) / NB - 1) & 1u) : 1u;
      tc_fence_after();
      const uint64_t p = desc_off(p0, (uint32_t)s * T::STAGE), q = desc_off(q0, (uint32_t)s * T::STAGE);
#pragma unroll
      for (int k = 0; k < kKb / 32; ++k)
        mma_f8_w(tmem + (uint32_t)buf * BN, desc_off(p, k * 32), desc_off(q, k * 32), g.idesc, k > 0 ? 1u : 0u);
      mma_commit_w(&sums[buf]);
      mma_commit_w(&empty[s]);
    }
    mma_commit_w(&drain);
    mbar_wait_warp(&drain, 0, nullptr, ctl, kid | W_DRAIN);
  } else {
    // warps 0-3: the first half of the tile's columns, warps 4-7 the second
    const int half = warp >> 2, r = (warp & 3) * 32 + lane, row = row0 + r, col = col0 + half * HALF;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const bool in = row < g.M, col_in = COLV ? r < HALF && col + r < g.N : col < g.N;
    const float* pa = g.sa + (in ? row >> g.sa_shift : 0) + kb0 * g.sa_ld;
    const float* pb = g.sb + (col_in ? (COLV ? col + r : col) >> g.sb_shift : 0) + kb0 * g.sb_ld;
    uint64_t acc[HALF / 2];
#pragma unroll
    for (int j = 0; j < HALF / 2; ++j) acc[j] = 0ull;
    // a thread brings in the scales of its row and of a column, AHEAD blocks before their use
    const int me = (int)threadIdx.x;
    auto fetch = [&](int n) {
      if (n < kbs) {
        copy4(scales + (n % AHEAD) * 512 + me, in ? pa + n * g.sa_ld : g.sa, in);
        copy4(scales + (n % AHEAD) * 512 + 256 + me, col_in ? pb + n * g.sb_ld : g.sb, col_in);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    cudaGridDependencySynchronize();
    for (int i = 0; i < AHEAD - 2; ++i) fetch(i);
    begin();
    uint32_t here = 0;                         // the next block's sums are known to be complete
    // a failed wait: the loop goes on, past the barriers, without work
    for (int n = 0; n < kbs; ++n) {
      const int buf = n % NB;
      asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD - 3) : "memory");
      if (COLV) asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
      fetch(n + AHEAD - 2);
      const float* w = scales + (n % AHEAD) * 512 + 256;
      const float f = COLV ? scales[(n % AHEAD) * 512 + me] : scales[(n % AHEAD) * 512 + me] * w[me];
      if (ok) ok = mbar_wait_warp_tested(&sums[buf], (uint32_t)(n / NB) & 1u, here, abort_flag, ctl, kid | W_SUMS);
      if (!ok) continue;
      tc_fence_after();
      const uint64_t f2 = f2_pack(f, f);
      w += half * 128;
      uint32_t v[HALF];
      const uint32_t from = tmem + lane_off + (uint32_t)(buf * BN + half * HALF);
      if constexpr (HALF == 16) tmem_ld16(from, v); else tmem_ld32(from, v);
      if constexpr (HALF == 64) tmem_ld32(from + 32, v + 32);
      tmem_ld_wait16(v);
      if constexpr (HALF > 16) tmem_pass<HALF - 16>(v + 16);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&freed[buf]);
      here = mbar_test(&sums[(n + 1) % NB], (uint32_t)((n + 1) / NB) & 1u);
#pragma unroll
      for (int j = 0; j < HALF / 2; j += 2) {
        uint64_t x = f2_pack(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
        uint64_t y = f2_pack(__uint_as_float(v[2 * j + 2]), __uint_as_float(v[2 * j + 3]));
        if (COLV) {
          const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(w + 2 * j);
          x = mul2(x, c.x);
          y = mul2(y, c.y);
        }
        acc[j] = fma2(x, f2, acc[j]);
        acc[j + 1] = fma2(y, f2, acc[j + 1]);
      }
    }
    // The sums take the stages' place: all products have read them.  SWAP: [column]
    // [row]; else [row][column], the 16-byte units of a row swapped by the row.
    if (ok) {
      float* part = reinterpret_cast<float*>(ring);
#pragma unroll
      for (int j = 0; j < HALF / 2; j += 2) {
        float x[4];
        f2_unpack(acc[j], x[0], x[1]);
        f2_unpack(acc[j + 1], x[2], x[3]);
        const int c = half * HALF + 2 * j;
        if constexpr (SWAP) {
#pragma unroll
          for (int i = 0; i < 4; ++i) part[(c + i) * 128 + r] = x[i];
        } else {
          *reinterpret_cast<float4*>(part + r * BN + (((c >> 2) ^ (r & 7)) << 2)) = make_float4(x[0], x[1], x[2], x[3]);
        }
      }
    }
  }
  if (!ok) abort_word = 1;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssueWarp) tmem_dealloc(tmem, T::TMEM);
  if (g.split > 1) cluster_sync();
  // this CTA's part of the tile: SWAP: columns, else rows
  constexpr int UNITS = 32 * BN;                         // of 4 values
  const int first = UNITS * rank / g.split, last = UNITS * (rank + 1) / g.split;
  if (warp < 8 && !*abort_flag) {
    auto put = [&](int u, float4 v) {
      const int line = SWAP ? u / 32 : u / (BN / 4), q = SWAP ? u % 32 : u % (BN / 4);
      if constexpr (SWAP) store4<F32>(g, g.N, g.M, col0 + line, row0 + 4 * q, v);
      else store4<F32>(g, g.M, g.N, row0 + line, col0 + 4 * q, v);
    };
    auto place = [&](int u) { return SWAP ? u : u / (BN / 4) * (BN / 4) + (u % (BN / 4) ^ (u / (BN / 4) & 7)); };
    if (g.split == 1) {
      const float4* part = reinterpret_cast<const float4*>(ring);
#pragma unroll 4
      for (int i = 0; i < UNITS / 256; ++i) {
        const int u = i * 256 + (int)threadIdx.x;
        put(u, part[place(u)]);
      }
    } else {
      // all CTAs' parts are asked for before the first is added
      for (int u = first + (int)threadIdx.x; u < last; u += 256) {
        const uint32_t at = smem_u32(ring) + 16u * (uint32_t)place(u);
        float4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < g.split) x[k] = cluster_load(at, (uint32_t)k);
        float4 v = x[0];
#pragma unroll
        for (int k = 1; k < 8; ++k)
          if (k < g.split) v.x += x[k].x, v.y += x[k].y, v.z += x[k].z, v.w += x[k].w;
        put(u, v);
      }
    }
  }
  if (g.split > 1) cluster_sync();                       // no CTA leaves while its sums are read
}

// The kernel may come before the one in front of it on the stream is done, and lets the
// next product come early in its turn, once each CTA has its tensor memory (what comes may take the rest
// of an SM's, and keeps it until this kernel is done): it waits for that one (cudaGridDependencySynchronize) before it
// touches memory that others use.  What it reads then is not read-only while it runs, so
// nothing here goes by way of the read-only path.  Back to back a call takes 2 to 3 us less
// (one token x [2048, 2048]: 8.2 -> 5.6 us).
template <typename... P, typename... A>
cudaError_t launch_early(void (*kern)(P...), unsigned grid, unsigned block, size_t smem, unsigned cluster, cudaStream_t st,
                         const A&... args) {
  cudaLaunchAttribute at[2]{};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}
template <int BN, bool DUAL, bool SWAP, bool COLV, bool F32>
cudaError_t small_t(const CUtensorMap& tmP, const CUtensorMap& tmQ, const MmArgs& g, const Ctl& ctl, cudaStream_t st) {
  using T = SmallTraits<BN, DUAL>;
  auto kern = matmul_small_kernel<BN, DUAL, SWAP, COLV, F32>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, T::SMEM);
  if (e != cudaSuccess) return e;
  return launch_early(kern, (unsigned)(g.tm * g.tn * g.split), kSmallThreads, T::SMEM, (unsigned)g.split, st, tmP, tmQ, g, ctl);
}
template <int BN, bool DUAL, bool SWAP>
cudaError_t small_of(const CUtensorMap& tmP, const CUtensorMap& tmQ, const MmArgs& g, bool colv, bool f32, const Ctl& ctl,
                     cudaStream_t st) {
  if (colv)
    return f32 ? small_t<BN, DUAL, SWAP, true, true>(tmP, tmQ, g, ctl, st) : small_t<BN, DUAL, SWAP, true, false>(tmP, tmQ, g, ctl, st);
  return f32 ? small_t<BN, DUAL, SWAP, false, true>(tmP, tmQ, g, ctl, st) : small_t<BN, DUAL, SWAP, false, false>(tmP, tmQ, g, ctl, st);
}
template <int BN, bool SWAP>
cudaError_t small_pick(const CUtensorMap& tmP, const CUtensorMap& tmQ, const MmArgs& g, bool colv, bool f32, const Ctl& ctl,
                       bool dual, cudaStream_t st) {
  if constexpr (BN == 32) {
    if (dual) return small_of<BN, true, SWAP>(tmP, tmQ, g, colv, f32, ctl, st);
  }
  return small_of<BN, false, SWAP>(tmP, tmQ, g, colv, f32, ctl, st);
}

// ---------------------------------------------------------------------------
// Pairs of CTAs: a tile of 256 x 256
// ---------------------------------------------------------------------------
// The two CTAs of a cluster, on neighbouring SMs, work on one tile of C: each
// holds 128 rows of a and 128 rows of b of a block of K, and the tensor cores of
// both SMs run one product of M = 256, N = 256 that the first CTA issues; each
// CTA gets the sums of its own 128 rows.  An SM so reads 32 KB of operands from
// shared memory for the 512 clocks of a block, and takes in as much: with a tile
// of its own, 128 x 128, it would be twice that, more than shared memory gives.
// Measured: 8192^3 429 us, 2.56 PFLOP/s (526 with a scale for each column); 61440 x 6144
// x 2048 652 us, 2.37; 6144 x 2048 x 17154 with a scale for each column 235 us, 1.83.  A
// block takes 850 clocks and not 512: its products, word of them, the sums' way into
// registers and word of that to the first CTA follow each other, over two buffers.
// With the same inputs again and again 8192^3 took 414 us, without
// b's copies 406, with half of the products 371.
constexpr int kPairThreads = 384;          // 4 warps that copy and issue, 8 that scale
constexpr int kPairStages = 5, kPairHalf = 128 * kKb, kPairStage = 2 * kPairHalf;
constexpr int kScaleSlots = 8, kScaleWords = 384;     // scales of a block: see the scale warp
constexpr int kPairSmem = kPairStages * kPairStage + kStoreBytes + kScaleSlots * kScaleWords * 4 + 1024;
static_assert(!fits_beside_owner(kPairSmem), "beside a kernel that takes all tensor memory");

// What the first CTA learns of the second, at the cluster's scope.
// Operands: the second CTA's tensor copies count on the first one's barrier themselves,
// and the issuing warp acquires.
__device__ __forceinline__ void pair_load_2d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int x, int y) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %4, 0;\n\t"
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], "
      "[a];\n\t}" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}
// Tensor memory that has been read: an arrival on the barrier at this place in the first
// CTA.  It needs the order of the two threads' instructions and of their tensor memory
// accesses, which the tcgen05 fences on both sides give, and hands over no memory, so it
// is relaxed; a release of the cluster's scope takes some 800 clocks a block (8192^3 782 us and
// not 400; the acquire on the other side takes none).
__device__ __forceinline__ void mbar_arrive_first(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %0, 0;\n\t"
      "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [a];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void pair_alloc(uint32_t* slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void pair_mma_w(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b32 r;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on the barrier at this place in both CTAs when all products issued so far are done.
__device__ __forceinline__ void pair_commit_w(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\t.reg .b16 m;\n\t"
      "mov.b16 m, 3;\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(
          smem_u32(bar))
      : "memory");
}
// Tiles in the order they are worked on: `group` columns of tiles at a time,
// row by row, so that the tiles under work share rows of a, and the group's
// rows of b stay in L2 while all of a passes once.
__device__ __forceinline__ void tile_at(const MmArgs& g, int t, int* m, int* n) {
  const int per = g.group * g.tm, first = t / per * g.group, wide = min(g.group, g.tn - first), i = t % per;
  *m = i / wide;
  *n = first + i % wide;
}

template <bool COLV, bool F32, bool ADD>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    matmul_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ CUtensorMap tmC, MmArgs g, Ctl ctl) {
  constexpr int NST = kPairStages, BN = 256;
  extern __shared__ uint8_t raw[];
  uint8_t* ring = smem_align1024(raw);
  float* scales = reinterpret_cast<float*>(ring + NST * kPairStage + kStoreBytes);   // [slot][kScaleWords]
  __shared__ uint64_t full[NST], empty[NST], sums[2], freed[2], drain;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const unsigned int kid = KID_MATMUL << 8;
  // Every warp meets the others once it has done what they wait for.  (First copies and
  // scales before that, as small products have them: 14.4 and not 12.4 us at 4864 x
  // 1000 x 1160, the CTAs meet later.)
  uint32_t tmem = 0;
  auto begin = [&] {
    tc_fence_before();
    cta_meets();
    cluster_sync();
    tc_fence_after();
    tmem = *reinterpret_cast<volatile uint32_t*>(&tmem_slot);
    cudaGridDependencySynchronize();
  };
  const int tiles = g.tm * g.tn, t0 = (int)blockIdx.x >> 1, step = (int)gridDim.x >> 1;

  if (warp < 4) {
    regs_dec<72>();
    if (warp == 0) {
      uint32_t n = 0;
      int t = t0, kb = 0, row = 0, col = 0;
      auto load = [&] {                              // the next block, to a slot that is free
        if (kb == 0) {
          int tm, tn;
          tile_at(g, t, &tm, &tn);
          row = tm * 256 + (int)rank * 128, col = tn * 256 + (int)rank * 128;
        }
        const int s = (int)(n % NST);
        // the second CTA's bytes may come before this: the slot's phase waits for the arrival all the same
        if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kPairStage);
        pair_load_2d(ring + s * kPairStage, &tmA, &full[s], kb * kKb, row);
        pair_load_2d(ring + s * kPairStage + kPairHalf, &tmB, &full[s], kb * kKb, col);
        ++n;
        if (++kb == g.kbs) kb = 0, t += step;
      };
      if (lane == 0) {
        for (int i = 0; i < NST; ++i) {
          mbar_init(&full[i], 1);                    // the first CTA's, for both CTAs' copies
          mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
          mbar_init(&sums[i], 2);                     // the products, and the scales
          mbar_init(&freed[i], rank == 0 ? 9 : 8);   // the first CTA's: its 8 warps, and word of the other's
        }
        mbar_init(&drain, 1);
        abort_word = 0;
        fence_mbar_init();
      }
      __syncwarp();
      begin();
      if (lane > 0) t = tiles;                       // one lane copies
      while (t < tiles && n < NST) load();
      bool ok = true;
      while (t < tiles) {
        ok = mbar_wait(&empty[n % NST], (n / NST - 1) & 1u, abort_flag, ctl, kid | W_EMPTY);
        if (!ok) break;
        load();
      }
      // Every copy of the pair must land before its CTAs exit, which they do together.  The
      // first CTA's barriers count those of both.  Blocks that only the second has asked for,
      // after a wait that gave up, get the time that a copy takes, many times over.
      if (rank == 0) {
        for (uint32_t i = n > NST ? n - NST : 0u; i < n; ++i)
          mbar_wait<true>(&full[i % NST], (i / NST) & 1u, nullptr, ctl, kid | W_DRAIN);
      }
      if (!ok) {
        const uint64_t from = globaltimer();
        while (globaltimer() - from < 10000000ull) __nanosleep(10000);
      }
    } else if (warp == 1 && rank == 1) {
      pair_alloc(&tmem_slot, 2 * BN);
      cudaTriggerProgrammaticLaunchCompletion();
      begin();
      // the first CTA's last arrival here must land before this CTA exits
      mbar_wait_warp(&drain, 0, nullptr, ctl, kid | W_DRAIN);
    } else if (warp == 2 && rank == 1) {
      // Tell the first CTA which of this one's sums have been read.  (The 8 warps that read them would
      // stand still for an arrival at the other CTA, 210 clocks: 576 -> 513 us at 8192^3.)
      begin();
      uint32_t n = 0;
      bool ok = true;
      for (int t = t0; ok && t < tiles; t += step) {
        for (int kb = 0; kb < g.kbs; ++kb, ++n) {
          ok = mbar_wait_warp(&freed[n & 1u], (n / 2) & 1u, abort_flag, ctl, kid | W_FREE);
          if (!ok) break;
          tc_fence_after();                          // behind the reads that the 8 warps told of
          tc_fence_before();
          if (lane == 0) mbar_arrive_first(&freed[n & 1u]);
        }
      }
    } else if (warp == 3) {
      // The scale warp: a block's scales into a slot in shared memory, four blocks
      // ahead and beside what the warp does: those of the 128 rows, and then (COLV) of the
      // 256 columns; else sa sb for the rows and the first 128 columns, and the others.  A slot is free when its block's scales
      // are read: at block n the products of block n - 2 are done, which waited for the
      // sums of block n - 4 to be read, and a warp reads the scales before it says so.
      // (Loads into registers and then stores held a block up by 660 clocks with a
      // scale for each column: 359 -> 237 us at 6144 x 2048 x 17152.)
      constexpr int AHEAD = kScaleSlots - 4;
      int st = t0, skb = 0, a_left = 0, b_left = 0, slot = 0;
      const float *pa = nullptr, *pb = nullptr;
      const int a_step = g.sa_shift ? 0 : 32;        // 128 rows at a multiple of 128 share a scale, or have one each
      // of 16 columns, the 4 that a reading lane scales are neighbours: 8 i + 2 q + e goes to 4 q + 2 i + e
      const int spread = (lane & 16) + (lane >> 1 & 3) * 4 + (lane >> 3 & 1) * 2 + (lane & 1);
      auto fetch = [&] {
        if (st < tiles) {
          if (skb == 0) {
            int tm, tn;
            tile_at(g, st, &tm, &tn);
            const int row = tm * 256 + (int)rank * 128 + lane, col = tn * 256 + (COLV ? lane : 128 * (lane & 1));
            a_left = g.M - row;
            b_left = g.N - col;
            pa = g.sa + (a_left > 0 ? row >> g.sa_shift : 0);
            pb = g.sb + (b_left > 0 ? col >> g.sb_shift : 0);
          }
          float* to = scales + slot * kScaleWords;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool in = 32 * i < a_left;
            copy4(to + 32 * i + lane, in ? pa + i * a_step : g.sa, in);
          }
          if constexpr (COLV) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const bool in = 32 * i < b_left;
              copy4(to + 128 + 32 * i + spread, in ? pb + 32 * i : g.sb, in);
            }
          } else if (lane < 2) {
            copy4(to + 256 + lane, b_left > 0 ? pb : g.sb, b_left > 0);
          }
          slot = slot + 1 < kScaleSlots ? slot + 1 : 0;
          pa += g.sa_ld;
          pb += g.sb_ld;
          if (++skb == g.kbs) {
            skb = 0;
            st += step;
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      begin();
      for (int i = 0; i < AHEAD; ++i) fetch();
      uint32_t n = 0;
      bool ok = true;
      for (int t = t0; ok && t < tiles; t += step) {
        for (int kb = 0; kb < g.kbs; ++kb, ++n) {
          if (n >= 2) ok = mbar_wait_warp(&sums[n & 1u], (n / 2 - 1) & 1u, abort_flag, ctl, kid | W_SUMS);
          if (!ok) break;
          fetch();
          asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD) : "memory");
          __syncwarp();
          if constexpr (!COLV) {
            float* to = scales + (n % kScaleSlots) * kScaleWords;
            const float b0 = to[256], b1 = to[257];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float f = to[32 * i + lane];
              to[32 * i + lane] = f * b0;
              to[128 + 32 * i + lane] = f * b1;
            }
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(&sums[n & 1u]);
        }
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else if (warp == 1) {
      pair_alloc(&tmem_slot, 2 * BN);
      cudaTriggerProgrammaticLaunchCompletion();
      begin();
      const uint64_t a0 = sdesc_sw128(smem_u32(ring), 16, 1024);
      const uint64_t b0 = sdesc_sw128(smem_u32(ring + kPairHalf), 16, 1024);
      uint32_t n = 0, here = 0;                  // here: the next block's operands are known to be in place
      bool ok = true;
      for (int t = t0; ok && t < tiles; t += step) {
        for (int kb = 0; kb < g.kbs; ++kb, ++n) {
          const int s = (int)(n % NST), buf = (int)(n & 1u);
          ok = mbar_wait_warp_tested<true>(&full[s], (n / NST) & 1u, here, abort_flag, ctl, kid | W_FULL);
          if (ok && n >= 2) ok = mbar_wait_warp<true>(&freed[buf], (n / 2 - 1) & 1u, abort_flag, ctl, kid | W_FREE);
          if (!ok) break;
          tc_fence_after();
          const uint64_t a = desc_off(a0, (uint32_t)s * kPairStage), b = desc_off(b0, (uint32_t)s * kPairStage);
#pragma unroll
          for (int k = 0; k < kKb / 32; ++k)
            pair_mma_w(tmem + (uint32_t)buf * BN, desc_off(a, k * 32), desc_off(b, k * 32), g.idesc, k > 0 ? 1u : 0u);
          pair_commit_w(&sums[buf]);
          pair_commit_w(&empty[s]);
          here = mbar_test<true>(&full[(n + 1) % NST], ((n + 1) / NST) & 1u);
        }
      }
      pair_commit_w(&drain);
      mbar_wait_warp(&drain, 0, nullptr, ctl, kid | W_DRAIN);
    } else {                                         // warp 2 of the first CTA has nothing to do
      begin();
    }
  } else {
    regs_inc<216>();
    begin();
    // warps 4-7: the tile's first 128 columns, warps 8-11 the others
    const int half = (warp - 4) >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    uint32_t n = 0, here = 0;                  // here: the next block's sums are known to be complete
    bool ok = true;
    for (int t = t0; ok && t < tiles; t += step) {
      int tm, tn;
      tile_at(g, t, &tm, &tn);
      const int row0 = tm * 256 + (int)rank * 128 + (warp & 3) * 32, col = tn * 256 + half * 128;
      uint64_t acc[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = 0ull;
      for (int kb = 0; kb < g.kbs; ++kb, ++n) {
        const int buf = (int)(n & 1u);
        if (ok) ok = mbar_wait_warp_tested(&sums[buf], (n / 2) & 1u, here, abort_flag, ctl, kid | W_SUMS);
        if (!ok) break;
        tc_fence_after();
        const uint32_t from = tmem + lane_off + (uint32_t)(buf * BN + half * 128);
        const float* at = scales + (n % kScaleSlots) * kScaleWords;
        auto done = [&] {                      // this block's sums are in registers
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&freed[buf]);
          here = mbar_test(&sums[buf ^ 1], ((n + 1) / 2) & 1u);
        };
        if constexpr (COLV) {
          // 16 rows x 32 columns in turn, a lane with 4 rows and a quarter of the columns, so that it
          // reads 8 of the columns' scales for 32 sums (with a row of its own, 32: 64 KB out of shared
          // memory a block and SM beside the operands' 32)
          uint32_t p[16], q[16];
          uint64_t rs[4];
          tmem_ld_rows16(from, p);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float f = at[(warp & 3) * 32 + 8 * i + lane / 4];
            rs[i] = f2_pack(f, f);
          }
          const float* w = at + 128 + half * 128 + (lane & 3) * 4;
          auto add = [&](const uint32_t* v, const uint64_t* cs, int c, int h) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              uint64_t& a = acc[c * 16 + h * 8 + j];
              a = fma2(mul2(f2_pack(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), cs[j / 2]), rs[2 * h + j % 2], a);
            }
          };
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const ulonglong2 c0 = *reinterpret_cast<const ulonglong2*>(w + 32 * c);
            const ulonglong2 c1 = *reinterpret_cast<const ulonglong2*>(w + 32 * c + 16);
            const uint64_t cs[4] = {c0.x, c0.y, c1.x, c1.y};
            tmem_ld_wait16(p);
            tmem_ld_rows16(from + (16u << 16) + 32 * c, q);
            add(p, cs, c, 0);
            tmem_ld_wait16(q);
            if (c < 3) tmem_ld_rows16(from + 32 * c + 32, p); else done();
            add(q, cs, c, 1);
          }
        } else {
          // 32 and 16 columns in turn: the next ones come in while these are scaled
          uint32_t p[32], q[16];
          tmem_ld32(from, p);
          const float sc = at[half * 128 + r];
          const uint64_t sc2 = f2_pack(sc, sc);
          auto add = [&](const uint32_t* v, int c0, int pairs) {
#pragma unroll
            for (int j = 0; j < pairs; ++j)
              acc[c0 / 2 + j] =
                  fma2(f2_pack(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), sc2, acc[c0 / 2 + j]);
          };
          tmem_ld_wait32(p);
          tmem_ld16(from + 32, q);
          add(p, 0, 16);
          tmem_ld_wait16(q);
          tmem_ld32(from + 48, p);
          add(q, 32, 8);
          tmem_ld_wait32(p);
          tmem_ld16(from + 80, q);
          add(p, 48, 16);
          tmem_ld_wait16(q);
          tmem_ld32(from + 96, p);
          add(q, 80, 8);
          tmem_ld_wait32(p);
          done();
          add(p, 96, 16);
        }
      }
      if (ok) store_rows<F32, ADD, COLV>(g, &tmC, ring + NST * kPairStage + (warp - 4) * 4096, row0, col, acc);
    }
    stores_done(g);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) pair_dealloc(tmem, 2 * BN);
}

template <bool COLV, bool F32, bool ADD>
cudaError_t pair_t(const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmC, MmArgs g, const Ctl& ctl,
                   cudaStream_t st) {
  auto kern = matmul_pair_kernel<COLV, F32, ADD>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem);
  if (e != cudaSuccess) return e;
  g.tm = (g.M + 255) / 256;
  g.tn = (g.N + 255) / 256;
  // a group's rows of b: at most 32 MB of the L2's 129
  const long long rows = (32LL << 20) / ((long long)g.kbs * kKb);
  g.group = (int)(rows / 256 < 1 ? 1 : rows / 256 < g.tn ? rows / 256 : g.tn);
  const int tiles = g.tm * g.tn;
  return launch_early(kern, 2u * (unsigned)(tiles < kPairs ? tiles : kPairs), kPairThreads, kPairSmem, 1u, st, tmA, tmB, tmC, g,
                      ctl);
}

template <bool COLV>
cudaError_t pair_pick(const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmC, const MmArgs& g, bool f32,
                      const Ctl& ctl, cudaStream_t st) {
  if (!f32) return pair_t<COLV, false, false>(tmA, tmB, tmC, g, ctl, st);
  return g.accumulate ? pair_t<COLV, true, true>(tmA, tmB, tmC, g, ctl, st)
                      : pair_t<COLV, true, false>(tmA, tmB, tmC, g, ctl, st);
}

}  // namespace

// How a product is worked on: by pairs of CTAs or in small tiles, and there over
// how many CTAs, up to eight, a tile's blocks of K are split.  The times behind the choice
// are those measured (in 10 ns; 152 SMs): a block of K 0.34 us in a small tile and 0.47
// in a pair's (0.49 and 0.57 with a scale for each column), a tile's beginning and
// end 4.5 us, or 1.4 in a pair that goes on to the next tile; joining the sums 1.2 to
// 3.6 us; and a cluster of so many CTAs finds so many SMs at once (two CTAs each: the second
// row, for tiles of 32 columns, which then share 0.34 us a block and begin and end beside
// each other: one token x [24576, 2048] 24 -> 19 us, 13 by what came after).  Measured when chosen
// and estimated, split 1, 2, 3, 4, 5: 552 x 968 x 37776 112, 63, 47, 67, 62 us, 105, 57, 40, 61,
// 52; 640 x 1160 x 40000 with a scale for each column 138, 76, 102, 82, 69 us, 158, 83, 114, 88, 73.
MatmulPlan matmul_plan(const dsv_matmul& p) {
  MatmulPlan plan = {0, 0, 128, 1, 0, 0};
  const int kbs = (p.K + kKb - 1) / kKb;
  plan.swap = p.M <= 64 && p.M < p.N;
  const int rows = plan.swap ? p.N : p.M, cols = plan.swap ? p.M : p.N;
  const bool colv = (plan.swap ? p.a_rows : p.b_rows) == 1;
  plan.bn = cols <= 32 ? 32 : cols <= 64 ? 64 : 128;
  const long long tiles = (long long)((rows + 127) / 128) * ((cols + plan.bn - 1) / plan.bn);
  const int block = colv && plan.bn == 128 ? 49 : 34;
  static const int slots[2][8] = {{kSMs, kSMs, 138, 144, 140, 138, 105, 120}, {304, 304, 291, 296, 290, 276, 266, 288}};
  static const int join[8] = {0, 120, 120, 130, 150, 170, 250, 300};
  long long best = 0;
  for (int split = 1; split <= 8 && split <= kbs; ++split) {
    const int i = split - 1;
    const long long n = tiles * split, rounds = (n + slots[0][i] - 1) / slots[0][i];
    const long long waves = plan.bn == 32 ? (n + slots[1][i] - 1) / slots[1][i] : rounds;
    const long long time = rounds * ((kbs + i) / split) * block + waves * 450 + join[i] + (i > 0 && plan.bn == 128 ? 60 : 0);
    if (split == 1 || time < best) best = time, plan.split = split;
  }
  if (p.M > 128 && p.N > 128) {
    const long long pairs = (long long)((p.M + 255) / 256) * ((p.N + 255) / 256);
    const long long time = (pairs + kPairs - 1) / kPairs * ((long long)kbs * (p.b_rows == 1 ? 57 : 47) + 140) + 350;
    if (time <= best) plan.pair = 1, plan.split = 1;
  }
  plan.dual = plan.bn == 32 && tiles * plan.split > kSMs;
  plan.smem = plan.pair        ? kPairSmem
              : plan.dual      ? SmallTraits<32, true>::SMEM
              : plan.bn == 32  ? SmallTraits<32, false>::SMEM
              : plan.bn == 64  ? SmallTraits<64, false>::SMEM
                               : SmallTraits<128, false>::SMEM;
  return plan;
}

cudaError_t launch_matmul_fp8(const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap* tmC, const dsv_matmul& p,
                              bool a_e5, bool b_e5, const float* sa, const float* sb, const dsv_rows& c, const Ctl& ctl,
                              cudaStream_t st) {
  MmArgs g;
  g.M = p.M;
  g.N = p.N;
  g.kbs = (p.K + kKb - 1) / kKb;
  g.tm = (p.M + 127) / 128;
  g.tn = (p.N + 127) / 128;
  g.sa = sa;
  g.sb = sb;
  g.sa_ld = p.a_rows == 1 ? p.M : (p.M + 127) / 128;
  g.sb_ld = p.b_rows == 1 ? p.N : (p.N + 127) / 128;
  g.sa_shift = p.a_rows == 1 ? 0 : 7;
  g.sb_shift = p.b_rows == 1 ? 0 : 7;
  g.c = c.ptr;
  g.ldc = c.stride;
  g.accumulate = p.accumulate;
  g.group = 0;
  const bool f32 = c.type == DSV_F32;
  g.tma = tmC == nullptr ? 0 : (long long)p.N * (f32 ? 4 : 2) % 16 == 0 ? 2 : 1;
  const CUtensorMap& tm_c = tmC != nullptr ? *tmC : tmA;      // not used without
  g.split = 1;
  const int size = f32 ? 4 : 2;
  g.vec = reinterpret_cast<uintptr_t>(c.ptr) % (4 * size) == 0 && c.stride % 4 == 0;
  const MatmulPlan plan = matmul_plan(p);
  if (plan.pair) {
    g.idesc = idesc_f8(256, 256, a_e5, b_e5);
    return p.b_rows == 1 ? pair_pick<true>(tmA, tmB, tm_c, g, f32, ctl, st)
                         : pair_pick<false>(tmA, tmB, tm_c, g, f32, ctl, st);
  }
  g.split = plan.split;
  if (plan.swap) {
    g.M = p.N, g.N = p.M;
    g.sa = sb, g.sb = sa;
    const MmArgs h = g;
    g.sa_ld = h.sb_ld, g.sb_ld = h.sa_ld;
    g.sa_shift = h.sb_shift, g.sb_shift = h.sa_shift;
    g.idesc = idesc_f8(128, plan.bn, b_e5, a_e5);
  } else {
    g.idesc = idesc_f8(128, plan.bn, a_e5, b_e5);
  }
  g.tm = (g.M + 127) / 128;
  g.tn = (g.N + plan.bn - 1) / plan.bn;
  const bool colv = (plan.swap ? p.a_rows : p.b_rows) == 1;
  if (plan.swap)
    return plan.bn == 32 ? small_pick<32, true>(tmB, tmA, g, colv, f32, ctl, plan.dual, st)
                         : small_pick<64, true>(tmB, tmA, g, colv, f32, ctl, plan.dual, st);
  return plan.bn == 32   ? small_pick<32, false>(tmA, tmB, g, colv, f32, ctl, plan.dual, st)
         : plan.bn == 64 ? small_pick<64, false>(tmA, tmB, g, colv, f32, ctl, plan.dual, st)
                         : small_pick<128, false>(tmA, tmB, g, colv, f32, ctl, plan.dual, st);
}

// Rows of the boxes that a's and b's tensor maps have.
void matmul_boxes(const dsv_matmul& p, int* a, int* b) {
  const MatmulPlan plan = matmul_plan(p);
  *a = plan.pair || !plan.swap ? 128 : plan.bn;
  *b = plan.pair || plan.swap ? 128 : plan.bn;
}

}  // namespace dsv
