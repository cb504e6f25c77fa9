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

#include "dsv_launch.h"

namespace dsv {

namespace {

constexpr int kMmThreads = 320;            // 8 warps that scale, then the copying and the issuing warp
constexpr int kCopyWarp = 8, kIssueWarp = 9;
constexpr int kPairs = 76;                 // pairs of SMs
constexpr int kKb = 128;                   // elements and bytes of a block along K: one swizzle row

constexpr int kStoreBytes = 8 * 4096;       // on C's way out, 4 KB a warp

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

template <int BN>
struct MmTraits {
  static constexpr int BM = 128, STAGES = 5;
  static constexpr int A_BYTES = BM * kKb, B_BYTES = BN * kKb, STAGE = A_BYTES + B_BYTES;
  static constexpr int SMEM = STAGES * STAGE + kStoreBytes + 1024;
  static constexpr int TMEM = 2 * BN;
};

// A warp's part of C: 32 rows from `row0` (a lane has one of them), 2 PAIRS
// columns from `col`, by way of 4 KB of shared memory: 32 rows of 128 bytes, the
// 16-byte units of a row swapped by the row, as tensor copies with the 128-byte
// swizzle have them.  The tensor copy out runs beside the next tile; where C's
// rows do not lie on 16 bytes, or are added to, the warp writes row by row.
// (A lane that stores its row itself takes 32 lines an instruction: 13 % of a
// product with K = 2048.)
template <bool F32, int PAIRS>
__device__ __forceinline__ void store_rows(const MmArgs& g, const CUtensorMap* tmC, uint8_t* stage, int row0, int col,
                                           const uint64_t* acc) {
  constexpr int COLS = F32 ? 32 : 64;                    // columns of a chunk
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c0 = 0; c0 < 2 * PAIRS; c0 += COLS) {
    // the last chunk has left shared memory
    if (g.tma && lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
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
    } else {
      __syncwarp();
      const int rows = min(32, g.M - row0);
      for (int i = 0; i < rows; ++i) {
#pragma unroll
        for (int j = 0; j < COLS; j += 32) {
          const int c = j + lane, at = c * (F32 ? 4 : 2);
          const uint8_t* from = stage + i * 128 + (((at >> 4) ^ (i & 7)) << 4) + (at & 15);
          if (col + c0 + c < g.N) {
            if constexpr (F32) {
              float* out = static_cast<float*>(g.c) + (long long)(row0 + i) * g.ldc + col + c0 + c;
              const float v = *reinterpret_cast<const float*>(from);
              *out = g.accumulate ? *out + v : v;
            } else {
              static_cast<__nv_bfloat16*>(g.c)[(long long)(row0 + i) * g.ldc + col + c0 + c] =
                  *reinterpret_cast<const __nv_bfloat16*>(from);
            }
          }
        }
      }
    }
  }
}
// Every copy out must be done before the CTA exits.
__device__ __forceinline__ void stores_done(const MmArgs& g) {
  if (g.tma && (threadIdx.x & 31) == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// COLV: b has a scale for each row (a column of C); else one for 128.
template <int BN, bool COLV, bool F32>
__global__ void __launch_bounds__(kMmThreads, 1)
    matmul_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ CUtensorMap tmC, MmArgs g, Ctl ctl) {
  using T = MmTraits<BN>;
  constexpr int NST = T::STAGES, HALF = BN / 2;
  extern __shared__ uint8_t raw[];
  uint8_t* ring = smem_align1024(raw);
  __shared__ uint64_t full[NST], empty[NST], sums[2], freed[2], drain;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  __shared__ float colscale[2][2][HALF];
  volatile int* abort_flag = &abort_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned int kid = KID_MATMUL << 8;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sums[i], 1);
      mbar_init(&freed[i], 8);
    }
    mbar_init(&drain, 1);
    abort_word = 0;
    fence_mbar_init();
  }
  if (warp == kIssueWarp) {
    tmem_alloc(&tmem_slot, T::TMEM);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&tmem_slot);
  const int tiles = g.tm * g.tn;

  if (warp == kCopyWarp) {
    if (lane == 0) {
      uint32_t n = 0;
      bool ok = true;
      for (int t = (int)blockIdx.x; ok && t < tiles; t += (int)gridDim.x) {
        const int row = (t % g.tm) * T::BM, col = (t / g.tm) * BN;
        for (int kb = 0; kb < g.kbs; ++kb, ++n) {
          const int s = (int)(n % NST);
          if (n >= NST && !mbar_wait(&empty[s], (n / NST - 1) & 1u, abort_flag, ctl, kid | W_EMPTY)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[s], T::STAGE);
          tma_load_2d(ring + s * T::STAGE, &tmA, &full[s], kb * kKb, row);
          tma_load_2d(ring + s * T::STAGE + T::A_BYTES, &tmB, &full[s], kb * kKb, col);
        }
      }
      // every copy this thread started must land before the CTA exits
      for (uint32_t i = n > NST ? n - NST : 0u; i < n; ++i)
        mbar_wait(&full[i % NST], (i / NST) & 1u, nullptr, ctl, kid | W_DRAIN);
    }
  } else if (warp == kIssueWarp) {
    const uint64_t a0 = sdesc_sw128(smem_u32(ring), 16, 1024);
    const uint64_t b0 = sdesc_sw128(smem_u32(ring + T::A_BYTES), 16, 1024);
    uint32_t n = 0;
    bool ok = true;
    for (int t = (int)blockIdx.x; ok && t < tiles; t += (int)gridDim.x) {
      for (int kb = 0; kb < g.kbs; ++kb, ++n) {
        const int s = (int)(n % NST), buf = (int)(n & 1u);
        if (n >= 2) ok = mbar_wait_warp(&freed[buf], (n / 2 - 1) & 1u, abort_flag, ctl, kid | W_FREE);
        if (ok) ok = mbar_wait_warp(&full[s], (n / NST) & 1u, abort_flag, ctl, kid | W_FULL);
        if (!ok) break;
        tc_fence_after();
        const uint64_t a = desc_off(a0, (uint32_t)s * T::STAGE), b = desc_off(b0, (uint32_t)s * T::STAGE);
#pragma unroll
        for (int k = 0; k < kKb / 32; ++k)
          mma_f8_w(tmem + (uint32_t)buf * BN, desc_off(a, k * 32), desc_off(b, k * 32), g.idesc, k > 0 ? 1u : 0u);
        mma_commit_w(&empty[s]);
        mma_commit_w(&sums[buf]);
      }
    }
    mma_commit_w(&drain);
    mbar_wait_warp(&drain, 0, nullptr, ctl, kid | W_DRAIN);
  } else {
    // warps 0-3: the first half of the tile's columns, warps 4-7 the second
    const int half = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    uint32_t n = 0;
    bool ok = true;                            // a failed wait: the loops go on, past the barriers, without work
    for (int t = (int)blockIdx.x; t < tiles; t += (int)gridDim.x) {
      const int row = (t % g.tm) * T::BM + r, col = (t / g.tm) * BN + half * HALF;
      const bool in = row < g.M;
      const float* pa = g.sa + (row >> g.sa_shift);
      const float* pb = COLV ? g.sb + col + r : g.sb + (col >> 7);
      const bool col_in = COLV ? r < HALF && col + r < g.N : col < g.N;
      uint64_t acc[HALF / 2];
#pragma unroll
      for (int j = 0; j < HALF / 2; ++j) acc[j] = 0ull;
      float sa_next = in && g.kbs > 0 ? __ldg(pa) : 0.f, sb_next = col_in && g.kbs > 0 ? __ldg(pb) : 0.f;
      for (int kb = 0; kb < g.kbs; ++kb, ++n) {
        const int buf = (int)(n & 1u);
        const float sa = sa_next, sb = sb_next;
        if (kb + 1 < g.kbs) {
          sa_next = in ? __ldg(pa + (kb + 1) * g.sa_ld) : 0.f;
          sb_next = col_in ? __ldg(pb + (kb + 1) * g.sb_ld) : 0.f;
        }
        if (COLV) {
          if (r < HALF) colscale[half][buf][r] = sb;
          asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
        }
        if (ok) ok = mbar_wait_warp(&sums[buf], (n / 2) & 1u, abort_flag, ctl, kid | W_SUMS);
        if (!ok) continue;
        tc_fence_after();
        const float sc = COLV ? sa : sa * sb;
        const uint64_t sc2 = f2_pack(sc, sc);
#pragma unroll
        for (int c = 0; c < HALF / 32; ++c) {
          uint32_t p[32];
          tmem_ld32(tmem + lane_off + (uint32_t)(buf * BN + half * HALF + c * 32), p);
          tmem_ld_wait();
          if (c == HALF / 32 - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&freed[buf]);
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            uint64_t v = f2_pack(__uint_as_float(p[2 * j]), __uint_as_float(p[2 * j + 1]));
            if (COLV) v = mul2(v, *reinterpret_cast<const uint64_t*>(&colscale[half][buf][c * 32 + 2 * j]));
            acc[c * 16 + j] = fma2(v, sc2, acc[c * 16 + j]);
          }
        }
      }
      if (ok) store_rows<F32, HALF / 2>(g, &tmC, ring + NST * T::STAGE + warp * 4096, row - lane, col, acc);
    }
    stores_done(g);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssueWarp) tmem_dealloc(tmem, T::TMEM);
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
constexpr int kPairThreads = 384;          // 4 warps that copy and issue, 8 that scale
constexpr int kPairStages = 5, kPairHalf = 128 * kKb, kPairStage = 2 * kPairHalf;
constexpr int kScaleSlots = 4, kScaleWords = 384;     // scales of a block: see the scale warp
constexpr int kPairSmem = kPairStages * kPairStage + kStoreBytes + kScaleSlots * kScaleWords * 4 + 1024;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Arrive on the barrier at the same place in the cluster's first CTA.  What the
// arrival stands for (tensor memory read, operands in place) is ordered by the
// tcgen05 and copy instructions themselves; no thread reads memory that another
// CTA's thread wrote.  Release and acquire of the cluster's scope would cost a
// block 2350 clocks instead of the 900 it takes: each waits for all of the
// thread's memory accesses.
__device__ __forceinline__ void mbar_arrive_first(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %0, 0;\n\t"
      "mbarrier.arrive.shared::cluster.b64 _, [a];\n\t}" ::"r"(smem_u32(bar))
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
// Tiles in the order they are worked on: `group` columns of tiles at a time,
// row by row, so that the tiles under work share rows of a, and the group's
// rows of b stay in L2 while all of a passes once.
__device__ __forceinline__ void tile_at(const MmArgs& g, int t, int* m, int* n) {
  const int per = g.group * g.tm, first = t / per * g.group, wide = min(g.group, g.tn - first), i = t % per;
  *m = i / wide;
  *n = first + i % wide;
}

template <bool COLV, bool F32>
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
  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&full[i], rank == 0 ? 2 : 1);    // the first CTA's: its own copies, and word of the other's
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
  if (warp == 1) pair_alloc(&tmem_slot, 2 * BN);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&tmem_slot);
  const int tiles = g.tm * g.tn, t0 = (int)blockIdx.x >> 1, step = (int)gridDim.x >> 1;

  if (warp < 4) {
    regs_dec<72>();
    if (warp == 0 && lane == 0) {
      uint32_t n = 0;
      bool ok = true;
      for (int t = t0; ok && t < tiles; t += step) {
        int tm, tn;
        tile_at(g, t, &tm, &tn);
        const int row = tm * 256 + (int)rank * 128, col = tn * 256 + (int)rank * 128;
        for (int kb = 0; kb < g.kbs; ++kb, ++n) {
          const int s = (int)(n % NST);
          if (n >= NST && !mbar_wait(&empty[s], (n / NST - 1) & 1u, abort_flag, ctl, kid | W_EMPTY)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[s], kPairStage);
          tma_load_2d(ring + s * kPairStage, &tmA, &full[s], kb * kKb, row);
          tma_load_2d(ring + s * kPairStage + kPairHalf, &tmB, &full[s], kb * kKb, col);
        }
      }
      // every copy this thread started must land before the CTA exits
      for (uint32_t i = n > NST ? n - NST : 0u; i < n; ++i)
        mbar_wait(&full[i % NST], (i / NST) & 1u, nullptr, ctl, kid | W_DRAIN);
    } else if (warp == 1 && rank == 1) {
      // tell the first CTA which of this one's operands are here
      uint32_t n = 0;
      bool ok = true;
      for (int t = t0; ok && t < tiles; t += step) {
        for (int kb = 0; kb < g.kbs; ++kb, ++n) {
          const int s = (int)(n % NST);
          ok = mbar_wait_warp(&full[s], (n / NST) & 1u, abort_flag, ctl, kid | W_FULL);
          if (!ok) break;
          if (lane == 0) mbar_arrive_first(&full[s]);
        }
      }
      // the first CTA's last arrival here must land before this CTA exits
      mbar_wait_warp(&drain, 0, nullptr, ctl, kid | W_DRAIN);
    } else if (warp == 2 && rank == 1) {
      // and which of its sums have been read.  (The 8 warps that read them would
      // stand still for an arrival at the other CTA, 210 clocks: 576 -> 513 us at 8192^3.)
      uint32_t n = 0;
      bool ok = true;
      for (int t = t0; ok && t < tiles; t += step) {
        for (int kb = 0; kb < g.kbs; ++kb, ++n) {
          ok = mbar_wait_warp(&freed[n & 1u], (n / 2) & 1u, abort_flag, ctl, kid | W_FREE);
          if (!ok) break;
          if (lane == 0) mbar_arrive_first(&freed[n & 1u]);
        }
      }
    } else if (warp == 3) {
      // The scale warp: a block's scales, four blocks ahead in registers, into a
      // slot in shared memory.  One for each row and half of the columns, sa sb;
      // or (COLV) those of the 128 rows and then those of the 256 columns.  A slot
      // is free when the products of the block two before are done: they waited for
      // the sums of the block four before to be read, and its scales are read first.
      constexpr int NB = COLV ? 8 : 2;
      float ra[kScaleSlots][4], rb[kScaleSlots][NB];
      int st = t0, skb = 0, a_left = 0, b_left = 0;
      const float *pa = nullptr, *pb = nullptr;
      const int a_step = g.sa_shift ? 0 : 32;        // 128 rows at a multiple of 128 share a scale, or have one each
      auto fetch = [&](float* va, float* vb) {
        if (st >= tiles) return;
        if (skb == 0) {
          int tm, tn;
          tile_at(g, st, &tm, &tn);
          const int row = tm * 256 + (int)rank * 128 + lane, col = tn * 256 + (COLV ? lane : 0);
          a_left = g.M - row;
          b_left = g.N - col;
          pa = g.sa + (row >> g.sa_shift);
          pb = g.sb + (col >> g.sb_shift);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) va[i] = 32 * i < a_left ? __ldg(pa + i * a_step) : 0.f;
#pragma unroll
        for (int i = 0; i < NB; ++i) vb[i] = (COLV ? 32 : 128) * i < b_left ? __ldg(pb + (COLV ? 32 : 1) * i) : 0.f;
        pa += g.sa_ld;
        pb += g.sb_ld;
        if (++skb == g.kbs) {
          skb = 0;
          st += step;
        }
      };
#pragma unroll
      for (int i = 0; i < kScaleSlots; ++i) fetch(ra[i], rb[i]);
      const long long blocks = t0 < tiles ? (long long)((tiles - 1 - t0) / step + 1) * g.kbs : 0;
      bool ok = true;
      for (long long n0 = 0; ok && n0 < blocks; n0 += kScaleSlots) {
#pragma unroll
        for (int i = 0; i < kScaleSlots; ++i) {
          const long long n = n0 + i;
          if (!ok || n >= blocks) break;
          if (n >= 2) ok = mbar_wait_warp(&sums[i & 1], (uint32_t)(n / 2 - 1) & 1u, abort_flag, ctl, kid | W_SUMS);
          if (!ok) break;
          float* to = scales + i * kScaleWords + lane;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (COLV) {
              to[32 * j] = ra[i][j];
            } else {
              to[32 * j] = ra[i][j] * rb[i][0];
              to[128 + 32 * j] = ra[i][j] * rb[i][1];
            }
          }
          if constexpr (COLV) {
#pragma unroll
            for (int j = 0; j < NB; ++j) to[128 + 32 * j] = rb[i][j];
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sums[i & 1]);
          fetch(ra[i], rb[i]);
        }
      }
    } else if (warp == 1) {
      const uint64_t a0 = sdesc_sw128(smem_u32(ring), 16, 1024);
      const uint64_t b0 = sdesc_sw128(smem_u32(ring + kPairHalf), 16, 1024);
      uint32_t n = 0, here = 0;                  // here: the next block's operands are known to be in place
      bool ok = true;
      for (int t = t0; ok && t < tiles; t += step) {
        for (int kb = 0; kb < g.kbs; ++kb, ++n) {
          const int s = (int)(n % NST), buf = (int)(n & 1u);
          ok = mbar_wait_warp_tested(&full[s], (n / NST) & 1u, here, abort_flag, ctl, kid | W_FULL);
          if (ok && n >= 2) ok = mbar_wait_warp(&freed[buf], (n / 2 - 1) & 1u, abort_flag, ctl, kid | W_FREE);
          if (!ok) break;
          tc_fence_after();
          const uint64_t a = desc_off(a0, (uint32_t)s * kPairStage), b = desc_off(b0, (uint32_t)s * kPairStage);
#pragma unroll
          for (int k = 0; k < kKb / 32; ++k)
            pair_mma_w(tmem + (uint32_t)buf * BN, desc_off(a, k * 32), desc_off(b, k * 32), g.idesc, k > 0 ? 1u : 0u);
          pair_commit_w(&sums[buf]);
          pair_commit_w(&empty[s]);
          here = mbar_test(&full[(n + 1) % NST], ((n + 1) / NST) & 1u);
        }
      }
      pair_commit_w(&drain);
      mbar_wait_warp(&drain, 0, nullptr, ctl, kid | W_DRAIN);
    }
  } else {
    regs_inc<216>();
    // warps 4-7: the tile's first 128 columns, warps 8-11 the others
    const int half = (warp - 4) >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const float* my_scale = scales + (COLV ? r : half * 128 + r);
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
        // 32 and 16 columns in turn: the next ones come in while these are scaled
        uint32_t p[32], q[16];
        const uint32_t from = tmem + lane_off + (uint32_t)(buf * BN + half * 128);
        tmem_ld32(from, p);
        const float sc = my_scale[(n % kScaleSlots) * kScaleWords];
        const uint64_t sc2 = f2_pack(sc, sc);
        const float* w = scales + (n % kScaleSlots) * kScaleWords + 128 + half * 128;
        auto add = [&](const uint32_t* v, int c0, int pairs) {
#pragma unroll
          for (int j = 0; j < pairs; j += 2) {
            uint64_t v0 = f2_pack(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
            uint64_t v1 = f2_pack(__uint_as_float(v[2 * j + 2]), __uint_as_float(v[2 * j + 3]));
            if (COLV) {
              const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(w + c0 + 2 * j);
              v0 = mul2(v0, x.x);
              v1 = mul2(v1, x.y);
            }
            acc[c0 / 2 + j] = fma2(v0, sc2, acc[c0 / 2 + j]);
            acc[c0 / 2 + j + 1] = fma2(v1, sc2, acc[c0 / 2 + j + 1]);
          }
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
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&freed[buf]);
        here = mbar_test(&sums[buf ^ 1], ((n + 1) / 2) & 1u);
        add(p, 96, 16);
      }
      if (ok) store_rows<F32, 64>(g, &tmC, ring + NST * kPairStage + (warp - 4) * 4096, row0, col, acc);
    }
    stores_done(g);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) pair_dealloc(tmem, 2 * BN);
}

template <bool COLV, bool F32>
cudaError_t pair_t(const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmC, MmArgs g, const Ctl& ctl,
                   cudaStream_t st) {
  auto kern = matmul_pair_kernel<COLV, F32>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem);
  if (e != cudaSuccess) return e;
  g.tm = (g.M + 255) / 256;
  g.tn = (g.N + 255) / 256;
  // a group's rows of b: at most 32 MB of the L2's 129
  const long long rows = (32LL << 20) / ((long long)g.kbs * kKb);
  g.group = (int)(rows / 256 < 1 ? 1 : rows / 256 < g.tn ? rows / 256 : g.tn);
  const int tiles = g.tm * g.tn;
  kern<<<2 * (tiles < kPairs ? tiles : kPairs), kPairThreads, kPairSmem, st>>>(tmA, tmB, tmC, g, ctl);
  return cudaGetLastError();
}

template <int BN, bool COLV, bool F32>
cudaError_t matmul_t(const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmC, MmArgs g, const Ctl& ctl,
                   cudaStream_t st) {
  using T = MmTraits<BN>;
  auto kern = matmul_kernel<BN, COLV, F32>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, T::SMEM);
  if (e != cudaSuccess) return e;
  const int tiles = g.tm * g.tn;
  kern<<<tiles < 152 ? tiles : 152, kMmThreads, T::SMEM, st>>>(tmA, tmB, tmC, g, ctl);
  return cudaGetLastError();
}

}  // namespace

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
  g.idesc = idesc_f8(128, 128, a_e5, b_e5);
  if (p.M > 128 && p.N > 128) {
    g.idesc = idesc_f8(256, 256, a_e5, b_e5);
    if (p.b_rows == 1)
      return f32 ? pair_t<true, true>(tmA, tmB, tm_c, g, ctl, st) : pair_t<true, false>(tmA, tmB, tm_c, g, ctl, st);
    return f32 ? pair_t<false, true>(tmA, tmB, tm_c, g, ctl, st) : pair_t<false, false>(tmA, tmB, tm_c, g, ctl, st);
  }
  if (p.b_rows == 1)
    return f32 ? matmul_t<128, true, true>(tmA, tmB, tm_c, g, ctl, st) : matmul_t<128, true, false>(tmA, tmB, tm_c, g, ctl, st);
  return f32 ? matmul_t<128, false, true>(tmA, tmB, tm_c, g, ctl, st) : matmul_t<128, false, false>(tmA, tmB, tm_c, g, ctl, st);
}

}  // namespace dsv
