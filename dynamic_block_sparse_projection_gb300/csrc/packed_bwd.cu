// packed_bwd.cu — gradient of the packed-sequence attention, without atomics.
//
// With P_ij = exp(s_ij - lse_i) over the pairs that the forward's mask leaves:
//   D_i  = sum_c dO_ic O_ic,   dS_ij = P_ij (dO_i . v_j - D_i)
//   dV_j = sum_i P_ij dO_i,  dK_j = scale sum_i dS_ij q_i   (i over every query
//          head that shares the key head),  dQ_i = scale sum_j dS_ij k_j
//
// The dense companion of attn_bwd.cu, with its two kernels and their pipelines
// over packed.cuh's tiles (a query tile's rows are tokens x shared heads):
//   prepare  D_i and -lse_i log2(e) into 128-row slots, one per query tile.  A
//            row that saw no key (lse = -inf), and a row behind the tile's
//            tokens, gets -inf there, so its P is exp2(-inf) = 0.
//   rows     D_i = sum_j P_ij dP_ij instead, for the query tiles whose keys all
//            lie in one key tile (below).
//   kv       one CTA per key tile and key head, over the sequence's query
//            tiles: S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q.
//            Shared heads add up inside the product, and every output tile has
//            one writer.  With far fewer key tiles than SMs the query tiles of
//            each are split over several CTAs (bwd_splits) and the join kernel
//            adds their fp32 sums in order.
//   q        one CTA per SM over the query tiles, taking over the grid's other
//            CTAs as it goes (packed_fwd.cu): S = Q K^T, dP = dO V^T, dQ += dS K.
// S and dP are computed twice (seven products per tile pair instead of five),
// which buys results that do not depend on the order CTAs run in.
//
// P and dS are rounded to bf16, the type of the products' other operand; sums
// stay in fp32 in tensor memory.  Measured, d = 128: 24 heads of four clips of
// 515 to 8192 tokens, kv 1237 us (1722 TFLOP/s of its four products, 92 % of what
// a large library product reaches in a burst), q 960 us (1664 TFLOP/s), prepare
// 31 us; causal, 24 heads over 8 key heads, five clips of 64 to 6000 tokens, kv
// 380 us (1655), q 299 us (1577), prepare 27, rows 13; text (16 384 and 8192
// tokens against 226 and 512 keys, 24 heads), prepare 49 us (HBM), kv 187, q 152
// alone, most of it beside kv, the call 335.
// Tensor cores bound kv and q, under the power cap when calls follow closely.
//
// D_i from O.  O is bf16, so dO . O is off by some 2^-9 |dO| |O| / sqrt(d).  Over
// many keys O is small against the v_j and that vanishes beside the rounding
// of dS to bf16 (the tensor core's operand); over a handful of keys it does not:
// in sequences of 1 to 20 keys dQ and dK were off by up to twice what their own
// rounding to bf16 costs, with the rows kernel by 1.4 times, as everywhere else.
//
// Rows of a tile that belong to no token of it are other sequences' data.  As
// rows of the A operands they only reach accumulator rows that are not stored;
// as rows of the B operands they would meet a zero of P or dS, and 0 * NaN is
// not 0, so the last query tile of a sequence (kv) and its last key tile (q,
// K only) are zeroed from the end on in shared memory before the MMAs see them.
#include <math.h>

#include "packed.cuh"

namespace dsv {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kKVThreads = 320;        // producer, MMA issuer, 8 compute warps
constexpr int kQVWarp = 10;            // q kernel: V producer
constexpr int kQItemWarp = 11;         // q kernel: takes the work items
constexpr int kQThreads = 384;
constexpr int kAskAhead = 6;           // q kernel: key tiles before an item's last one at which the next is asked for
constexpr int kComputeThreads = 256;
constexpr int kRowsThreads = 160;      // rows kernel: 4 compute warps, one for copies and MMAs

// Whether the keys that a query tile sees (from token t0 of its sequence on) lie in one key tile.
__device__ __forceinline__ bool one_key_tile(const PackedGeom& g, const PackedSeq& q, int t0) {
  const int last = g.causal ? min(q.lk, q.lk - q.lq + t0 + min(g.TQ, q.lq - t0)) : q.lk;
  return last > 0 && last <= 128;
}

// ---------------------------------------------------------------------------
// D_i and -lse_i log2(e), 128 rows per query tile
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(256) packed_bwd_prep_kernel(const __grid_constant__ PackedGeom g,
                                                              const __nv_bfloat16* O, long long o_head,
                                                              long long o_tok, const __nv_bfloat16* dO,
                                                              long long d_head, long long d_tok,
                                                              const float* __restrict__ lse, float* __restrict__ Dw,
                                                              float* __restrict__ L2w, Ctl ctl) {
  constexpr int TPR = D / 8;             // threads per row, 16 bytes each
  constexpr int RPC = 256 / TPR;         // rows per pass
  const int slot = blockIdx.x, kvh = blockIdx.y;
  if (slot == 0 && kvh == 0 && threadIdx.x < 32) packed_check_ptrs(g, ctl, threadIdx.x);
  PackedSeq q;
  const bool found = packed_find(g, g.q_ptr, g.TQ, slot, q);
  const int t0 = found ? (slot - (q.q0 / g.TQ + q.s)) * g.TQ : 0;
  if (!found || t0 >= q.lq) {
    cudaGridDependencySynchronize();
    return;
  }
  const int rows = min(g.TQ, q.lq - t0) * g.group;
  const bool from_o = !one_key_tile(g, q, t0);   // else D is the rows kernel's
  const int c = threadIdx.x % TPR;
  const long long base = ((long long)kvh * g.nslot_q + slot) * 128;
  constexpr int BATCH = 4;               // rows of O and dO in flight per thread
  for (int r0 = threadIdx.x / TPR; r0 < 128; r0 += BATCH * RPC) {
    uint4 a[BATCH], b[BATCH];
    float L[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int r = r0 + k * RPC, rt = r / g.group, head = kvh * g.group + (r - rt * g.group);
      const long long tok = (long long)q.q0 + t0 + rt;
      a[k] = b[k] = make_uint4(0, 0, 0, 0);
      L[k] = -INFINITY;
      if (r < rows) {
        if (from_o) {
          a[k] = __ldcs(reinterpret_cast<const uint4*>(O + head * o_head + tok * o_tok) + c);
          b[k] = __ldcs(reinterpret_cast<const uint4*>(dO + head * d_head + tok * d_tok) + c);
        }
        if (c == 0) L[k] = lse[(long long)head * g.Tq + tok];
      }
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const uint32_t wa[4] = {a[k].x, a[k].y, a[k].z, a[k].w}, wb[4] = {b[k].x, b[k].y, b[k].z, b[k].w};
      float acc = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc = fmaf(__uint_as_float(wa[i] << 16), __uint_as_float(wb[i] << 16), acc);
        acc = fmaf(__uint_as_float(wa[i] & 0xFFFF0000u), __uint_as_float(wb[i] & 0xFFFF0000u), acc);
      }
#pragma unroll
      for (int o = TPR / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
      if (c == 0) {
        if (from_o) Dw[base + r0 + k * RPC] = acc;           // 0 behind the tile's rows
        L2w[base + r0 + k * RPC] = L[k] == -INFINITY ? -INFINITY : -L[k] * kLog2e;
      }
    }
  }
  cudaGridDependencySynchronize();       // what waits for this kernel waits for the rows kernel too
}

// 32 bf16 values of a row, a sector at a time where the rows' addresses allow it.
__device__ __forceinline__ void store_row32(__nv_bfloat16* dst, const uint32_t* w, bool wide) {
  if (wide) {
    st_global_32(dst, w);
    st_global_32(dst + 16, w + 8);
  } else {
#pragma unroll
    for (int p = 0; p < 4; ++p)
      reinterpret_cast<uint4*>(dst)[p] = make_uint4(w[4 * p], w[4 * p + 1], w[4 * p + 2], w[4 * p + 3]);
  }
}

enum : unsigned int {
  W_KV = 1, W_GFULL, W_GEMPTY, W_S, W_P, W_ACC, W_DRAIN, W_KFULL, W_VFULL, W_KVEMPTY, W_SPFREE, W_DSFULL, W_DSEMPTY,
  W_ITEM, W_ITEMFREE, W_TAIL, W_KVFULL
};

// ---------------------------------------------------------------------------
// D_i = sum_j P_ij dP_ij where a query tile's keys lie in one key tile
// ---------------------------------------------------------------------------
// One CTA per SM looks 128 slots at a time over for such tiles and takes them
// one after the other: S = Q K^T and dP = dO V^T, a row per thread.  Runs beside
// the prepare kernel, which leaves these tiles' D alone.  Rows of Q and dO that
// are no token of the tile reach only rows that are not kept; keys past a row's
// limit are left out by selection.
template <int D>
struct PRowsTraits {
  static constexpr int NCH = D / 64;
  static constexpr int CHUNK = 128 * 128;
  static constexpr int TILE = NCH * CHUNK;
  static constexpr int SMEM_USED = 1024 + 4 * TILE + 5 * 8 + 4 * 4 + 8;
  // at least 120 KB so that one CTA owns an SM (and its 512 TMEM columns)
  static constexpr int SMEM = SMEM_USED > 120 * 1024 ? SMEM_USED : 120 * 1024;
  static constexpr uint32_t TMEM_COLS = 512;      // two buffers of S and dP
};

template <int D>
__global__ void __launch_bounds__(kRowsThreads, 1)
    packed_bwd_rows_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmdO,
                           const __grid_constant__ PackedGeom g, const float* __restrict__ lse, float scale,
                           float* __restrict__ Dw, Ctl ctl) {
  using T = PRowsTraits<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  cudaTriggerProgrammaticLaunchCompletion();     // the prepare kernel may run beside this one
  uint8_t* sQ = smem_align1024(smem_raw);
  uint8_t* sdO = sQ + T::TILE;
  uint8_t* sK = sdO + T::TILE;
  uint8_t* sV = sK + T::TILE;
  uint64_t* full = reinterpret_cast<uint64_t*>(sV + T::TILE);   // the tiles landed
  uint64_t* acc_full = full + 1;                  // [2] S and dP in TMEM (and the tiles read)
  uint64_t* acc_free = full + 3;                  // [2]
  uint32_t* hits = reinterpret_cast<uint32_t*>(full + 5);       // [4] which of 128 slots
  uint32_t* tmem_slot = hits + 4;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned int kid = (unsigned int)KID_PACKED_ROWS << 8;
  const int total = g.Hkv * g.nslot_q;
  const float c2 = scale * kLog2e;
  bool ready = false, ok = true;                  // ready: the same in all threads
  uint32_t n = 0;                                 // tiles taken
  uint32_t tmem_base = 0;
  constexpr uint32_t tmem = 0;
  auto tile_of = [&](int idx, int& kvh, int& slot, PackedSeq& q, int& t0) -> bool {
    kvh = idx / g.nslot_q;
    slot = idx - kvh * g.nslot_q;
    if (!packed_find(g, g.q_ptr, g.TQ, slot, q)) return false;
    t0 = (slot - (q.q0 / g.TQ + q.s)) * g.TQ;
    return t0 < q.lq && one_key_tile(g, q, t0);
  };

  for (long long base = blockIdx.x; base < total; base += 128LL * gridDim.x) {
    auto index = [&](int bit) { return base + (long long)bit * gridDim.x; };
    if (warp < 4) {
      int kvh, slot, t0;
      PackedSeq q;
      const long long idx = index(threadIdx.x);
      const uint32_t hit = __ballot_sync(0xffffffffu, idx < total && tile_of((int)idx, kvh, slot, q, t0));
      if (lane == 0) hits[warp] = hit;
    }
    __syncthreads();
    if ((hits[0] | hits[1] | hits[2] | hits[3]) != 0u && !ready) {
      if (threadIdx.x == 0) {
        mbar_init(full, 1);
        for (int b = 0; b < 2; ++b) {
          mbar_init(&acc_full[b], 1);
          mbar_init(&acc_free[b], 128);
        }
        *abort_flag = 0;
        fence_mbar_init();
      }
      if (warp == 4) {
        tmem_alloc(tmem_slot, T::TMEM_COLS);
        tmem_relinquish();
      }
      tc_fence_before();
      __syncthreads();
      tc_fence_after();
      // one CTA owns the SM's whole TMEM, so its addresses start at 0 (attn_fwd.cu)
      tmem_base = *tmem_slot;
      ready = true;
      if (tmem_base != tmem) {
        if (threadIdx.x == 0) set_error(ctl, DSV_ERR_INTERNAL, blockIdx.x);
        ok = false;
      }
    }
#pragma unroll 1
    for (int w = 0; w < 4; ++w) {
#pragma unroll 1
      for (uint32_t left = hits[w]; ok && left != 0u; left &= left - 1u, ++n) {
        int kvh, slot, t0;
        PackedSeq q;
        tile_of((int)index(w * 32 + __ffs(left) - 1), kvh, slot, q, t0);
        const uint32_t b = n & 1u, use = n >> 1;
        if (warp == 4) {
          // the tiles are free when the MMAs before are done
          if (n > 0 && !mbar_wait_warp(&acc_full[b ^ 1u], ((n - 1) >> 1) & 1u, nullptr, ctl, kid | W_KVEMPTY)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            const uint32_t box = (uint32_t)(g.group * g.TQ) * D * 2;
            mbar_arrive_expect_tx(full, 2 * box + 2 * T::TILE);
            for (int c = 0; c < T::NCH; ++c) {
              tma_load_3d(sQ + c * T::CHUNK, &tmQ, full, c * 64, kvh * g.group, q.q0 + t0);
              tma_load_3d(sK + c * T::CHUNK, &tmK, full, c * 64, kvh, q.k0);
              tma_load_3d(sdO + c * T::CHUNK, &tmdO, full, c * 64, kvh * g.group, q.q0 + t0);
              tma_load_3d(sV + c * T::CHUNK, &tmV, full, c * 64, kvh, q.k0);
            }
          }
          // (its own copies: waited for whatever happens)
          const bool landed = mbar_wait_warp(full, n & 1u, nullptr, ctl, kid | W_KVFULL);
          if (!landed || !mbar_wait_warp(&acc_free[b], (use & 1u) ^ 1u, abort_flag, ctl, kid | W_SPFREE)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          tc_fence_after();
          constexpr uint32_t ID_S = idesc_bf16_f32(128, 128, false, false);
          const uint64_t dq = sdesc_sw128(smem_u32(sQ), 16, 1024), dk = sdesc_sw128(smem_u32(sK), 16, 1024);
          const uint64_t ddo = sdesc_sw128(smem_u32(sdO), 16, 1024), dv = sdesc_sw128(smem_u32(sV), 16, 1024);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t o = (kk >> 2) * T::CHUNK + (kk & 3) * 32;
            mma_ss_w(tmem + b * 256, desc_off(dq, o), desc_off(dk, o), ID_S, kk > 0 ? 1u : 0u);
            mma_ss_w(tmem + b * 256 + 128, desc_off(ddo, o), desc_off(dv, o), ID_S, kk > 0 ? 1u : 0u);
          }
          mma_commit_w(&acc_full[b]);
        } else {
          const int r = warp * 32 + lane, rt = r / g.group;
          const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
          const int ntok = min(g.TQ, q.lq - t0);
          const int head = kvh * g.group + (r - rt * g.group);
          const float L = rt < ntok ? lse[(long long)head * g.Tq + q.q0 + t0 + rt] : -INFINITY;
          const float nl = L == -INFINITY ? -INFINITY : -L * kLog2e;
          const int lim = g.causal ? min(q.lk, q.lk - q.lq + t0 + 1 + rt) : q.lk;
          if (!mbar_wait_warp(&acc_full[b], use & 1u, abort_flag, ctl, kid | W_S)) {
            ok = false;
            break;
          }
          tc_fence_after();
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t xs[32], xp[32];
            tmem_ld32(tmem + lane_off + b * 256 + c * 32, xs);
            tmem_ld32(tmem + lane_off + b * 256 + 128 + c * 32, xp);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (c * 32 + j < lim)
                sum[j & 3] = fmaf(ex2(fmaf(__uint_as_float(xs[j]), c2, nl)), __uint_as_float(xp[j]), sum[j & 3]);
          }
          tc_fence_before();
          mbar_arrive(&acc_free[b]);
          // a row without keys, and a row behind the tile's tokens: 0
          Dw[((long long)kvh * g.nslot_q + slot) * 128 + r] =
              rt < ntok && L != -INFINITY ? (sum[0] + sum[1]) + (sum[2] + sum[3]) : 0.f;
        }
      }
    }
    __syncthreads();                              // `hits` has been read
  }
  if (!ready) return;
  if (warp == 4 && n > 0) mbar_wait_warp(&acc_full[(n - 1) & 1u], ((n - 1) >> 1) & 1u, nullptr, ctl, kid | W_DRAIN);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 4) tmem_dealloc(tmem_base, T::TMEM_COLS);
}

// ---------------------------------------------------------------------------
// dK, dV: one CTA per key tile and key head
// ---------------------------------------------------------------------------
template <int D>
struct PKVTraits {
  static constexpr int NCH = D / 64;
  static constexpr int CHUNK = 128 * 128;
  static constexpr int TILE = NCH * CHUNK;
  // Q is read by S^T (early) and dK (late), dO by dP^T and dV (earlier): rings
  // of their own, each slot given back as its last product is done.  A tile's
  // copies then have about one and a half pairs' time to arrive; with two
  // common stages they had half a pair's, and a pair took 3465 clocks instead
  // of 2650 where Q and dO come from HBM.
  static constexpr int NQ = 3, ND = 2;
  static constexpr int VEC_BYTES = 128 * 4;                    // -lse2 or D of a query tile
  static constexpr int NBAR = 2 + 2 * NQ + 3 * ND + 7 + 2;
  static constexpr int SMEM_USED = (2 + NQ + ND) * TILE + 2 * ND * VEC_BYTES + NBAR * 8 + 16;
  static_assert(SMEM_USED <= 227 * 1024, "dK/dV tiles exceed shared memory");
  static constexpr int SMEM = SMEM_USED > 120 * 1024 ? SMEM_USED : 120 * 1024;
  // TMEM: S^T at 0, dP^T at 128, dV at 256, dK at 256 + D; P^T and dS^T (bf16
  // pairs) go over the columns they were read from, each warp half hf packing
  // its 64 queries into its first 32 columns, handed over in two chunks.
  static constexpr uint32_t S_COL = 0, DP_COL = 128, DV_COL = 256, DK_COL = 256 + D, TMEM_COLS = 512;
  static constexpr int W = 64;                                  // columns per compute warp
  __host__ __device__ static constexpr uint32_t packed_col(int q) { return (uint32_t)((q / W) * W + (q % W) / 2); }
  __host__ __device__ static constexpr int chunk_of(int q) { return (q % W) / (W / 2); }
};

// A key tile and the query tiles that see it, cut into `nsplit` runs of `per`
// (the last ones may be empty).
struct KeyTile {
  PackedSeq q;
  int kt0, keys;     // first key inside the sequence, keys in the tile
  int off;           // causal: query token t sees key k when k <= t + off
  int i0, cnt, per;
};
__device__ __forceinline__ bool key_tile(const PackedGeom& g, int slot, int nsplit, KeyTile& k) {
  if (!packed_find(g, g.k_ptr, 128, slot, k.q)) return false;
  k.kt0 = (slot - (k.q.k0 / 128 + k.q.s)) * 128;
  if (k.kt0 >= k.q.lk) return false;
  k.keys = min(128, k.q.lk - k.kt0);
  k.off = k.q.lk - k.q.lq;
  const int qtiles = (k.q.lq + g.TQ - 1) / g.TQ;
  // the first query token that sees the tile's first key
  const long long t = g.causal ? min((long long)k.q.lq, max(0LL, (long long)k.kt0 - k.off)) : 0;
  k.i0 = (int)t / g.TQ;
  k.cnt = max(0, qtiles - k.i0);
  k.per = max((k.cnt + nsplit - 1) / nsplit, nsplit > 1 ? kPackedMinPart : 1);
  return true;
}

template <int D>
__global__ void __launch_bounds__(kKVThreads, 1)
    packed_bwd_kv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmdO,
                         const __grid_constant__ PackedGeom g, const float* __restrict__ L2w,
                         const float* __restrict__ Dw, float scale, __nv_bfloat16* dK, long long dk_head,
                         long long dk_tok, __nv_bfloat16* dV, long long dv_head, long long dv_tok, int nsplit,
                         float* part, int wide, Ctl ctl) {
  using T = PKVTraits<D>;
  constexpr int NQ = T::NQ, ND = T::ND;
  constexpr int W = T::W;
  extern __shared__ __align__(1024) uint8_t smem_raw[];

  cudaTriggerProgrammaticLaunchCompletion();     // the q kernel may start as SMs become free
  // the CTA's key tile; every thread works it out (the same loads for all)
  int kvh, slot;
  packed_order(g, g.nslot_k, false, blockIdx.x / nsplit, kvh, slot);
  KeyTile kt;
  if (!key_tile(g, slot, nsplit, kt)) return;
  const PackedSeq& q = kt.q;
  const int kt0 = kt.kt0, keys = kt.keys, off = kt.off;
  const int piece = blockIdx.x % nsplit;
  const int i0 = kt.i0 + piece * kt.per;                      // first query tile of this CTA
  const int cnt = max(0, min(kt.per, kt.cnt - piece * kt.per));
  const int qslot0 = q.q0 / g.TQ + q.s + i0;

  // the tiles take all but ~800 bytes, so the base itself has to be aligned
  // (the array is declared so; a launch that broke it is reported)
  if ((smem_u32(smem_raw) & 1023u) != 0u) {
    if (threadIdx.x == 0) set_error(ctl, DSV_ERR_INTERNAL, blockIdx.x);
    return;
  }
  uint8_t* sK = smem_raw;
  uint8_t* sV = sK + T::TILE;
  uint8_t* sQ = sV + T::TILE;                     // [NQ]
  uint8_t* sdO = sQ + NQ * T::TILE;               // [ND]
  uint8_t* sVec = sdO + ND * T::TILE;             // [ND] -lse2 | D
  uint64_t* bars = reinterpret_cast<uint64_t*>(sVec + 2 * ND * T::VEC_BYTES);
  uint64_t* kt_full = bars;                       // the key tile, and V's
  uint64_t* vt_full = bars + 1;
  uint64_t* q_full = bars + 2;
  uint64_t* q_empty = q_full + NQ;                // dK of the slot's tile is done (also frees its vectors)
  uint64_t* d_full = q_empty + NQ;
  uint64_t* d_empty = d_full + ND;                // dV of the slot's tile is done
  uint64_t* v_full = d_empty + ND;
  uint64_t* s_full = v_full + ND;                 // S^T in TMEM
  uint64_t* dp_full = s_full + 1;                 // dP^T in TMEM
  uint64_t* p_full = dp_full + 1;                 // [2] P^T chunk written back (bf16)
  uint64_t* ds_full = p_full + 2;                 // [2] dS^T chunk written back (bf16)
  uint64_t* acc_done = ds_full + 2;
  uint64_t* q_tail = acc_done + 1;                // the sequence's last query tile, before its rows are cut
  uint64_t* d_tail = q_tail + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(d_tail + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned int kid = (unsigned int)KID_PACKED_KV << 8;
  const long long krow0 = (long long)q.k0 + kt0;

  if (cnt == 0) {
    if (nsplit > 1) return;                       // the join knows how many parts there are
    // no query sees these keys
    for (int i = threadIdx.x; i < keys * (D / 8); i += blockDim.x) {
      const int r = i / (D / 8), c = i % (D / 8);
      *reinterpret_cast<uint4*>(dK + kvh * dk_head + (krow0 + r) * dk_tok + c * 8) = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(dV + kvh * dv_head + (krow0 + r) * dv_tok + c * 8) = make_uint4(0, 0, 0, 0);
    }
    return;
  }

  const int box = g.group * g.TQ;                 // rows a query tile's copy brings
  if (threadIdx.x == 0) {
    mbar_init(kt_full, 1);
    mbar_init(vt_full, 1);
    for (int s = 0; s < NQ; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 1);
    }
    for (int s = 0; s < ND; ++s) {
      mbar_init(&d_full[s], 1);
      mbar_init(&d_empty[s], 1);
      mbar_init(&v_full[s], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    for (int c = 0; c < 2; ++c) {
      mbar_init(&p_full[c], kComputeThreads);
      mbar_init(&ds_full[c], kComputeThreads);
    }
    mbar_init(acc_done, 1);
    mbar_init(q_tail, 1);
    mbar_init(d_tail, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  // rows of the last tile, when the box reaches past the sequence's end
  const int last_rows = min(g.TQ, q.lq - (i0 + cnt - 1) * g.TQ) * g.group;
  const bool cut = last_rows < box;
  const uint32_t tx = (uint32_t)box * D * 2;
  auto load = [&](const CUtensorMap* map, uint8_t* dst, uint64_t* bar, int n) {
    if (lane == 0) {
      mbar_arrive_expect_tx(bar, tx);
      for (int c = 0; c < T::NCH; ++c)
        tma_load_3d(dst + c * T::CHUNK, map, bar, c * 64, kvh * g.group, q.q0 + (i0 + n) * g.TQ);
    }
  };
  auto load_q = [&](int n) {
    load(&tmQ, sQ + (n % NQ) * T::TILE, cut && n == cnt - 1 ? q_tail : &q_full[n % NQ], n);
  };
  auto load_do = [&](int n) {
    load(&tmdO, sdO + (n % ND) * T::TILE, cut && n == cnt - 1 ? d_tail : &d_full[n % ND], n);
  };
  auto load_vec = [&](int n) {
    if (lane == 0) {
      const long long vec = ((long long)kvh * g.nslot_q + qslot0 + n) * 128;
      uint8_t* dst = sVec + (n % ND) * 2 * T::VEC_BYTES;
      mbar_arrive_expect_tx(&v_full[n % ND], 2 * T::VEC_BYTES);
      bulk_load(dst, L2w + vec, T::VEC_BYTES, &v_full[n % ND]);
      bulk_load(dst + T::VEC_BYTES, Dw + vec, T::VEC_BYTES, &v_full[n % ND]);
    }
  };
  int nd = min(cnt, ND), nq = min(cnt, NQ);        // tiles whose dO and vectors, Q are under way
  if (warp == 0) {
    // the first copies, before the tensor memory is there: K and Q first, which S^T(0) needs
    __syncwarp();
    if (lane == 0) {
      mbar_arrive_expect_tx(kt_full, T::TILE);
      for (int c = 0; c < T::NCH; ++c) tma_load_3d(sK + c * T::CHUNK, &tmK, kt_full, c * 64, kvh, (int)krow0);
    }
    load_q(0);
    if (lane == 0) {
      mbar_arrive_expect_tx(vt_full, T::TILE);
      for (int c = 0; c < T::NCH; ++c) tma_load_3d(sV + c * T::CHUNK, &tmV, vt_full, c * 64, kvh, (int)krow0);
    }
    load_do(0);
    load_vec(0);
    for (int n = 1; n < nq; ++n) {
      load_q(n);
      if (n < nd) {
        load_do(n);
        load_vec(n);
      }
    }
  }
  // every copy warp 0 started must land before the CTA exits
  auto drain = [&]() {
    mbar_wait(kt_full, 0, nullptr, ctl, kid | W_DRAIN);
    mbar_wait(vt_full, 0, nullptr, ctl, kid | W_DRAIN);
    for (int n = max(0, nq - NQ); n < nq; ++n)
      if (!(cut && n == cnt - 1)) mbar_wait(&q_full[n % NQ], (uint32_t)(n / NQ) & 1u, nullptr, ctl, kid | W_DRAIN);
    for (int n = max(0, nd - ND); n < nd; ++n) {
      if (!(cut && n == cnt - 1)) mbar_wait(&d_full[n % ND], (uint32_t)(n / ND) & 1u, nullptr, ctl, kid | W_DRAIN);
      mbar_wait(&v_full[n % ND], (uint32_t)(n / ND) & 1u, nullptr, ctl, kid | W_DRAIN);
    }
  };
  // rows box..127 of every query tile are never loaded (sQ and sdO are adjacent)
  if (box < 128 && warp >= 2 && warp < 2 + NQ + ND) zero_tile_rows(sQ + (warp - 2) * T::TILE, T::NCH, box, lane);
  if (warp == 1) {
    tmem_alloc(tmem_slot, T::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // one CTA owns the SM's whole TMEM, so its addresses start at 0 (attn_fwd.cu)
  const uint32_t tmem_base = *tmem_slot;
  constexpr uint32_t tmem = 0;

  if (tmem_base != tmem) {
    if (threadIdx.x == 0) set_error(ctl, DSV_ERR_INTERNAL, blockIdx.x);
    if (warp == 0) {
      if (cut && nq == cnt) mbar_wait(q_tail, 0, nullptr, ctl, kid | W_DRAIN);
      if (cut && nd == cnt) mbar_wait(d_tail, 0, nullptr, ctl, kid | W_DRAIN);
      drain();
    }
  } else if (warp == 0) {
    // ---------------- TMA producer: the tiles after the first ----------------
    for (int n = 0; n + ND < cnt; ++n) {
      if (!mbar_wait_warp(&d_empty[n % ND], (uint32_t)(n / ND) & 1u, abort_flag, ctl, kid | W_GEMPTY)) break;
      load_do(n + ND);
      ++nd;
      const bool freed = mbar_wait_warp(&q_empty[n % NQ], (uint32_t)(n / NQ) & 1u, abort_flag, ctl, kid | W_GEMPTY);
      load_vec(n + ND);                            // (loaded even on an abort: nd counts both)
      if (!freed) break;
      if (n + NQ < cnt) {
        load_q(n + NQ);
        ++nq;
      }
    }
    if (cut && nq == cnt && nd == cnt) {
      if (mbar_wait_warp(q_tail, 0, nullptr, ctl, kid | W_TAIL)) {
        zero_tile_rows(sQ + ((cnt - 1) % NQ) * T::TILE, T::NCH, last_rows, lane);
        if (lane == 0) mbar_arrive(&q_full[(cnt - 1) % NQ]);
      } else {
        *abort_flag = 1;
      }
      if (mbar_wait_warp(d_tail, 0, nullptr, ctl, kid | W_TAIL)) {
        zero_tile_rows(sdO + ((cnt - 1) % ND) * T::TILE, T::NCH, last_rows, lane);
        if (lane == 0) mbar_arrive(&d_full[(cnt - 1) % ND]);
      } else {
        *abort_flag = 1;
      }
    } else if (cut) {                              // an abort: only the drain is left
      if (nq == cnt) mbar_wait(q_tail, 0, nullptr, ctl, kid | W_DRAIN);
      if (nd == cnt) mbar_wait(d_tail, 0, nullptr, ctl, kid | W_DRAIN);
    }
    drain();
  } else if (warp == 1) {
    // ---------------- MMA issuer (whole warp, one elected lane issues) ----------------
    // Order, as in attn_bwd.cu: S^T(0), dP^T(0), then per query tile n
    //   dV(n) [P^T(n) written], S^T(n+1), dK(n) [dS^T(n) written], dP^T(n+1),
    // so the tensor core runs the next tile's products while the compute warps
    // convert; each barrier is tested half-way through the products before it.
    constexpr uint32_t ID_S = idesc_bf16_f32(128, 128, false, false);
    constexpr uint32_t ID_G = idesc_bf16_f32(128, D, false, true);
    const uint64_t dK0 = sdesc_sw128(smem_u32(sK), 16, 1024);
    const uint64_t dV0 = sdesc_sw128(smem_u32(sV), 16, 1024);
    const uint64_t dQ0 = sdesc_sw128(smem_u32(sQ), 16, 1024);               // K-major views
    const uint64_t ddO0 = sdesc_sw128(smem_u32(sdO), 16, 1024);
    const uint64_t dQmn0 = sdesc_sw128(smem_u32(sQ), T::CHUNK, 1024);       // MN-major views
    const uint64_t ddOmn0 = sdesc_sw128(smem_u32(sdO), T::CHUNK, 1024);
    // S^T = K Q^T (t = 0) or dP^T = V dO^T (t = 1); returns the test of `probe`
    auto issue_sdp = [&](int n, int t, uint64_t* probe, uint32_t probe_par) -> uint32_t {
      const uint64_t a0 = t ? dV0 : dK0;
      const uint64_t b0 = t ? desc_off(ddO0, (uint32_t)(n % ND) * T::TILE) : desc_off(dQ0, (uint32_t)(n % NQ) * T::TILE);
      uint32_t r = 0u;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t o = (kk >> 2) * T::CHUNK + (kk & 3) * 32;
        mma_ss_w(tmem + (t ? T::DP_COL : T::S_COL), desc_off(a0, o), desc_off(b0, o), ID_S, kk > 0 ? 1u : 0u);
        if (kk == D / 32 - 1 && probe != nullptr) r = mbar_test(probe, probe_par);
      }
      mma_commit_w(t ? dp_full : s_full);
      return r;
    };
    // chunk c of dV += P^T dO (t = 0) or dK += dS^T Q (t = 1); returns the test of `probe`
    auto issue_grad = [&](int n, int t, int c, uint64_t* probe, uint32_t probe_par) -> uint32_t {
      const uint64_t b0 = t ? desc_off(dQmn0, (uint32_t)(n % NQ) * T::TILE) : desc_off(ddOmn0, (uint32_t)(n % ND) * T::TILE);
      uint32_t r = 0u;
      int m = 0;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        if (T::chunk_of(kk * 16) != c) continue;
        mma_ts_w(tmem + (t ? T::DK_COL : T::DV_COL), tmem + (t ? T::DP_COL : T::S_COL) + T::packed_col(kk * 16),
                 desc_off(b0, kk * 16 * 128), ID_G, (n > 0 || kk > 0) ? 1u : 0u);
        if (++m == 2 && probe != nullptr) r = mbar_test(probe, probe_par);
      }
      return r;
    };
    bool ok = mbar_wait_warp(kt_full, 0, abort_flag, ctl, kid | W_KV) &&
              mbar_wait_warp(&q_full[0], 0, abort_flag, ctl, kid | W_GFULL);
    uint32_t tp0 = 0u;
    if (ok) {
      tc_fence_after();
      issue_sdp(0, 0, nullptr, 0u);
      ok = mbar_wait_warp(vt_full, 0, abort_flag, ctl, kid | W_KV) &&
           mbar_wait_warp(&d_full[0], 0, abort_flag, ctl, kid | W_GFULL);
      if (ok) {
        tc_fence_after();
        tp0 = issue_sdp(0, 1, &p_full[0], 0u);
      }
    }
    for (int n = 0; ok && n < cnt; ++n) {
      const bool more = n + 1 < cnt;
      const uint32_t par = (uint32_t)n & 1u;
      const uint32_t tq = more ? mbar_test(&q_full[(n + 1) % NQ], (uint32_t)((n + 1) / NQ) & 1u) : 0u;
      if (!mbar_wait_warp_tested(&p_full[0], par, tp0, abort_flag, ctl, kid | W_P)) break;
      tc_fence_after();
      const uint32_t tp1 = issue_grad(n, 0, 0, &p_full[1], par);
      if (!mbar_wait_warp_tested(&p_full[1], par, tp1, abort_flag, ctl, kid | W_P)) break;
      tc_fence_after();
      issue_grad(n, 0, 1, nullptr, 0u);
      mma_commit_w(&d_empty[n % ND]);
      uint32_t td0 = 0u;
      if (more) {
        if (!mbar_wait_warp_tested(&q_full[(n + 1) % NQ], (uint32_t)((n + 1) / NQ) & 1u, tq, abort_flag, ctl,
                                   kid | W_GFULL))
          break;
        tc_fence_after();
        td0 = issue_sdp(n + 1, 0, &ds_full[0], par);
      }
      const uint32_t tdo = more ? mbar_test(&d_full[(n + 1) % ND], (uint32_t)((n + 1) / ND) & 1u) : 0u;
      if (!mbar_wait_warp_tested(&ds_full[0], par, td0, abort_flag, ctl, kid | W_DSFULL)) break;
      tc_fence_after();
      const uint32_t td1 = issue_grad(n, 1, 0, &ds_full[1], par);
      if (!mbar_wait_warp_tested(&ds_full[1], par, td1, abort_flag, ctl, kid | W_DSFULL)) break;
      tc_fence_after();
      issue_grad(n, 1, 1, nullptr, 0u);
      mma_commit_w(&q_empty[n % NQ]);
      if (more) {
        if (!mbar_wait_warp_tested(&d_full[(n + 1) % ND], (uint32_t)((n + 1) / ND) & 1u, tdo, abort_flag, ctl,
                                   kid | W_GFULL))
          break;
        tc_fence_after();
        tp0 = issue_sdp(n + 1, 1, &p_full[0], par ^ 1u);
      }
    }
    mma_commit_w(acc_done);
    mbar_wait_warp(acc_done, 0, nullptr, ctl, kid | W_DRAIN);
  } else {
    // ------------- compute warps: key row kr, 64 rows of the query tile -------------
    const int sp = warp & 3;
    const int hf = (warp - 2) >> 2;
    const int kr = sp * 32 + lane;
    const uint32_t lane_off = (uint32_t)(sp * 32) << 16;
    const float scale_log2 = scale * kLog2e;
    const uint64_t c2 = f2_pack(scale_log2, scale_log2);
    const uint32_t cs = tmem + lane_off + T::S_COL + hf * W;
    const uint32_t cp = tmem + lane_off + T::DP_COL + hf * W;
    const int q0 = hf * W;                         // first tile row of this warp's columns
    bool ok = true;
    for (int n = 0; ok && n < cnt; ++n) {
      if (!mbar_wait_warp(&v_full[n % ND], (uint32_t)(n / ND) & 1u, abort_flag, ctl, kid | W_GFULL) ||
          !mbar_wait_warp(s_full, (uint32_t)n & 1u, abort_flag, ctl, kid | W_S)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const float4* l4 = reinterpret_cast<const float4*>(sVec + (n % ND) * 2 * T::VEC_BYTES) + q0 / 4;
      const float4* d4 = l4 + 32;
      // causal: tile row q sees this thread's key from q >= lo on (tokens in order, heads inside a token)
      const int first = (i0 + n) * g.TQ + off;     // last key that the tile's first token sees
      const bool mask = g.causal && first < kt0 + 127;
      const int lo = mask ? (kt0 + kr - first) * g.group - q0 : 0;
      uint32_t x[W];
      uint64_t p2[W / 2];                          // P^T of this row's 64 queries, fp32 pairs
      tmem_ld_w<W>(cs, x);
      tmem_ld_wait();
      if (mask) {
#pragma unroll
        for (int i = 0; i < W; ++i) x[i] = i >= lo ? x[i] : 0xff800000u;   // -inf: P = 0
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t pw[W / 4];
#pragma unroll
        for (int qq = c * (W / 8); qq < (c + 1) * (W / 8); ++qq) {
          const float4 L = l4[qq];                 // -lse*log2(e) of four queries
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j0 = 4 * qq + 2 * e;
            float x0, x1;
            f2_unpack(fma2(f2_pack(__uint_as_float(x[j0]), __uint_as_float(x[j0 + 1])), c2,
                           e ? f2_pack(L.z, L.w) : f2_pack(L.x, L.y)), x0, x1);
            const float a = ex2(x0), b = ex2(x1);
            p2[2 * qq + e] = f2_pack(a, b);
            pw[2 * qq + e - c * (W / 4)] = pack_bf16x2(a, b);
          }
        }
        // each warp overwrites only the TMEM lanes and columns it has read
        tmem_st_w<W / 4>(cs + c * (W / 4), pw);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&p_full[c]);
      }
      if (!mbar_wait_warp(dp_full, (uint32_t)n & 1u, abort_flag, ctl, kid | W_S)) {
        ok = false;
        break;
      }
      tc_fence_after();
      tmem_ld_w<W>(cp, x);
      tmem_ld_wait();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t dw[W / 4];
#pragma unroll
        for (int qq = c * (W / 8); qq < (c + 1) * (W / 8); ++qq) {
          const float4 Dd = d4[qq];                // D of four queries
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j0 = 4 * qq + 2 * e;
            const uint64_t t = sub2(f2_pack(__uint_as_float(x[j0]), __uint_as_float(x[j0 + 1])),
                                    e ? f2_pack(Dd.z, Dd.w) : f2_pack(Dd.x, Dd.y));
            float d0, d1;
            f2_unpack(mul2(p2[2 * qq + e], t), d0, d1);
            dw[2 * qq + e - c * (W / 4)] = pack_bf16x2(d0, d1);
          }
        }
        tmem_st_w<W / 4>(cp + c * (W / 4), dw);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&ds_full[c]);
      }
    }
    if (ok) ok = mbar_wait_warp(acc_done, 0, abort_flag, ctl, kid | W_ACC);
    if (ok) {
      tc_fence_after();
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint32_t col = (t == 0 ? T::DV_COL : T::DK_COL) + hf * (D / 2);
        const float mul = t == 0 ? 1.0f : scale;
        __nv_bfloat16* outp = (t == 0 ? dV + kvh * dv_head + (krow0 + kr) * dv_tok
                                      : dK + kvh * dk_head + (krow0 + kr) * dk_tok) + hf * (D / 2);
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint32_t o[32];
          tmem_ld32(tmem + lane_off + col + c * 32, o);
          tmem_ld_wait();
          if (nsplit > 1) {
            float* dst = part + (((long long)blockIdx.x * 2 + t) * 128 + kr) * D + hf * (D / 2) + c * 32;
#pragma unroll
            for (int p = 0; p < 4; ++p) st_global_32(dst + p * 8, o + p * 8);
          } else if (kr < keys) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
              w[i] = pack_bf16x2(__uint_as_float(o[2 * i]) * mul, __uint_as_float(o[2 * i + 1]) * mul);
            store_row32(outp + c * 32, w, wide);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, T::TMEM_COLS);
}

// Adds the parts of dV and dK (fp32, unscaled) in order.  CTAs per (key tile,
// key head; matrix; sixteenth of the rows), D/4 threads a row.
template <int D>
__global__ void __launch_bounds__(256) packed_bwd_join_kernel(const __grid_constant__ PackedGeom g, int nsplit,
                                                              const float* __restrict__ part, float scale,
                                                              __nv_bfloat16* dK, long long dk_head, long long dk_tok,
                                                              __nv_bfloat16* dV, long long dv_head, long long dv_tok) {
  int kvh, slot;
  packed_order(g, g.nslot_k, false, blockIdx.x, kvh, slot);
  KeyTile kt;
  if (!key_tile(g, slot, nsplit, kt)) return;
  const int parts = (kt.cnt + kt.per - 1) / kt.per, t = blockIdx.y;
  const float mul = t == 0 ? 1.0f : scale;
  __nv_bfloat16* out = t == 0 ? dV + kvh * dv_head : dK + kvh * dk_head;
  const long long tok = t == 0 ? dv_tok : dk_tok;
  const int c = threadIdx.x % (D / 4);
  for (int r = blockIdx.z * 8 + threadIdx.x / (D / 4); r < min(kt.keys, (int)blockIdx.z * 8 + 8); r += 256 / (D / 4)) {
    const float4* src = reinterpret_cast<const float4*>(part) +
                        (((long long)blockIdx.x * nsplit * 2 + t) * 128 + r) * (D / 4) + c;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int p = 0; p < parts; ++p) {
      const float4 v = __ldcs(src + (long long)p * 2 * 128 * (D / 4));
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    *reinterpret_cast<uint2*>(out + ((long long)kt.q.k0 + kt.kt0 + r) * tok + c * 4) =
        make_uint2(pack_bf16x2(s.x * mul, s.y * mul), pack_bf16x2(s.z * mul, s.w * mul));
  }
}

// ---------------------------------------------------------------------------
// dQ: one CTA per SM over the query tiles
// ---------------------------------------------------------------------------
struct QItem {
  int valid;
  int kvh;
  int tok;      // first query token of the tile (absolute)
  int ntok;
  int key0;     // first key (absolute)
  int nt;       // key tiles
  int lim0;     // keys that the first token sees (may be <= 0)
  int left;     // keys of the sequence
  int slot;     // query slot: rows of D and -lse2
  int pad;
};

template <int D>
struct PQTraits {
  static constexpr int NCH = D / 64;
  static constexpr int CHUNK = 128 * 128;
  static constexpr int TILE = NCH * CHUNK;
  // K_j is read by S (early) and by dQ (late); V_j only by dP: separate rings.
  // Q and dO twice where there is room.  (At d = 128 the room would have to
  // come from the rings: two K, one V and Q, dO twice took 161 us instead of
  // 149 even where an item has two to four key tiles, the text case.)
  static constexpr int NQD = D == 64 ? 2 : 1, NK = 3, NV = D == 64 ? 3 : 2;
  static constexpr int BARS = 3 * NQD + 2 * NK + 2 * NV + 7 + 4 + 2;
  static constexpr int NBAR = (BARS + 1) / 2 * 2;   // even: the answer after it is 16-byte aligned
  static constexpr int SMEM_USED = (2 * NQD + NK + NV) * TILE + NBAR * 8 + 16 + 16 + 2 * (int)sizeof(QItem) +
                                   1024 * NQD;
  static_assert(SMEM_USED <= 227 * 1024, "dQ tiles exceed shared memory");
  static constexpr int SMEM = SMEM_USED > 120 * 1024 ? SMEM_USED : 120 * 1024;
  static constexpr uint32_t S_COL = 0, DP_COL = 128, DQ_COL = 256, DS_COL = 256 + D, TMEM_COLS = 512;
  static constexpr uint32_t TX = 128 * D * 2;
  static constexpr int HALF = 64;
  static constexpr int CONSUMERS = 11;            // warps 0..10 read each item
};

template <int D>
__global__ void __launch_bounds__(kQThreads, 1)
    packed_bwd_q_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmdO,
                        const __grid_constant__ PackedGeom g, const float* __restrict__ L2w,
                        const float* __restrict__ Dw, float scale, __nv_bfloat16* dQ, long long dq_head,
                        long long dq_tok, int wide, Ctl ctl) {
  using T = PQTraits<D>;
  constexpr int NK = T::NK, NV = T::NV, NQD = T::NQD;
  constexpr int HALF = T::HALF;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // the tiles take all but ~800 bytes, so the base itself has to be aligned
  // (the array is declared so; a launch that broke it is reported)
  if ((smem_u32(smem_raw) & 1023u) != 0u) {
    if (threadIdx.x == 0) set_error(ctl, DSV_ERR_INTERNAL, blockIdx.x);
    cudaGridDependencySynchronize();
    return;
  }
  uint8_t* sdO = smem_raw;                        // [NQD]
  uint8_t* sQ = sdO + NQD * T::TILE;              // [NQD]
  uint8_t* sK = sQ + NQD * T::TILE;
  uint8_t* sV = sK + NK * T::TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sV + NV * T::TILE);
  uint64_t* qd_full = bars;                       // [NQD] Q, dO and the rows' vectors landed in smem
  uint64_t* qd_free = qd_full + NQD;              // [NQD] the item's last dP product is done
  uint64_t* vec_free = qd_free + NQD;             // [NQD] the compute warps have read the rows' vectors
  uint64_t* k_full = vec_free + NQD;
  uint64_t* k_empty = k_full + NK;
  uint64_t* v_full = k_empty + NK;
  uint64_t* v_empty = v_full + NV;
  uint64_t* s_full = v_empty + NV;
  uint64_t* sp_free = s_full + 1;                 // compute threads have read S, dP
  uint64_t* ds_full = sp_free + 1;
  uint64_t* ds_empty = ds_full + 1;
  uint64_t* acc_done = ds_empty + 1;              // dQ of the current tile is complete
  uint64_t* mma_drain = acc_done + 1;
  uint64_t* k_tail = mma_drain + 1;                // the last K tile of a sequence, before its rows are cut
  uint64_t* item_full = k_tail + 1;               // [2]
  uint64_t* item_free = item_full + 2;            // [2]
  uint64_t* near_end = item_free + 2;             // the K producer is about to finish its item
  uint64_t* clc_full = near_end + 1;              // the work request's answer is there
  void* clc = bars + T::NBAR;                     // 16 bytes
  float* sVec = reinterpret_cast<float*>(bars + T::NBAR + 2);   // [NQD] -lse2 of the tile's rows, then D
  QItem* items = reinterpret_cast<QItem*>(sVec + 256 * NQD);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(items + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned int kid = (unsigned int)KID_PACKED_Q << 8;
  const uint32_t q_bytes = (uint32_t)(g.group * g.TQ) * D * 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NQD; ++s) {
      mbar_init(&qd_full[s], 1);
      mbar_init(&qd_free[s], 1);
      mbar_init(&vec_free[s], 8);
    }
    for (int s = 0; s < NK; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < NV; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(sp_free, kComputeThreads);
    mbar_init(ds_full, kComputeThreads);
    mbar_init(ds_empty, 1);
    mbar_init(acc_done, 1);
    mbar_init(mma_drain, 1);
    mbar_init(k_tail, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&item_full[s], 1);
      mbar_init(&item_free[s], T::CONSUMERS);
    }
    mbar_init(near_end, 1);
    mbar_init(clc_full, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, T::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // one CTA owns the SM's whole TMEM, so its addresses start at 0 (attn_fwd.cu)
  const uint32_t tmem_base = *tmem_slot;
  constexpr uint32_t tmem = 0;

  // the next item of the ring, copied to registers; false at the end or on an abort
  auto take = [&](uint32_t i, QItem& it) -> bool {
    if (!mbar_wait_warp(&item_full[i & 1], (i >> 1) & 1u, abort_flag, ctl, kid | W_ITEM)) return false;
    it = items[i & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_free[i & 1]);
    return it.valid != 0;
  };

  if (tmem_base != tmem) {
    if (threadIdx.x == 0) set_error(ctl, DSV_ERR_INTERNAL, blockIdx.x);
  } else if (warp == kQItemWarp) {
    // ---------------- work items (as in packed_fwd.cu) ----------------
    int idx = blockIdx.x;
    for (uint32_t i = 0, asked = 0;; ++asked) {
      QItem it = {};
      int slot;
      packed_order(g, g.nslot_q, true, idx, it.kvh, slot);
      PackedSeq q;
      if (packed_find(g, g.q_ptr, g.TQ, slot, q)) {
        const int t0 = (slot - (q.q0 / g.TQ + q.s)) * g.TQ;
        if (t0 < q.lq) {
          it.valid = 1;
          it.tok = q.q0 + t0;
          it.ntok = min(g.TQ, q.lq - t0);
          const int last = g.causal ? min(q.lk, q.lk - q.lq + t0 + it.ntok) : q.lk;
          it.nt = last > 0 ? (last + 127) / 128 : 0;
          it.key0 = q.k0;
          it.left = q.lk;
          it.lim0 = g.causal ? min(q.lk, q.lk - q.lq + t0 + 1) : q.lk;
          it.slot = slot;
        }
      }
      if (it.valid && it.nt == 0) {
        // no key for any of its rows: written here, so that an item in the ring always has tiles
        for (int r = lane; r < it.ntok * g.group; r += 32) {
          const int rt = r / g.group, head = it.kvh * g.group + (r - rt * g.group);
          uint4* dst = reinterpret_cast<uint4*>(dQ + head * dq_head + ((long long)it.tok + rt) * dq_tok);
          for (int q = 0; q < D / 8; ++q) dst[q] = make_uint4(0, 0, 0, 0);
        }
      } else if (it.valid) {
        if (!mbar_wait_warp(&item_free[i & 1], ((i >> 1) & 1u) ^ 1u, abort_flag, ctl, kid | W_ITEMFREE)) break;
        if (lane == 0) {
          items[i & 1] = it;
          mbar_arrive(&item_full[i & 1]);
        }
        if (!mbar_wait_warp(near_end, i & 1u, abort_flag, ctl, kid | W_ITEM)) break;
        ++i;
      }
      if (lane == 0) clc_request(clc, clc_full);
      if (!mbar_wait_warp(clc_full, asked & 1u, nullptr, ctl, kid | W_ITEM)) {
        *abort_flag = 1;
        break;
      }
      idx = clc_answer(clc);
      fence_proxy_async_smem();        // read before the next answer is written
      __syncwarp();
      if (idx < 0) {
        if (mbar_wait_warp(&item_free[i & 1], ((i >> 1) & 1u) ^ 1u, abort_flag, ctl, kid | W_ITEMFREE) && lane == 0) {
          items[i & 1].valid = 0;
          mbar_arrive(&item_full[i & 1]);
        }
        break;
      }
    }
  } else if (warp == kQVWarp) {
    // ---------------- the V ring ----------------
    if (lane == 0) tma_prefetch_desc(&tmV);
    uint32_t gq = 0;
    bool ok = true;
    QItem it;
    for (uint32_t i = 0; ok && take(i, it); ++i) {
      for (int n = 0; n < it.nt; ++n) {
        const int s = (int)(gq % NV);
        if (!mbar_wait_warp(&v_empty[s], ((gq / NV) & 1u) ^ 1u, abort_flag, ctl, kid | W_KVEMPTY)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(&v_full[s], T::TX);
          for (int c = 0; c < T::NCH; ++c)
            tma_load_3d(sV + s * T::TILE + c * T::CHUNK, &tmV, &v_full[s], c * 64, it.kvh, it.key0 + n * 128);
        }
        ++gq;
      }
    }
    for (uint32_t n = (gq > NV ? gq - NV : 0u); n < gq; ++n)
      mbar_wait(&v_full[n % NV], (n / NV) & 1u, nullptr, ctl, kid | W_DRAIN);
  } else if (warp == 0) {
    // ---------------- Q, dO and the K ring ----------------
    if (lane == 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmdO);
      tma_prefetch_desc(&tmQ);
    }
    uint32_t gq = 0, tails = 0;
    uint32_t qd_issued = 0;
    bool ok = true;
    QItem it;
    for (uint32_t i = 0; ok && take(i, it); ++i) {
      for (int n = 0; n < it.nt; ++n) {
        // With one buffer for them the first K tile goes ahead of Q and dO, whose
        // place is free only when the item before is through with it.
        if (n == min(NQD == 1 ? 1 : 0, it.nt - 1)) {
          const int b = (int)(i % NQD);
          const uint32_t before = i / NQD - 1;     // the use of this buffer before this one
          if (i >= NQD && (!mbar_wait_warp(&qd_free[b], before & 1u, abort_flag, ctl, kid | W_KVEMPTY) ||
                           !mbar_wait_warp(&vec_free[b], before & 1u, abort_flag, ctl, kid | W_SPFREE))) {
            ok = false;
            break;
          }
          if (lane == 0) {
            const long long vec = ((long long)it.kvh * g.nslot_q + it.slot) * 128;
            mbar_arrive_expect_tx(&qd_full[b], 2 * q_bytes + 1024);
            for (int c = 0; c < T::NCH; ++c)
              tma_load_3d(sQ + b * T::TILE + c * T::CHUNK, &tmQ, &qd_full[b], c * 64, it.kvh * g.group, it.tok);
            for (int c = 0; c < T::NCH; ++c)
              tma_load_3d(sdO + b * T::TILE + c * T::CHUNK, &tmdO, &qd_full[b], c * 64, it.kvh * g.group, it.tok);
            bulk_load(sVec + b * 256, L2w + vec, 512, &qd_full[b]);
            bulk_load(sVec + b * 256 + 128, Dw + vec, 512, &qd_full[b]);
          }
          ++qd_issued;
        }
        const int s = (int)(gq % NK);
        if (!mbar_wait_warp(&k_empty[s], ((gq / NK) & 1u) ^ 1u, abort_flag, ctl, kid | W_KVEMPTY)) {
          ok = false;
          break;
        }
        const int have = it.left - n * 128;
        const bool tail = have < 128;
        uint64_t* bar = tail ? k_tail : &k_full[s];
        if (lane == 0) {
          mbar_arrive_expect_tx(bar, T::TX);
          for (int c = 0; c < T::NCH; ++c)
            tma_load_3d(sK + s * T::TILE + c * T::CHUNK, &tmK, bar, c * 64, it.kvh, it.key0 + n * 128);
          if (n == max(0, it.nt - kAskAhead)) mbar_arrive(near_end);
        }
        if (tail) {
          const bool landed = mbar_wait_warp(k_tail, tails & 1u, nullptr, ctl, kid | W_TAIL);
          ++tails;
          if (!landed) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          zero_tile_rows(sK + s * T::TILE, T::NCH, have, lane);
          if (lane == 0) mbar_arrive(&k_full[s]);
        }
        ++gq;
      }
    }
    // every copy this warp started must land before the CTA exits
    for (uint32_t n = (qd_issued > NQD ? qd_issued - NQD : 0u); n < qd_issued; ++n)
      mbar_wait(&qd_full[n % NQD], (n / NQD) & 1u, nullptr, ctl, kid | W_DRAIN);
    for (uint32_t n = (gq > NK ? gq - NK : 0u); n < gq; ++n)
      mbar_wait(&k_full[n % NK], (n / NK) & 1u, nullptr, ctl, kid | W_DRAIN);
  } else if (warp == 1) {
    // ---------------- MMA issuer (whole warp, one elected lane issues) ----------------
    constexpr uint32_t ID_S = idesc_bf16_f32(128, 128, false, false);
    constexpr uint32_t ID_Q = idesc_bf16_f32(128, D, false, true);
    const uint64_t ddO0 = sdesc_sw128(smem_u32(sdO), 16, 1024);
    const uint64_t dQ0 = sdesc_sw128(smem_u32(sQ), 16, 1024);
    const uint64_t dK0 = sdesc_sw128(smem_u32(sK), 16, 1024);
    const uint64_t dV0 = sdesc_sw128(smem_u32(sV), 16, 1024);
    const uint64_t dKmn0 = sdesc_sw128(smem_u32(sK), T::CHUNK, 1024);
    // S and dP run one tile ahead of dQ, their MMAs in turn (two chains of
    // accumulation: 967 -> 960 us on four clips of up to 8192 tokens).  Step
    // n = -1 issues an item's first ones, so that each product has one place in
    // the code: instructions that run once an item are fetched anew each time
    // and issue several times slower.
    uint32_t gq = 0;
    bool ok = true;
    QItem it;
    for (uint32_t i = 0; ok && take(i, it); ++i) {
      const uint32_t qb = i % NQD;
      if (!mbar_wait_warp(&qd_full[qb], (i / NQD) & 1u, abort_flag, ctl, kid | W_KV)) break;
      const uint64_t dq = desc_off(dQ0, qb * T::TILE), ddo = desc_off(ddO0, qb * T::TILE);
      int n = -1;
      for (; n < it.nt; ++n) {
        const uint32_t gn = gq + (uint32_t)n;
        uint32_t td = 0u;
        if (n + 1 < it.nt) {
          const int sk = (int)((gn + 1) % NK), sv = (int)((gn + 1) % NV);
          const uint32_t phk = ((gn + 1) / NK) & 1u, phv = ((gn + 1) / NV) & 1u;
          const uint32_t tk = mbar_test(&k_full[sk], phk);
          const uint32_t tv = mbar_test(&v_full[sv], phv);
          // S and dP are single-buffered: overwrite them once the compute warps hold
          // tile n (before the first tile gn is -1 and its parity passes at once)
          if (!mbar_wait_warp(sp_free, gn & 1u, abort_flag, ctl, kid | W_SPFREE) ||
              !mbar_wait_warp_tested(&k_full[sk], phk, tk, abort_flag, ctl, kid | W_KFULL) ||
              !mbar_wait_warp_tested(&v_full[sv], phv, tv, abort_flag, ctl, kid | W_VFULL)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t kb = desc_off(dK0, (uint32_t)sk * T::TILE), vb = desc_off(dV0, (uint32_t)sv * T::TILE);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t o = (kk >> 2) * T::CHUNK + (kk & 3) * 32;
            mma_ss_w(tmem + T::S_COL, desc_off(dq, o), desc_off(kb, o), ID_S, kk > 0 ? 1u : 0u);
            mma_ss_w(tmem + T::DP_COL, desc_off(ddo, o), desc_off(vb, o), ID_S, kk > 0 ? 1u : 0u);
          }
          td = mbar_test(ds_full, gn & 1u);
          mma_commit_w(s_full);
          mma_commit_w(&v_empty[sv]);                     // V_j is only needed by dP
          if (n + 2 == it.nt) mma_commit_w(&qd_free[qb]);      // the item's last read of Q and dO
        }
        if (n < 0) continue;
        // ds_full of an item's first tile also means that the previous item's dQ has been read
        if (!mbar_wait_warp_tested(ds_full, gn & 1u, td, abort_flag, ctl, kid | W_DSFULL)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int s = (int)(gn % NK);
        const uint64_t kmn = desc_off(dKmn0, (uint32_t)s * T::TILE);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts_w(tmem + T::DQ_COL, tmem + T::DS_COL + kk * 8, desc_off(kmn, kk * 16 * 128), ID_Q,
                   (n > 0 || kk > 0) ? 1u : 0u);
        mma_commit_w(&k_empty[s]);
        mma_commit_w(ds_empty);
      }
      if (!ok) break;
      mma_commit_w(acc_done);
      gq += (uint32_t)it.nt;
    }
    // TMEM is freed after the closing CTA-wide sync only once every MMA is done
    mma_commit_w(mma_drain);
    mbar_wait_warp(mma_drain, 0, nullptr, ctl, kid | W_DRAIN);
  } else {
    // ------------- compute warps: query row r, key half hf -------------
    const int sp = warp & 3;
    const int hf = (warp - 2) >> 2;
    const int r = sp * 32 + lane;
    const int rt = r / g.group, rh = r - rt * g.group;   // the row's token and head in the tile
    const uint32_t lane_off = (uint32_t)(sp * 32) << 16;
    const float scale_log2 = scale * kLog2e;
    bool ok = true;
    uint32_t gq = 0;
    int ne = 0;
    QItem it;
    for (uint32_t i = 0; ok && take(i, it); ++i) {
      const bool row_ok = rt < it.ntok;
      __nv_bfloat16* out = dQ + (long long)(it.kvh * g.group + rh) * dq_head + ((long long)it.tok + rt) * dq_tok +
                           hf * (D / 2);
      const uint32_t qb = i % NQD;
      if (!mbar_wait_warp(&qd_full[qb], (i / NQD) & 1u, abort_flag, ctl, kid | W_KV)) break;
      const float nlse2 = sVec[qb * 256 + r];      // -lse*log2(e); -inf for a row without keys
      const float dd = sVec[qb * 256 + 128 + r];
      __syncwarp();
      if (lane == 0) mbar_arrive(&vec_free[qb]);
      const int lim_r = g.causal ? min(it.left, it.lim0 + rt) : it.left;   // keys that the row sees

      uint32_t s_tested = 0u;
      for (int n = 0; n < it.nt; ++n) {
        const uint32_t gn = gq + (uint32_t)n;
        if (!mbar_wait_warp_tested(s_full, gn & 1u, s_tested, abort_flag, ctl, kid | W_S)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t xs[HALF], xp[HALF];
#pragma unroll
        for (int c = 0; c < HALF / 32; ++c) {
          tmem_ld32(tmem + lane_off + T::S_COL + hf * HALF + c * 32, xs + c * 32);
          tmem_ld32(tmem + lane_off + T::DP_COL + hf * HALF + c * 32, xp + c * 32);
        }
        tmem_ld_wait();
        tc_fence_before();
        mbar_arrive(sp_free);
        const uint32_t e_tested = mbar_test(ds_empty, (gn & 1u) ^ 1u);
        if (n * 128 + 128 > it.lim0) {
          // past the row's limit: P = 0 by s = -inf, and dP = 0 so that no NaN of it is left
          const int lim = lim_r - n * 128 - hf * HALF;
#pragma unroll
          for (int j = 0; j < HALF; ++j) {
            xs[j] = j < lim ? xs[j] : 0xff800000u;
            xp[j] = j < lim ? xp[j] : 0u;
          }
        }
        // exponent, dP - D and dS on packed fp32 pairs
        uint32_t dw[HALF / 2];
        const uint64_t c2 = f2_pack(scale_log2, scale_log2), nl2 = f2_pack(nlse2, nlse2), dd2 = f2_pack(dd, dd);
#pragma unroll
        for (int j = 0; j < HALF / 2; ++j) {
          float x0, x1, d0, d1;
          f2_unpack(fma2(f2_pack(__uint_as_float(xs[2 * j]), __uint_as_float(xs[2 * j + 1])), c2, nl2), x0, x1);
          const float p0 = ex2(x0), p1 = ex2(x1);
          const uint64_t t = sub2(f2_pack(__uint_as_float(xp[2 * j]), __uint_as_float(xp[2 * j + 1])), dd2);
          f2_unpack(mul2(f2_pack(p0, p1), t), d0, d1);
          dw[j] = pack_bf16x2(d0, d1);
        }
        // the single dS buffer is free once dQ of the previous tile is done
        if (n + 1 < it.nt) s_tested = mbar_test(s_full, (gn + 1) & 1u);
        if (!mbar_wait_warp_tested(ds_empty, (gn & 1u) ^ 1u, e_tested, abort_flag, ctl, kid | W_DSEMPTY)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < HALF / 32; ++c)
          tmem_st16(tmem + lane_off + T::DS_COL + hf * (HALF / 2) + c * 16, dw + c * 16);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(ds_full);
      }
      if (ok) ok = mbar_wait_warp(acc_done, (uint32_t)ne & 1u, abort_flag, ctl, kid | W_ACC);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t o[32];
        tmem_ld32(tmem + lane_off + T::DQ_COL + hf * (D / 2) + c * 32, o);
        tmem_ld_wait();
        if (row_ok) {
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 16; ++j)
            w[j] = pack_bf16x2(__uint_as_float(o[2 * j]) * scale, __uint_as_float(o[2 * j + 1]) * scale);
          store_row32(out + c * 32, w, wide);
        }
      }
      gq += (uint32_t)it.nt;
      ++ne;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, T::TMEM_COLS);
  // the call's work is done when this kernel is: not before the kv kernel's
  cudaGridDependencySynchronize();
}

template <int D>
cudaError_t launch_t(const PackedMaps& m, const PackedGeom& g, const dsv_view& O, const dsv_view& dO, const float* lse,
                     float scale, const dsv_view& dQ, const dsv_view& dK, const dsv_view& dV, void* ws,
                     int nsplit, const Ctl& ctl, cudaStream_t st) {
  cudaError_t e;
  const size_t vec = (size_t)g.Hkv * g.nslot_q * 128;
  float* Dw = static_cast<float*>(ws);
  float* L2w = Dw + vec;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = g.Tk > 0 && g.Tq > 0 ? 1 : 0;
  if (g.Tk > 0 && g.Tq > 0) {
    auto rows = packed_bwd_rows_kernel<D>;
    constexpr int smem = PRowsTraits<D>::SMEM;
    if ((e = cudaFuncSetAttribute(rows, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
    const long long slots = (long long)g.Hkv * g.nslot_q;
    rows<<<(unsigned)(slots < kPackedSMs ? slots : kPackedSMs), kRowsThreads, smem, st>>>(m.Q, m.K, m.V, m.dO, g, lse,
                                                                                          scale, Dw, ctl);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  // beside the rows kernel; it ends no earlier (its last lines).  Without
  // queries one CTA is left of it, for its check of the pointers.
  cfg.gridDim = g.Tq > 0 ? dim3((unsigned)g.nslot_q, (unsigned)g.Hkv) : dim3(1);
  cfg.blockDim = dim3(256);
  if ((e = cudaLaunchKernelEx(&cfg, packed_bwd_prep_kernel<D>, g, static_cast<const __nv_bfloat16*>(O.ptr),
                              (long long)O.head_stride, (long long)O.token_stride,
                              static_cast<const __nv_bfloat16*>(dO.ptr), (long long)dO.head_stride,
                              (long long)dO.token_stride, lse, Dw, L2w, ctl)) != cudaSuccess)
    return e;
  if (g.Tk > 0) {
    auto kv = packed_bwd_kv_kernel<D>;
    constexpr int smem = PKVTraits<D>::SMEM;
    if ((e = cudaFuncSetAttribute(kv, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
    const unsigned tiles = (unsigned)((long long)g.Hkv * g.nslot_k);
    float* part = L2w + vec;
    __nv_bfloat16* k_out = static_cast<__nv_bfloat16*>(dK.ptr);
    __nv_bfloat16* v_out = static_cast<__nv_bfloat16*>(dV.ptr);
    kv<<<tiles * nsplit, kKVThreads, smem, st>>>(m.Q, m.K, m.V, m.dO, g, L2w, Dw, scale, k_out, dK.head_stride,
                                                 dK.token_stride, v_out, dV.head_stride, dV.token_stride, nsplit,
                                                 part, wide_rows(dK) && wide_rows(dV), ctl);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (g.Tq == 0) return cudaSuccess;
  auto qk = packed_bwd_q_kernel<D>;
  constexpr int smem = PQTraits<D>::SMEM;
  if ((e = cudaFuncSetAttribute(qk, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
  // The q kernel needs what the prepare kernel wrote, not what the kv kernel
  // does: its CTAs start as the kv kernel's last ones leave SMs free, and it
  // ends no earlier than the kv kernel (packed_bwd_q_kernel's last lines).
  cfg.gridDim = dim3((unsigned)((long long)g.Hkv * g.nslot_q));
  cfg.blockDim = dim3(kQThreads);
  cfg.dynamicSmemBytes = smem;
  if ((e = cudaLaunchKernelEx(&cfg, qk, m.Q, m.K, m.V, m.dO, g, static_cast<const float*>(L2w),
                              static_cast<const float*>(Dw), scale, static_cast<__nv_bfloat16*>(dQ.ptr),
                              (long long)dQ.head_stride, (long long)dQ.token_stride, wide_rows(dQ), ctl)) !=
      cudaSuccess)
    return e;
  if (nsplit > 1) {
    packed_bwd_join_kernel<D><<<dim3((unsigned)((long long)g.Hkv * g.nslot_k), 2, 16), 256, 0, st>>>(
        g, nsplit, L2w + vec, scale, static_cast<__nv_bfloat16*>(dK.ptr), dK.head_stride, dK.token_stride,
        static_cast<__nv_bfloat16*>(dV.ptr), dV.head_stride, dV.token_stride);
    return cudaGetLastError();
  }
  return cudaGetLastError();
}

}  // namespace

// Runs of query tiles per key tile in the kv kernel.  With at least one key
// tile per SM each CTA takes all query tiles of its own.  With fewer they may be
// cut into `n` runs of at least kPackedMinPart tiles, whose fp32 sums the join
// kernel adds.  The q kernel's CTAs fill the SMs that the kv kernel leaves free,
// so what counts is when both are done: worked out below for n that fill half
// an SM's rounds, in microseconds at d = 128 (a pair of tiles 1.4 and 1.0, a
// CTA's start 5 and 4, the join 4 and 0.033 for each run's 131 KB), the lengths, which the host does not know,
// taken half-way between equal ones and a single long one.  It ranks the choices
// of n and no more: for the text call below it says 459 us whole and 476 in two,
// as it takes an item of dQ for 4.5 key tiles where those have two and four.
// The constants decide d = 64 as well, where they were not measured.  Measured with and
// without runs: 24 heads of two clips against 226 and 512 keys 344 / 315 us, 2
// heads of one clip of 4000 83 / 57 us, but one head of 20 000 against 300 keys
// 41 / 225 us, three heads over one of three clips up to 5095 72 / 156 us.
static int bwd_splits(const dsv_packed& p) {
  if (p.S <= 0 || p.Tq <= 0 || p.Tk <= 0) return 1;
  const long long TQ = 128 / (p.H / p.Hkv);
  const long long k_tiles = (p.Tk + 127) / 128, q_tiles = (p.Tq + TQ - 1) / TQ;
  const long long ctas = (long long)p.Hkv * (k_tiles > p.S ? k_tiles : p.S);
  if (ctas >= kPackedSMs) return 1;
  const long long items = (long long)p.Hkv * (q_tiles > p.S ? q_tiles : p.S);
  const double part = 0.5 * (1.0 + 1.0 / p.S);
  const double q = q_tiles * part < 1 ? 1 : q_tiles * part, k = k_tiles * part < 1 ? 1 : k_tiles * part;
  const double item_us = k * 1.0 + 4;
  const long long most = (long long)ceil(q / kPackedMinPart);
  double best = 0;
  long long splits = 1, last = 0;
  for (long long half = 0; half <= 8; ++half) {
    long long n = half == 0 ? 1 : half * kPackedSMs / 2 / ctas;
    if (n > most) n = most;
    if (n <= last) continue;
    last = n;
    const double run_us = ceil(q / n) * 1.4 + 5;
    const long long rounds = ctas * n / kPackedSMs, rest = ctas * n % kPackedSMs, open = kPackedSMs - rest;
    // items per SM that is free after the full rounds; the others come `late` items later
    const long long late = (long long)ceil(run_us / item_us);
    long long each = (items + open - 1) / open;
    if (each > late) each = (items + rest * late + kPackedSMs - 1) / kPackedSMs;
    const double kv_us = (rounds + (rest > 0)) * run_us, q_us = rounds * run_us + each * item_us;
    const double us = (kv_us > q_us ? kv_us : q_us) + (n > 1 ? 4 + 0.033 * (ctas * n) : 0);
    if (half == 0 || us < best) {
      best = us;
      splits = n;
    }
  }
  return (int)splits;
}

size_t packed_bwd_ws_bytes(const dsv_packed& p) {
  const size_t vec = 2 * (size_t)p.Hkv * packed_slots(p.Tq, 128 / (p.H / p.Hkv), p.S) * 128 * sizeof(float);
  const int n = bwd_splits(p);
  return n == 1 ? vec : vec + (size_t)p.Hkv * packed_slots(p.Tk, 128, p.S) * n * 2 * 128 * p.d * sizeof(float);
}

cudaError_t launch_packed_bwd(const PackedMaps& m, const dsv_packed& p, const int32_t* q_ptr, const int32_t* k_ptr,
                              int causal, float scale, const dsv_view& O, const dsv_view& dO, const float* lse,
                              const dsv_view& dQ, const dsv_view& dK, const dsv_view& dV, void* ws, const Ctl& ctl,
                              cudaStream_t st) {
  const PackedGeom g = packed_geom(p, q_ptr, k_ptr, causal);
  const int n = bwd_splits(p);
  return p.d == 128 ? launch_t<128>(m, g, O, dO, lse, scale, dQ, dK, dV, ws, n, ctl, st)
                    : launch_t<64>(m, g, O, dO, lse, scale, dQ, dK, dV, ws, n, ctl, st);
}

}  // namespace dsv
