// packed_fwd.cu — softmax attention of packed sequences, forward, on tcgen05.
//
//   s_ij = scale q_i . k_j over the keys j of i's own sequence (causal: also
//   j <= i + Lk - Lq, positions counted inside the sequence),
//   O_i = sum_j softmax(s_i)_j v_j,  lse_i = ln sum_j exp(s_ij);
//   a row that sees no key gets O = 0, lse = -inf.
//
// The dense companion of the block-sparse forward (attn_fwd.cu): the same
// pipeline of one 128-row query tile against a stream of 128-key tiles with S,
// P and O in tensor memory and an online softmax whose reference is the first
// tile's row maximum, redone only when a later value of P would pass 2^64 (or no
// score before was finite).
// What differs: tiles come from packed.cuh's slots (a tile's rows are tokens x
// shared heads), rows end at their own limit, and where there are fewer tiles
// than SMs each tile's keys are split over several CTAs.
//
// Key limit.  Row r (token t of the tile) sees keys [0, lim_r).  A tile of
// keys that every row sees whole takes the unmasked path; in the others a key
// at or past the row's limit is set to -inf by selection, so whatever the
// loaded row holds there (the next sequence's keys) never enters.  The last
// tile's V rows past the sequence's end are zeroed in shared memory: their P
// is 0, but 0 * NaN is not.
//
// Warp roles (three warpgroups): warp 0 loads Q and the K ring, warp 1 issues
// the MMAs, warp 2 loads the V ring, warp 3 takes the work items (one CTA of
// the grid each, taken over while they have not started) and hands them to the
// others through a two-entry ring, so that a search in the row pointers never
// stops the others; warps 4..7 softmax, warps 8..11 write O (one row per
// thread each).  The softmax of the next item starts while the last PV product
// and the output of this one are still under way: the writers copy O out of
// tensor memory and give it back (o_free) before they store it.
//
// Registers.  A softmax row holds 128 scores and their 64 packed P at once (a
// row whose sum overflows is redone), more than the 168 registers of 384 equal
// threads: the warpgroups split the CTA's registers 88 : 256 : 160.
//
// Measured, d = 128: 24 heads of 16 384 tokens 2050 us alone (1609 TFLOP/s, 86 % of
// what a large library product reaches in a burst), 2250 us back to back under
// the power cap; causal, 24 heads over 8 key heads, eight clips of 1 to 8191
// tokens, 422 us (1509 TFLOP/s of the tiles it multiplies); one new token of
// eight streams against up to 30 720 keys each, 62 us (6.2 TB/s), 68 a call with
// the join.  Long clips are bound by the softmax warps' chain beside the products,
// single tokens by HBM.
//
// Split over the keys.  Each part writes its normalised O (fp32) and base-2
// log-sum to the workspace and packed_combine_kernel joins them in an order of
// its own: results do not depend on which part finished first.  A tile with one
// part writes its result at once.
#include <math.h>

#include <type_traits>

#include "packed.cuh"

namespace dsv {

namespace {

constexpr float kLn2 = 0.69314718055994530942f;

struct FwdItem {
  int valid;
  int kvh;     // key head
  int tok;     // first query token of the tile (absolute)
  int ntok;    // tokens in the tile
  int key0;    // first key of this part (absolute)
  int nt;      // key tiles of this part
  int lim0;    // keys of this part that the first token sees (may be <= 0, may exceed the part)
  int left;    // keys of the sequence from key0 on
  int part;    // where a split item's part of O goes
  int parts;   // parts of its tile: one alone is the result
};

template <int D>
struct PFwdTraits {
  static constexpr int NCH = D / 64;
  static constexpr int CHUNK = 128 * 128;
  static constexpr int TILE = NCH * CHUNK;
  static constexpr int NST = 3;
  static constexpr int NBAR = 1 + 2 * NST + 3 * NST + 2 + 1 + 4 + 2 + 2 + 1;   // even: the answer after it is 16-byte aligned
  static constexpr int SMEM_USED = 1024 + TILE + 2 * NST * TILE + NBAR * 8 + 16 + 16 + 2 * (int)sizeof(FwdItem) + 1024;
  static_assert(NBAR % 2 == 0, "alignment of the work request's answer");
  static_assert(SMEM_USED <= 227 * 1024, "forward tiles exceed shared memory");
  // at least 120 KB so that one CTA owns an SM (and its 512 TMEM columns)
  static constexpr int SMEM = SMEM_USED > kTmemOwnerSmem ? SMEM_USED : kTmemOwnerSmem;
  static constexpr uint32_t S_COL = 128, O_COL = 384, TMEM_COLS = 512;
  static constexpr uint32_t TX = 128 * D * 2;
};

constexpr int kVWarp = 2, kItemWarp = 3, kFwdThreads = 384, kConsumers = 11;
// Key tiles before an item's last one at which the next item is asked for: an
// answer, the search and the loads take ~6000 clocks, a tile ~1600.
constexpr int kAskAhead = 6;
constexpr int kRegsControl = 88, kRegsSoftmax = 256, kRegsOut = 160, kRegsLaunch = 168;
static_assert(kRegsControl + kRegsSoftmax + kRegsOut <= 3 * kRegsLaunch, "warpgroup registers exceed the launch's");

enum : unsigned int { W_Q = 1, W_KEMPTY, W_K, W_P, W_V, W_S, W_O, W_OFINAL, W_DRAIN, W_QEMPTY, W_ITEM, W_ITEMFREE,
                      W_TAIL, W_OFREE, W_STAT };

template <int D>
__global__ void __launch_bounds__(kFwdThreads, 1)
    packed_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PackedGeom g, int part_keys,
                      int part_rows, int head_items, float scale_log2, __nv_bfloat16* O, long long o_head, long long o_tok,
                      float* LSE, float* Opart, float* Lpart, int wide, Ctl ctl) {
  using T = PFwdTraits<D>;
  constexpr int NST = T::NST;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sbase = smem_align1024(smem_raw);
  uint8_t* sQ = sbase;
  uint8_t* sK = sQ + T::TILE;
  uint8_t* sV = sK + NST * T::TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sV + NST * T::TILE);
  uint64_t* q_full = bars;
  uint64_t* k_full = bars + 1;
  uint64_t* v_full = k_full + NST;
  uint64_t* s_full = v_full + NST;    // [3] S(n) in buffer n%3; also frees K slot n%3
  uint64_t* p_full = s_full + NST;    // [3] P(n) written over S(n)
  uint64_t* o_done = p_full + NST;    // [3] O += P(n) V_n done; also frees V slot n%3
  uint64_t* o_final = o_done + NST;   // all PV products of the current item are done
  uint64_t* mma_drain = o_final + 1;
  uint64_t* v_tail = mma_drain + 1;   // the last V tile of a sequence, before its rows are cut
  uint64_t* item_full = v_tail + 1;   // [2]
  uint64_t* item_free = item_full + 2;  // [2]
  uint64_t* near_end = item_free + 2;   // the K producer is about to finish its item
  uint64_t* clc_full = near_end + 1;    // the work request's answer is there
  uint64_t* stat_full = clc_full + 1;   // l and m of the item's rows are in `stat`
  uint64_t* o_free = stat_full + 1;     // O and `stat` of the item have been read
  void* clc = bars + T::NBAR;           // 16 bytes
  float2* stat = reinterpret_cast<float2*>(bars + T::NBAR + 2);   // [128] 1 / l, base-2 log-sum
  FwdItem* items = reinterpret_cast<FwdItem*>(stat + 128);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(items + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned int kid = (unsigned int)KID_PACKED_FWD << 8;
  const uint32_t q_bytes = (uint32_t)(g.group * g.TQ) * D * 2;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < NST; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 128);
      mbar_init(&o_done[s], 1);
    }
    mbar_init(o_final, 1);
    mbar_init(mma_drain, 1);
    mbar_init(v_tail, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&item_full[s], 1);
      mbar_init(&item_free[s], kConsumers);
    }
    mbar_init(near_end, 1);
    mbar_init(clc_full, 1);
    mbar_init(stat_full, 128);
    mbar_init(o_free, 128);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, T::TMEM_COLS);
    tmem_relinquish();
  }
  cudaTriggerProgrammaticLaunchCompletion();     // the combine kernel may come to wait (packed_combine_kernel)
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // one CTA owns the SM's whole TMEM, so its addresses start at 0 (attn_fwd.cu)
  const uint32_t tmem_base = *tmem_slot;
  constexpr uint32_t tmem = 0;

  // the next item of the ring, copied to registers; false at the end or on an abort
  auto take = [&](uint32_t i, FwdItem& it) -> bool {
    if (!mbar_wait_warp(&item_full[i & 1], (i >> 1) & 1u, abort_flag, ctl, kid | W_ITEM)) return false;
    it = items[i & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_free[i & 1]);
    return it.valid != 0;
  };

  if (tmem_base != tmem) {
    if (threadIdx.x == 0) set_error(ctl, DSV_ERR_INTERNAL, blockIdx.x);
  } else if (warp < 4) {
    regs_dec<kRegsControl>();
    if (warp == kItemWarp) {
      // ---------------- work items ----------------
      // The grid has a CTA for every item; the ones that run take over those
      // that have not started, one at a time and only when the item in hand is
      // nearly loaded, so that none waits in a queue while another SM idles.
      int idx = blockIdx.x;
      for (uint32_t i = 0, asked = 0;; ++asked) {
        if (idx == 0) packed_check_ptrs(g, ctl, lane);
        FwdItem it = {};
        PackedSeq q;
        int tile = 0, k_from = 0, k_to = 0;      // the item's query tile, its keys inside the sequence
        bool found;
        if (part_keys == 0) {
          int slot;
          packed_order(g, g.nslot_q, true, idx, it.kvh, slot);
          found = packed_find(g, g.q_ptr, g.TQ, slot, q);
          if (found) {
            tile = slot - (q.q0 / g.TQ + q.s);
            k_to = q.lk;
          }
        } else {
          it.kvh = idx / head_items;
          const PackedPart part = packed_part(g, part_keys, idx - it.kvh * head_items, lane, q);
          found = part.part >= 0;
          tile = part.tile;
          k_from = part.part * part_keys;
          k_to = found ? min(q.lk, k_from + part_keys) : 0;
          it.part = idx;
          it.parts = part.parts;
          // (parts that do not fit take overlapping sequences: bad pointers)
          found = found && idx - it.kvh * head_items - part.part + part.parts <= head_items;
        }
        const int t0 = tile * g.TQ;
        if (found && t0 < q.lq) {
          it.valid = 1;
          it.tok = q.q0 + t0;
          it.ntok = min(g.TQ, q.lq - t0);
          // keys that the first and the last token of the tile see
          const int first = g.causal ? min(q.lk, q.lk - q.lq + t0 + 1) : q.lk;
          const int last = min(k_to, g.causal ? min(q.lk, q.lk - q.lq + t0 + it.ntok) : q.lk);
          it.nt = last > k_from ? (last - k_from + 127) / 128 : 0;
          it.key0 = q.k0 + k_from;
          it.left = q.lk - k_from;
          it.lim0 = first - k_from;
        }
        if (it.valid && it.nt == 0) {
          // no key for any of its rows: written here, so that an item in the ring always has tiles
          for (int r = lane; r < it.ntok * g.group; r += 32) {
            if (it.parts > 1) {
              Lpart[(long long)it.part * part_rows + r] = -INFINITY;
              continue;
            }
            const int rt = r / g.group, head = it.kvh * g.group + (r - rt * g.group);
            const long long tok = (long long)it.tok + rt;
            uint4* dst = reinterpret_cast<uint4*>(O + head * o_head + tok * o_tok);
            for (int q = 0; q < D / 8; ++q) dst[q] = make_uint4(0, 0, 0, 0);
            LSE[(long long)head * g.Tq + tok] = -INFINITY;
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
    } else if (warp == 0) {
      // ---------------- Q and the K ring ----------------
      if (lane == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
      }
      uint32_t gq = 0;                            // tiles issued so far
      int q_issued = 0;
      bool ok = true;
      FwdItem it;
      for (uint32_t i = 0; ok && take(i, it); ++i) {
        // the first two K tiles go ahead of Q, whose buffer is free only when
        // the previous item's last S product is done
        for (int n = 0; n < it.nt; ++n) {
          if (n == min(2, it.nt - 1)) {
            const uint32_t last = gq - (uint32_t)n - 1;        // the previous item's last tile
            if (q_issued > 0 && !mbar_wait_warp(&s_full[last % NST], (last / NST) & 1u, abort_flag, ctl, kid | W_QEMPTY)) {
              ok = false;
              break;
            }
            if (lane == 0) {
              mbar_arrive_expect_tx(q_full, q_bytes);
              for (int c = 0; c < T::NCH; ++c)
                tma_load_3d(sQ + c * T::CHUNK, &tmQ, q_full, c * 64, it.kvh * g.group, it.tok);
            }
            ++q_issued;
          }
          const int s = (int)(gq % NST);
          if (gq >= NST && !mbar_wait_warp(&s_full[s], ((gq - NST) / NST) & 1u, abort_flag, ctl, kid | W_KEMPTY)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            mbar_arrive_expect_tx(&k_full[s], T::TX);
            for (int c = 0; c < T::NCH; ++c)
              tma_load_3d(sK + s * T::TILE + c * T::CHUNK, &tmK, &k_full[s], c * 64, it.kvh, it.key0 + n * 128);
            if (n == max(0, it.nt - kAskAhead)) mbar_arrive(near_end);
          }
          ++gq;
        }
      }
      // every copy this warp started must land before the CTA exits
      if (q_issued > 0) mbar_wait(q_full, (uint32_t)(q_issued - 1) & 1u, nullptr, ctl, kid | W_DRAIN);
      for (uint32_t n = (gq > NST ? gq - NST : 0u); n < gq; ++n)
        mbar_wait(&k_full[n % NST], (n / NST) & 1u, nullptr, ctl, kid | W_DRAIN);
    } else if (warp == kVWarp) {
      // ---------------- the V ring ----------------
      if (lane == 0) tma_prefetch_desc(&tmV);
      uint32_t gq = 0, tails = 0;
      bool ok = true;
      FwdItem it;
      for (uint32_t i = 0; ok && take(i, it); ++i) {
        for (int n = 0; n < it.nt; ++n) {
          const int s = (int)(gq % NST);
          if (gq >= NST && !mbar_wait_warp(&o_done[s], ((gq - NST) / NST) & 1u, abort_flag, ctl, kid | W_KEMPTY)) {
            ok = false;
            break;
          }
          const int have = it.left - n * 128;
          const bool tail = have < 128;
          uint64_t* bar = tail ? v_tail : &v_full[s];
          if (lane == 0) {
            mbar_arrive_expect_tx(bar, T::TX);
            for (int c = 0; c < T::NCH; ++c)
              tma_load_3d(sV + s * T::TILE + c * T::CHUNK, &tmV, bar, c * 64, it.kvh, it.key0 + n * 128);
          }
          if (tail) {
            // rows past the sequence's end belong to the next one (or to nobody)
            const bool landed = mbar_wait_warp(v_tail, tails & 1u, nullptr, ctl, kid | W_TAIL);
            ++tails;
            if (!landed) {
              *abort_flag = 1;
              ok = false;
              break;
            }
            zero_tile_rows(sV + s * T::TILE, T::NCH, have, lane);
            if (lane == 0) mbar_arrive(&v_full[s]);
          }
          ++gq;
        }
      }
      for (uint32_t n = (gq > NST ? gq - NST : 0u); n < gq; ++n)
        mbar_wait(&v_full[n % NST], (n / NST) & 1u, nullptr, ctl, kid | W_DRAIN);
    } else if (warp == 1) {
      // ---------------- MMA issuer (whole warp, one elected lane issues) ----------------
      constexpr uint32_t IDS = idesc_bf16_f32(128, 128, false, false);
      constexpr uint32_t IDO = idesc_bf16_f32(128, D, false, true);
      const uint64_t dQ0 = sdesc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t dK0 = sdesc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t dV0 = sdesc_sw128(smem_u32(sV), T::CHUNK, 1024);
      // S runs up to three tiles ahead of PV, over item ends too: the next
      // item's first scores are issued as soon as its Q is there, so that the
      // softmax finds them when it is done with this item.  S(t+3) follows
      // PV(t) without a wait between them (its K was tested before P(t) was
      // waited for): the MMA queue holds only a few products and drains in any
      // gap.  Each product has one place in the code: instructions that run
      // once an item are fetched anew each time, and 8 MMAs then took ~3000
      // clocks to issue.
      uint32_t sg = 0, pg = 0;                   // tiles issued: S, PV
      uint32_t i = 0, k_tested = 0;              // items taken; K of tile sg known to be there
      int s_left = 0, pv_n = 0, ne = 0;          // S tiles left of item i - 1; PV tiles done of the current item, items done
      int nt0 = 0, nt1 = 0, nt2 = 0;             // tiles of the items between PV's and S's, PV's first
      bool ok = true, more = true, q_wait = false;
      auto tested = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_test(bar, parity) != 0u); };
      // the next item and its Q; without `block` only if they are there
      auto acquire = [&](bool block) -> bool {
        if (s_left == 0) {
          if (!more || (!block && !tested(&item_full[i & 1], (i >> 1) & 1u))) return false;
          FwdItem it;
          more = take(i, it);
          if (!more) return false;
          ++i;
          s_left = it.nt;
          q_wait = true;
          if (nt0 == 0) nt0 = it.nt; else if (nt1 == 0) nt1 = it.nt; else nt2 = it.nt;
        }
        if (!block && !tested(q_full, (i - 1) & 1u)) return false;
        ok = mbar_wait_warp(q_full, (i - 1) & 1u, abort_flag, ctl, kid | W_Q);
        q_wait = !ok;
        return ok;
      };
      while (true) {
        while (sg - pg < 3) {
          // S into buffer sg % 3: the PV product of tile sg - 3 is queued
          if ((s_left == 0 || q_wait) && !acquire(sg - pg <= 1)) break;
          const int s = (int)(sg % NST);
          ok = mbar_wait_warp_tested(&k_full[s], (sg / NST) & 1u, k_tested, abort_flag, ctl, kid | W_K);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d_tmem = tmem + (uint32_t)s * T::S_COL;
          const uint64_t kb = desc_off(dK0, (uint32_t)s * T::TILE);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * T::CHUNK + (kk & 3) * 32;
            mma_ss_w(d_tmem, desc_off(dQ0, off), desc_off(kb, off), IDS, kk > 0 ? 1u : 0u);
          }
          mma_commit_w(&s_full[s]);
          ++sg;
          --s_left;
          k_tested = 0;
        }
        if (!ok || pg == sg) break;
        const int s = (int)(pg % NST);
        const uint32_t ph = (pg / NST) & 1u;
        const uint32_t v_tested = mbar_test(&v_full[s], ph);   // V normally landed long ago
        k_tested = mbar_test(&k_full[sg % NST], (sg / NST) & 1u);
        // the first PV product overwrites O: the previous item's must have been read
        if (pv_n == 0 && ne > 0 && !mbar_wait_warp(o_free, (uint32_t)(ne - 1) & 1u, abort_flag, ctl, kid | W_OFREE))
          break;
        if (!mbar_wait_warp(&p_full[s], ph, abort_flag, ctl, kid | W_P)) break;
        if (!mbar_wait_warp_tested(&v_full[s], ph, v_tested, abort_flag, ctl, kid | W_V)) break;
        tc_fence_after();
        const uint32_t p_tmem = tmem + (uint32_t)s * T::S_COL;
        const uint64_t vb = desc_off(dV0, (uint32_t)s * T::TILE);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts_w(tmem + T::O_COL, p_tmem + kk * 8, desc_off(vb, kk * 16 * 128), IDO, (pv_n > 0 || kk > 0) ? 1u : 0u);
        mma_commit_w(&o_done[s]);
        ++pg;
        if (++pv_n == nt0) {
          mma_commit_w(o_final);
          ++ne;
          pv_n = 0;
          nt0 = nt1;
          nt1 = nt2;
          nt2 = 0;
        }
      }
      // TMEM is freed after the closing CTA-wide sync only once every MMA is done
      mma_commit_w(mma_drain);
      mbar_wait_warp(mma_drain, 0, nullptr, ctl, kid | W_DRAIN);
    }
  } else if (warp < 8) {
    regs_inc<kRegsSoftmax>();
    // ---------------- softmax warpgroup (warps 4..7) ----------------
    const int sp = warp & 3;
    const int r = sp * 32 + lane;
    const int rt = r / g.group;                  // the row's token in the tile
    const uint32_t lane_off = (uint32_t)(sp * 32) << 16;
    uint32_t gq = 0;
    int ne = 0;
    bool ok = true;
    FwdItem it;
    for (uint32_t i = 0; ok && take(i, it); ++i) {
      const int lim_r = g.causal ? min(it.left, it.lim0 + rt) : it.left;   // keys of this part that the row sees
      // a token's row that sees keys: rows behind the tile's tokens hold another sequence's queries
      const bool counts = rt < it.ntok && lim_r > 0;
      float m = 0.f, l = 0.f;
      uint32_t s_tested = 0u;   // S(n) already known complete (tested during tile n-1)
      for (int n = 0; n < it.nt; ++n) {
        const uint32_t gn = gq + (uint32_t)n;
        const int s = (int)(gn % NST);
        if (!mbar_wait_warp_tested(&s_full[s], (gn / NST) & 1u, s_tested, abort_flag, ctl, kid | W_S)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sb = tmem + lane_off + (uint32_t)s * T::S_COL;
        uint32_t xr[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(sb + c * 32, xr + c * 32);
        s_tested = (n + 1 < it.nt) ? mbar_test(&s_full[(gn + 1) % NST], ((gn + 1) / NST) & 1u) : 0u;
        tmem_ld_wait();
        if (n * 128 + 128 > it.lim0) {
          // keys at or past the row's limit: 32 at a time, and only where some row of the warp has any
          const int lim = lim_r - n * 128;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int have = lim - c * 32;
            if (__any_sync(0xffffffffu, have < 32)) {
              const uint32_t keep = have >= 32 ? 0xffffffffu : have <= 0 ? 0u : (1u << have) - 1u;
#pragma unroll
              for (int j = 0; j < 32; ++j) xr[c * 32 + j] = (keep >> j) & 1u ? xr[c * 32 + j] : 0xff800000u;   // -inf
            }
          }
        }
        // row max as 8 independent partial maxima (short dependency chains)
        auto row_max = [&]() -> float {
          float mx8[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) mx8[j] = __uint_as_float(xr[j]);
#pragma unroll
          for (int j = 8; j < 128; j += 16)
#pragma unroll
            for (int q = 0; q < 8; ++q)
              mx8[q] = j + 8 < 128 ? max3f(mx8[q], __uint_as_float(xr[j + q]), __uint_as_float(xr[j + 8 + q]))
                                   : fmaxf(mx8[q], __uint_as_float(xr[j + q]));
          return fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                       fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
        };
        // P = exp2(S c - m): exponent and row sum on packed fp32 pairs.  P is
        // rounded to bf16 as the tensor core's operand (V's type); the row sum
        // takes the unrounded values, so the rounding errors of P average out.
        uint32_t pk[64];
        auto exponentiate = [&](float mref) -> float {
          const uint64_t c2 = f2_pack(scale_log2, scale_log2), nm2 = f2_pack(-mref, -mref);
          uint64_t rs2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
          for (int j = 0; j < 64; ++j) {
            float x0, x1;
            f2_unpack(fma2(f2_pack(__uint_as_float(xr[2 * j]), __uint_as_float(xr[2 * j + 1])), c2, nm2), x0, x1);
            const float p0 = ex2(x0);
            const float p1 = ex2(x1);
            rs2[j & 3] = add2(rs2[j & 3], f2_pack(p0, p1));
            pk[j] = pack_bf16x2(p0, p1);
          }
          float a0, a1;
          f2_unpack(add2(add2(rs2[0], rs2[1]), add2(rs2[2], rs2[3])), a0, a1);
          return a0 + a1;
        };
        // The reference is the first tile's row maximum (every row's limit
        // covers a prefix of the part's keys, so a row that sees any of them
        // sees one in the first tile; one that sees none keeps 0).  A later
        // tile keeps it unless one of its values would pass 2^64, or all scores
        // before it were -inf (l = 0): those set no reference, and against the 0
        // in its place finite scores far below it would all vanish.
        float tsum;
        bool take_max = n == 0;
        while (true) {
          if (take_max) {
            const float mx = row_max() * scale_log2;
            if (n == 0) {
              m = mx == -INFINITY ? 0.f : mx;
            } else {
              // rescale this warp's O rows once the previous PV product has landed
              const float m_new = l != 0.f ? fmaxf(m, mx) : mx == -INFINITY ? 0.f : mx;
              const uint32_t gp = gn - 1;
              ok = mbar_wait_warp(&o_done[gp % NST], (gp / NST) & 1u, abort_flag, ctl, kid | W_O);
              if (!ok) break;
              tc_fence_after();
              const float alpha = l != 0.f ? ex2(m - m_new) : 1.f;   // (O is 0 where l is)
              l *= alpha;
              m = m_new;
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(tmem + lane_off + T::O_COL + c * 32, o);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                tmem_st32(tmem + lane_off + T::O_COL + c * 32, o);
              }
              tmem_st_wait();
            }
          }
          tsum = exponentiate(m);
          if (take_max || !__any_sync(0xffffffffu, counts && !(tsum <= 18446744073709551616.0f && l != 0.f))) break;   // 2^64
          take_max = true;
        }
        if (!ok) break;
        l += tsum;
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_st16(sb + c * 16, pk + c * 16);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&p_full[s]);
      }
      // one slot for the rows' statistics: the previous item's must have been read
      if (ok && ne > 0) ok = mbar_wait_warp(o_free, (uint32_t)(ne - 1) & 1u, abort_flag, ctl, kid | W_OFREE);
      if (!ok) break;
      // a row that saw no key has l = 0 and an O of zeros
      stat[r] = make_float2(l > 0.f || l != l ? 1.0f / l : 0.f, m + log2f(l));
      mbar_arrive(stat_full);
      gq += (uint32_t)it.nt;
      ++ne;
    }
  } else {
    regs_dec<kRegsOut>();
    // ---------------- output warpgroup (warps 8..11) ----------------
    const int sp = warp & 3;
    const int r = sp * 32 + lane;
    const int rt = r / g.group, rh = r - rt * g.group;   // the row's token and head in the tile
    const uint32_t lane_off = (uint32_t)(sp * 32) << 16;
    int ne = 0;
    FwdItem it;
    for (uint32_t i = 0; take(i, it); ++i) {
      const bool row_ok = rt < it.ntok;
      const int head = it.kvh * g.group + rh;
      const long long tok = (long long)it.tok + rt;
      const long long prow = (long long)it.part * part_rows + r;
      __nv_bfloat16* dst = O + head * o_head + tok * o_tok;
      float* ls = it.parts > 1 ? Lpart + prow : LSE + (long long)head * g.Tq + tok;
      if (!mbar_wait_warp(stat_full, (uint32_t)ne & 1u, abort_flag, ctl, kid | W_STAT) ||
          !mbar_wait_warp(o_final, (uint32_t)ne & 1u, abort_flag, ctl, kid | W_OFINAL))
        break;
      tc_fence_after();
      uint32_t o[D];
#pragma unroll
      for (int c = 0; c < D / 32; ++c) tmem_ld32(tmem + lane_off + T::O_COL + c * 32, o + c * 32);
      const float2 st = stat[r];
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive(o_free);
      ++ne;
      if (row_ok) {
#pragma unroll
        for (int j = 0; j < D; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * st.x);
        if (it.parts > 1) {
#pragma unroll
          for (int q = 0; q < D / 8; ++q) st_global_32(Opart + prow * D + q * 8, o + q * 8);
          *ls = st.y;
        } else {
#pragma unroll
          for (int j = 0; j < D / 2; ++j)
            o[j] = pack_bf16x2(__uint_as_float(o[2 * j]), __uint_as_float(o[2 * j + 1]));
          if (wide) {
#pragma unroll
            for (int q = 0; q < D / 16; ++q) st_global_32(dst + q * 16, o + q * 8);
          } else {
#pragma unroll
            for (int q = 0; q < D / 8; ++q)
              reinterpret_cast<uint4*>(dst)[q] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
          }
          *ls = st.y * kLn2;
        }
      }
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, T::TMEM_COLS);
}

// Joins the parts of a tile: with L_p the base-2 log-sums, M = max L_p and
// w_p = 2^(L_p - M):  O = sum w_p O_p / sum w_p,  lse = (M + log2 sum w_p) ln 2.
// A part that saw nothing of the row wrote no O: its weight is 0 and its values
// are left out.  A NaN among the L_p makes M and with it the row NaN (fmaxf
// alone would drop it, and a row of NaN parts would pass for one without keys).
// One CTA per query slot and key head (along x) and run of rows
// (along y); `wpr` warps share a row, each adding up every wpr-th part, and the
// first adds their sums in order.  Latency-bound: what a CTA has to know of its
// tile it works out before it waits for the parts, and few enough registers
// that all CTAs of a call are there at once (one wave of 147 registers took 25
// us where the parts themselves took 20).
template <int D>
__global__ void __launch_bounds__(256, 4)
    packed_combine_kernel(const __grid_constant__ PackedGeom g, int part_keys, int head_items, int part_rows, int wpr,
                          const float* __restrict__ Opart, const float* __restrict__ Lpart, __nv_bfloat16* O,
                          long long o_head, long long o_tok, float* LSE) {
  constexpr int V = D / 32;            // channels per lane
  constexpr int BATCH = 8;             // parts in flight
  using Vec = std::conditional_t<V == 4, float4, float2>;
  __shared__ Vec acc_s[8][32];
  __shared__ float sum_s[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kvh = blockIdx.x / g.nslot_q, slot = blockIdx.x - kvh * g.nslot_q;
  PackedSeq q;
  int tile = 0, parts = 0, base = 0;
  if (packed_find(g, g.q_ptr, g.TQ, slot, q)) {
    tile = slot - (q.q0 / g.TQ + q.s);
    if (tile * g.TQ < q.lq) {
      base = packed_items_before(g, part_keys, q.s, lane);
      packed_items(g, part_keys, q.s, parts);
      base += tile * parts;
      if (base + parts > head_items) parts = 0;
    }
  }
  cudaGridDependencySynchronize();
  if (parts <= 1) return;              // the part wrote the result itself
  const int t0 = tile * g.TQ, rows = min(g.TQ, q.lq - t0) * g.group;
  const int k = warp % wpr, per = 8 / wpr;
  const long long item0 = (long long)kvh * head_items + base;
  for (int r0 = blockIdx.y * per; r0 < rows; r0 += per * gridDim.y) {
    const int r = r0 + warp / wpr;
    const bool live = r < rows;
    float M = -INFINITY, sum = 0.f;
    float acc[V] = {};
    if (live) {
      const float* L = Lpart + item0 * part_rows + r;
      const float* src = Opart + (item0 * part_rows + r) * D + lane * V;
      bool nan = false;
      for (int p = lane; p < parts; p += 32) {
        const float lp = L[(long long)p * part_rows];
        nan |= lp != lp;
        M = fmaxf(M, lp);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      if (__any_sync(0xffffffffu, nan)) M = NAN;
      for (int p0 = k; p0 < parts && M != -INFINITY; p0 += BATCH * wpr) {
        Vec x[BATCH];
        float lp[BATCH];
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
          const long long p = p0 + j * wpr;
          lp[j] = -INFINITY;
          if (p < parts) {
            lp[j] = L[p * part_rows];
            x[j] = *reinterpret_cast<const Vec*>(src + p * part_rows * D);
          }
        }
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
          if (lp[j] == -INFINITY) continue;
          const float w = ex2(lp[j] - M);
          sum += w;
          const float* xv = reinterpret_cast<const float*>(&x[j]);
#pragma unroll
          for (int i = 0; i < V; ++i) acc[i] = fmaf(w, xv[i], acc[i]);
        }
      }
    }
    if (wpr > 1) {
      if (k > 0) {
        acc_s[warp][lane] = *reinterpret_cast<const Vec*>(acc);
        if (lane == 0) sum_s[warp] = sum;
      }
      __syncthreads();
      if (k == 0) {
        for (int o = 1; o < wpr; ++o) {
          const Vec x = acc_s[warp + o][lane];
          const float* xv = reinterpret_cast<const float*>(&x);
          sum += sum_s[warp + o];
#pragma unroll
          for (int i = 0; i < V; ++i) acc[i] += xv[i];
        }
      }
      __syncthreads();
    }
    if (!live || k > 0) continue;
    const float inv = M != -INFINITY ? 1.0f / sum : 0.f;
    const int rt = r / g.group, head = kvh * g.group + (r - rt * g.group);
    const long long tok = (long long)q.q0 + t0 + rt;
    uint32_t* dst = reinterpret_cast<uint32_t*>(O + head * o_head + tok * o_tok + lane * V);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) dst[i] = pack_bf16x2(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    if (lane == 0) LSE[(long long)head * g.Tq + tok] = M != -INFINITY ? (M + log2f(sum)) * kLn2 : -INFINITY;
  }
}

// Split over the keys.  With at least one query tile per SM the keys stay
// whole.  With fewer, every tile's keys are cut into parts of equal size.  What
// a part costs beside its keys is its rows: the load of Q, the fp32 O written
// and read again.  With few rows (single new tokens) the parts are as small as
// fill four rounds of the SMs (the lengths are not known on the host: uneven
// ones even out over the rounds), of four key tiles at least; with 32 rows or
// more, two rounds and eight tiles.  Measured, the one rule against the other:
// eight streams of one token, 3 rows, 67 / 69 us, one stream of 1 row 12.7 /
// 14.6; one head of 4096 tokens 24 / 21 us, two heads of two clips up to 4173
// tokens 42 / 32, 48 rows against 16 000 keys 22.6 / 19.8.
struct FwdSplit {
  int part_keys;     // 0: not split
  int items;         // bound on the items of a key head
  int rows;          // rows of a part
};
FwdSplit fwd_split(const dsv_packed& p) {
  FwdSplit sp{0, 0, 0};
  if (p.S <= 0 || p.Tq <= 0 || p.Tk <= 0) return sp;
  const int group = p.H / p.Hkv, TQ = 128 / group;
  const long long q_tiles = (p.Tq + TQ - 1) / TQ;          // of one sequence at most
  const long long most = q_tiles > p.S ? q_tiles : p.S;    // of all, roughly
  if (p.Hkv * most >= kPackedSMs) return sp;
  const long long key_tiles = (long long)p.Hkv * ((p.Tk + 127) / 128) * ((most + p.S - 1) / p.S);
  sp.rows = group * (p.Tq < TQ ? p.Tq : TQ);
  const long long fill = (sp.rows < 32 ? 4LL : 2LL) * kPackedSMs, least = sp.rows < 32 ? 4 : 8;
  long long part = (key_tiles + fill - 1) / fill;
  part = part < least ? least : part;
  if ((p.Tk + 127) / 128 <= part) return sp;               // one part at most
  sp.part_keys = (int)part * 128;
  // sum over sequences of tiles x parts: no sequence has more tiles than q_tiles, nor more parts than all keys
  const long long by_parts = q_tiles * ((long long)p.Tk / sp.part_keys + p.S);
  const long long by_tiles = packed_slots(p.Tq, TQ, p.S) * (((long long)p.Tk + sp.part_keys - 1) / sp.part_keys);
  sp.items = (int)(by_parts < by_tiles ? by_parts : by_tiles);
  return sp;
}

template <int D>
cudaError_t launch_t(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV, const PackedGeom& g,
                     const FwdSplit& sp, float scale, const dsv_view& O, float* lse, void* ws, const Ctl& ctl,
                     cudaStream_t st) {
  using T = PFwdTraits<D>;
  auto kern = packed_fwd_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, T::SMEM);
  if (e != cudaSuccess) return e;
  // a build with fewer registers per thread could not serve the warpgroups' split: never launch that
  static const int launched = [&] {
    cudaFuncAttributes a{};
    return cudaFuncGetAttributes(&a, kern) == cudaSuccess ? a.numRegs : 0;
  }();
  if (launched < kRegsLaunch) return cudaErrorInvalidKernelImage;
  const int items = sp.part_keys > 0 ? sp.items : g.nslot_q;
  const long long total = (long long)g.Hkv * items;
  // workspace: the parts' O, their log-sums
  float* Opart = sp.part_keys > 0 ? static_cast<float*>(ws) : nullptr;
  float* Lpart = sp.part_keys > 0 ? Opart + (size_t)total * sp.rows * D : nullptr;
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(O.ptr);
  const int wide = wide_rows(O);     // rows are stored a sector at a time
  kern<<<(unsigned)total, kFwdThreads, T::SMEM, st>>>(tmQ, tmK, tmV, g, sp.part_keys, sp.rows, items,
                                                      scale * 1.4426950408889634f, o, O.head_stride, O.token_stride,
                                                      lse, Opart, Lpart, wide, ctl);
  if ((e = cudaGetLastError()) != cudaSuccess || sp.part_keys == 0) return e;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  // a row's warps: up to eight parts each in one batch of loads
  const int most_parts = (g.Tk + sp.part_keys - 1) / sp.part_keys;
  const int wpr = most_parts <= 8 ? 1 : most_parts <= 16 ? 2 : most_parts <= 32 ? 4 : 8;
  cfg.gridDim = dim3((unsigned)(g.Hkv * g.nslot_q), (unsigned)((sp.rows * wpr + 15) / 16));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, packed_combine_kernel<D>, g, sp.part_keys, items, sp.rows, wpr,
                            static_cast<const float*>(Opart), static_cast<const float*>(Lpart), o,
                            (long long)O.head_stride, (long long)O.token_stride, lse);
}

}  // namespace

size_t packed_fwd_ws_bytes(const dsv_packed& p) {
  const FwdSplit sp = fwd_split(p);
  if (sp.part_keys == 0) return 0;
  const size_t total = (size_t)p.Hkv * sp.items;
  return total * sp.rows * (p.d + 1) * sizeof(float);
}

cudaError_t launch_packed_fwd(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                              const dsv_packed& p, const int32_t* q_ptr, const int32_t* k_ptr, int causal, float scale,
                              const dsv_view& O, float* lse, void* ws, const Ctl& ctl, cudaStream_t st) {
  const PackedGeom g = packed_geom(p, q_ptr, k_ptr, causal);
  const FwdSplit sp = fwd_split(p);
  return p.d == 128 ? launch_t<128>(tmQ, tmK, tmV, g, sp, scale, O, lse, ws, ctl, st)
                    : launch_t<64>(tmQ, tmK, tmV, g, sp, scale, O, lse, ws, ctl, st);
}

}  // namespace dsv
