// packed.cuh — geometry of the packed-sequence attention, shared by its kernels.
//
// S sequences lie one behind the other on the token axis: sequence s owns the
// query tokens q_ptr[s] .. q_ptr[s+1]-1 and the keys k_ptr[s] .. k_ptr[s+1]-1.
// The row pointers live on the device and the host never reads them, so the
// tiles are found by the kernels.
//
// Query tile.  The 128 rows of a tile are TQ = 128 / group tokens times the
// `group` query heads that share one key head, row = token * group + head: one
// K/V tile then serves all of them, a single new token fills `group` rows, and
// the sums over shared heads in dK and dV are the product's own row sum.
//
// Slots.  Tile i of sequence s has the slot q_ptr[s] / TQ + s + i.  A
// sequence of L tokens gets at least ceil(L / TQ) slots before the next one's
// first, so slots never collide, their number is at most Tq / TQ + S (known on
// the host), and a slot's sequence is found by a binary search in q_ptr alone:
// no prefix sums over tile counts, no launch that makes a plan.  At most S
// slots are empty.  Key tiles (128 keys) have slots by the same rule on k_ptr.
#pragma once

#include "dsv_launch.h"

namespace dsv {

struct PackedGeom {
  const int32_t* q_ptr;
  const int32_t* k_ptr;
  int S, H, Hkv, group, TQ;      // group = H / Hkv, TQ = 128 / group
  int Tq, Tk;
  int nslot_q, nslot_k;
  int causal;
  int head_chunk;                // key heads whose tiles are taken together (L2 reuse)
};

// Heads per chunk: their K and V within ~48 MB of L2.
inline PackedGeom packed_geom(const dsv_packed& p, const int32_t* q_ptr, const int32_t* k_ptr, int causal) {
  PackedGeom g{};
  g.q_ptr = q_ptr;
  g.k_ptr = k_ptr;
  g.S = p.S;
  g.H = p.H;
  g.Hkv = p.Hkv;
  g.group = p.H / p.Hkv;
  g.TQ = 128 / g.group;
  g.Tq = p.Tq;
  g.Tk = p.Tk;
  g.nslot_q = (int)packed_slots(p.Tq, g.TQ, p.S);
  g.nslot_k = (int)packed_slots(p.Tk, 128, p.S);
  g.causal = causal;
  const long long head_bytes = 4LL * p.Tk * p.d;
  const long long hc = (48LL << 20) / (head_bytes > 0 ? head_bytes : 1);
  g.head_chunk = (int)(hc < 1 ? 1 : hc > p.Hkv ? p.Hkv : hc);
  return g;
}

// Rows on 32-byte boundaries.
inline int wide_rows(const dsv_view& v) {
  return reinterpret_cast<uintptr_t>(v.ptr) % 32 == 0 && v.head_stride % 16 == 0 && v.token_stride % 16 == 0;
}

struct PackedSeq {
  int s, q0, lq, k0, lk;
};

// Sequence of a slot (tile = rows per tile, ptr = q_ptr or k_ptr), false for
// a slot before the first sequence or a sequence whose pointers are out of
// range (packed_check_ptrs reports those).  Pointers that do not rise send the
// search anywhere, but what it returns true for is a sequence whose own
// pointers are in range and a slot at or after its first: tiles, and the slots
// of its rows in the workspace, stay in bounds.
__device__ __forceinline__ bool packed_find(const PackedGeom& g, const int32_t* ptr, int tile, int slot,
                                            PackedSeq& q) {
  int lo = 0, hi = g.S - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    // ptr[mid] / tile + mid <= slot
    if (ptr[mid] < (long long)(slot - mid + 1) * tile) lo = mid; else hi = mid - 1;
  }
  q.s = lo;
  const int a = g.q_ptr[lo], b = g.q_ptr[lo + 1], c = g.k_ptr[lo], d = g.k_ptr[lo + 1];
  if (a < 0 || b < a || b > g.Tq || c < 0 || d < c || d > g.Tk) return false;
  q.q0 = a;
  q.lq = b - a;
  q.k0 = c;
  q.lk = d - c;
  return ptr[lo] < (long long)(slot - lo + 1) * tile;
}

// Split tiles: item m of a key head, over the sequences in order, inside one
// over its query tiles, inside a tile over the parts of `part_keys` keys.  One
// warp adds up the sequences' item counts (they are few where tiles are split:
// fewer than SMs).  part < 0: m is past the last item.
struct PackedPart {
  int tile, part, parts;
};
__device__ __forceinline__ int packed_items(const PackedGeom& g, int part_keys, int s, int& parts) {
  const int a = g.q_ptr[s], b = g.q_ptr[s + 1], c = g.k_ptr[s], d = g.k_ptr[s + 1];
  parts = 0;
  if (a < 0 || b < a || b > g.Tq || c < 0 || d < c || d > g.Tk) return 0;
  parts = max(1, (d - c + part_keys - 1) / part_keys);
  return (b - a + g.TQ - 1) / g.TQ * parts;
}
__device__ __forceinline__ PackedPart packed_part(const PackedGeom& g, int part_keys, int m, int lane, PackedSeq& q) {
  int base = 0;
  for (int s0 = 0; s0 < g.S; s0 += 32) {
    int parts = 0;
    const int own = s0 + lane < g.S ? packed_items(g, part_keys, s0 + lane, parts) : 0;
    int inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, base + inc > m);
    if (hit != 0u) {
      const int l = __ffs(hit) - 1;
      const int first = base + __shfl_sync(0xffffffffu, inc - own, l);
      parts = __shfl_sync(0xffffffffu, parts, l);
      q.s = s0 + l;
      q.q0 = g.q_ptr[q.s];
      q.lq = g.q_ptr[q.s + 1] - q.q0;
      q.k0 = g.k_ptr[q.s];
      q.lk = g.k_ptr[q.s + 1] - q.k0;
      const int in = m - first;
      return {in / parts, in % parts, parts};
    }
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  return {0, -1, 0};
}
// The items of a key head that lie before sequence s's, by one warp.
__device__ __forceinline__ int packed_items_before(const PackedGeom& g, int part_keys, int s, int lane) {
  int n = 0, parts;
  for (int i = lane; i < s; i += 32) n += packed_items(g, part_keys, i, parts);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n;
}
// Both row pointers must rise within [0, T]: one warp reports a sequence that
// breaks it (its tiles are skipped by packed_find).
__device__ __forceinline__ void packed_check_ptrs(const PackedGeom& g, const Ctl& ctl, int lane) {
#pragma unroll 4
  for (int s = lane; s < g.S; s += 32) {
    const int a = g.q_ptr[s], b = g.q_ptr[s + 1], c = g.k_ptr[s], d = g.k_ptr[s + 1];
    if (a < 0 || b < a || b > g.Tq || c < 0 || d < c || d > g.Tk) set_error(ctl, DSV_ERR_BAD_INDEX, (unsigned)s);
  }
}

// (key head, slot) of work index idx: chunks of head_chunk key heads, inside a
// chunk the slots (descending where the later tiles of a causal sequence are
// the longest), inside a slot the heads.
__device__ __forceinline__ void packed_order(const PackedGeom& g, int nslot, bool descending, int idx, int& kvh,
                                             int& slot) {
  const unsigned per = (unsigned)g.head_chunk * (unsigned)nslot;   // Hkv * nslot < 2^31
  const int c = (int)((unsigned)idx / per);
  const int in = idx - c * (int)per;
  const int heads = min(g.head_chunk, g.Hkv - c * g.head_chunk);
  const int sl = (int)((unsigned)in / (unsigned)heads);
  kvh = c * g.head_chunk + (in - sl * heads);
  slot = descending ? nslot - 1 - sl : sl;
}

__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int x, int y,
                                            int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
          "r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// Zero rows [row0, 128) of a tile of `chunks` 64-column chunks of 128 rows x
// 128 bytes each (the swizzle permutes bytes inside a row only), by one warp,
// ordered before later tensor-core reads.
__device__ __forceinline__ void zero_tile_rows(uint8_t* tile, int chunks, int row0, int lane) {
  for (int c = 0; c < chunks; ++c) {
    uint4* z = reinterpret_cast<uint4*>(tile + c * 16384 + row0 * 128);
    for (int i = lane; i < (128 - row0) * 8; i += 32) z[i] = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

}  // namespace dsv
