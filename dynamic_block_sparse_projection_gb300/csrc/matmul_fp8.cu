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
constexpr int kKb = 128;                   // elements and bytes of a block along K: one swizzle row

enum : unsigned int { W_EMPTY = 1, W_FULL = 2, W_FREE = 3, W_SUMS = 4, W_DRAIN = 5 };

struct MmArgs {
  int M, N, kbs;                           // rows of C, columns, blocks of K
  int tm, tn;                              // tiles
  const float* sa;
  const float* sb;
  long long sa_ld, sb_ld;                  // scales of a block of K
  int sa_shift, sb_shift;                  // 0: a scale for each row, 7: for 128 rows
  void* c;
  long long ldc;
  int accumulate, vec;                     // vec: rows of C are 32-byte aligned
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
  static constexpr int BM = 128, STAGES = 6;
  static constexpr int A_BYTES = BM * kKb, B_BYTES = BN * kKb, STAGE = A_BYTES + B_BYTES;
  static constexpr int SMEM = STAGES * STAGE + 1024;
  static constexpr int TMEM = 2 * BN;
};

// COLV: b has a scale for each row (a column of C); else one for 128.
template <int BN, bool COLV, bool F32>
__global__ void __launch_bounds__(kMmThreads, 1)
    matmul_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, MmArgs g, Ctl ctl) {
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
      if (!ok || !in) continue;
      if constexpr (F32) {
        float* out = static_cast<float*>(g.c) + (long long)row * g.ldc + col;
#pragma unroll
        for (int j = 0; j < HALF / 2; j += 4) {
          float v[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) f2_unpack(acc[j + i], v[2 * i], v[2 * i + 1]);
          const int c = col + 2 * j;
          if (g.vec && c + 8 <= g.N) {
            if (g.accumulate) {
              const float4 x = *reinterpret_cast<const float4*>(out + 2 * j), y = *reinterpret_cast<const float4*>(out + 2 * j + 4);
              v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w, v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
            }
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[i]);
            st_global_32(out + 2 * j, w);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (c + i < g.N) out[2 * j + i] = g.accumulate ? out[2 * j + i] + v[i] : v[i];
          }
        }
      } else {
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(g.c) + (long long)row * g.ldc + col;
#pragma unroll
        for (int j = 0; j < HALF / 2; j += 8) {
          float v[16];
#pragma unroll
          for (int i = 0; i < 8; ++i) f2_unpack(acc[j + i], v[2 * i], v[2 * i + 1]);
          const int c = col + 2 * j;
          if (g.vec && c + 16 <= g.N) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
            st_global_32(out + 2 * j, w);
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (c + i < g.N) out[2 * j + i] = __float2bfloat16_rn(v[i]);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssueWarp) tmem_dealloc(tmem, T::TMEM);
}

template <int BN, bool COLV, bool F32>
cudaError_t matmul_t(const CUtensorMap& tmA, const CUtensorMap& tmB, MmArgs g, const Ctl& ctl, cudaStream_t st) {
  using T = MmTraits<BN>;
  auto kern = matmul_kernel<BN, COLV, F32>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, T::SMEM);
  if (e != cudaSuccess) return e;
  const int tiles = g.tm * g.tn;
  kern<<<tiles < 152 ? tiles : 152, kMmThreads, T::SMEM, st>>>(tmA, tmB, g, ctl);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_matmul_fp8(const CUtensorMap& tmA, const CUtensorMap& tmB, const dsv_matmul& p, bool a_e5, bool b_e5,
                              const float* sa, const float* sb, const dsv_rows& c, const Ctl& ctl, cudaStream_t st) {
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
  const bool f32 = c.type == DSV_F32;
  g.vec = (reinterpret_cast<uintptr_t>(c.ptr) & 31u) == 0 && (c.stride * (f32 ? 4 : 2)) % 32 == 0;
  g.idesc = idesc_f8(128, 128, a_e5, b_e5);
  if (p.b_rows == 1)
    return f32 ? matmul_t<128, true, true>(tmA, tmB, g, ctl, st) : matmul_t<128, true, false>(tmA, tmB, g, ctl, st);
  return f32 ? matmul_t<128, false, true>(tmA, tmB, g, ctl, st) : matmul_t<128, false, false>(tmA, tmB, g, ctl, st);
}

}  // namespace dsv
