// quantize.cu — rows to 8-bit floating point, a power-of-two scale for each
// block of 1 x 128 or 128 x 128 elements, and the transposed copy.
//
//   scale = 2^k with the least k for which the block's largest magnitude is at
//   most M 2^k (M = 448 for e4m3, 57344 for e5m2: both 1.75 times a power of
//   two),  q = round-to-nearest-even of x / scale.
// A power of two makes the division exact: q is the element rounded once, to
// half a step of the 8-bit type, and q * scale is exact in fp32.
// The gradient products of a projection sum over its rows, so they read the
// transposed matrix with blocks along the rows: both copies are made from one
// read of x.  A CTA holds a 128 x 128 tile in registers, 8 x 8 elements a
// thread, so both copies' block maxima are inside the CTA.
#include <cuda_fp8.h>

#include "dsv_launch.h"

namespace dsv {

namespace {

constexpr int kQThreads = 256, kTile = 128;

struct QuantArgs {
  const void* x;
  long long xs;
  int R, C;
  uint8_t* q;
  long long qs;
  float* scale;
  uint8_t* qt;             // [C, R], or null
  long long qts;
  float* scale_t;
};

// The block's scale and the multiplier that divides by it, from the bits of
// its largest magnitude.  TOP: the exponent of the type's largest value.  A
// block with an infinity or a NaN gets NaN for both.
template <int TOP>
__device__ __forceinline__ void block_scale(uint32_t amax, float* scale, float* inv) {
  int k = (int)(amax >> 23) - 127 - TOP + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);   // past 1.75
  k = max(k, -126);
  if (amax == 0u) k = 0;
  const bool bad = amax >= 0x7F800000u;
  *scale = bad ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float((uint32_t)(127 + k) << 23);
  *inv = bad ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float((uint32_t)(127 - k) << 23);
}
template <bool E5>
__device__ __forceinline__ uint32_t fp8x4(float a, float b, float c, float d) {
  constexpr __nv_fp8_interpretation_t T = E5 ? __NV_E5M2 : __NV_E4M3;
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, T);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, T);
  return lo | (hi << 16);
}
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// n of the 8 bytes of v, at an address that is a multiple of 8.
__device__ __forceinline__ void store_bytes(uint8_t* p, uint2 v, int n) {
  if (n >= 8) {
    *reinterpret_cast<uint2*>(p) = v;
  } else {
    for (int j = 0; j < n; ++j) p[j] = (uint8_t)((j < 4 ? v.x : v.y) >> (8 * (j & 3)));
  }
}

template <typename X, bool AL>
__device__ __forceinline__ void load_row8(const X* row, int c, int C, float* v) {
  if constexpr (AL && sizeof(X) == 2) {
    const uint4 q = c < C ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0, 0, 0, 0);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  } else if constexpr (AL) {
    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 p = c < C ? *reinterpret_cast<const float4*>(row + c) : z;
    const float4 q = c < C ? *reinterpret_cast<const float4*>(row + c + 4) : z;
    v[0] = p.x, v[1] = p.y, v[2] = p.z, v[3] = p.w, v[4] = q.x, v[5] = q.y, v[6] = q.z, v[7] = q.w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + j < C ? (float)row[c + j] : 0.f;
  }
}

// Thread: rows 8 u .. 8 u + 7 and columns 8 l .. 8 l + 7 of the tile, u = tid / 16, l = tid % 16.
template <typename X, bool AL, bool E5, bool SQUARE, bool TRANS>
__global__ void __launch_bounds__(kQThreads) quantize_kernel(QuantArgs a, int tiles_c) {
  constexpr int TOP = E5 ? 15 : 8;
  __shared__ uint32_t red[kQThreads / 32][kTile];
  __shared__ uint2 turn[TRANS ? kTile * 16 : 1];          // [column][8 rows each], its units swapped by column / 8
  const int u = threadIdx.x >> 4, l = threadIdx.x & 15, warp = threadIdx.x >> 5;
  const int tc = (int)(blockIdx.x % tiles_c), tr = (int)(blockIdx.x / tiles_c);
  const int row0 = tr * kTile + 8 * u, col0 = tc * kTile + 8 * l;
  const X* x = static_cast<const X*>(a.x);
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (row0 + i < a.R) {
      load_row8<X, AL>(x + (long long)(row0 + i) * a.xs, col0, a.C, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    }
  }
  // magnitudes as bit patterns: NaN ranks above infinity, infinity above numbers
  uint32_t rmax[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t m = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, mag(v[i][j]));
    rmax[i] = m;
  }
  float inv[8];
  if constexpr (SQUARE) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, rmax[i]);
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) red[0][warp] = m;
    __syncthreads();
    m = 0u;
#pragma unroll
    for (int w = 0; w < kQThreads / 32; ++w) m = max(m, red[0][w]);
    float sc;
    block_scale<TOP>(m, &sc, &inv[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) inv[i] = inv[0];
    if (threadIdx.x == 0) {
      a.scale[(long long)tc * ((a.R + kTile - 1) / kTile) + tr] = sc;
      if (TRANS) a.scale_t[(long long)tr * tiles_c + tc] = sc;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t m = rmax[i];
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      float sc;
      block_scale<TOP>(m, &sc, &inv[i]);
      if (l == 0 && row0 + i < a.R) a.scale[(long long)tc * a.R + row0 + i] = sc;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float f = inv[i];
    const uint2 b = make_uint2(fp8x4<E5>(v[i][0] * f, v[i][1] * f, v[i][2] * f, v[i][3] * f),
                               fp8x4<E5>(v[i][4] * f, v[i][5] * f, v[i][6] * f, v[i][7] * f));
    if (row0 + i < a.R && col0 < a.C) store_bytes(a.q + (long long)(row0 + i) * a.qs + col0, b, a.C - col0);
  }
  if constexpr (TRANS) {
    float ct[8];
    if constexpr (SQUARE) {
#pragma unroll
      for (int j = 0; j < 8; ++j) ct[j] = inv[0];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, mag(v[i][j]));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 16));
        if ((threadIdx.x & 31) < 16) red[warp][8 * l + j] = m;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t m = 0u;
#pragma unroll
        for (int w = 0; w < kQThreads / 32; ++w) m = max(m, red[w][8 * l + j]);
        float sc;
        block_scale<TOP>(m, &sc, &ct[j]);
        if (u == 0 && col0 + j < a.C) a.scale_t[(long long)tr * a.C + col0 + j] = sc;
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float f = ct[j];
      turn[(8 * l + j) * 16 + (u ^ l)] = make_uint2(fp8x4<E5>(v[0][j] * f, v[1][j] * f, v[2][j] * f, v[3][j] * f),
                                                    fp8x4<E5>(v[4][j] * f, v[5][j] * f, v[6][j] * f, v[7][j] * f));
    }
    __syncthreads();
    const int r0 = tr * kTile + 8 * l;                    // this thread writes rows r0 .. r0 + 7 of column 16 k + u
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = 16 * k + u, col = tc * kTile + c;
      if (col < a.C && r0 < a.R) store_bytes(a.qt + (long long)col * a.qts + r0, turn[c * 16 + (l ^ (c >> 3))], a.R - r0);
    }
  }
}

template <typename X, bool AL, bool E5>
cudaError_t quant_t(const QuantArgs& a, int rows, cudaStream_t st) {
  const int tc = (a.C + kTile - 1) / kTile;
  const unsigned grid = (unsigned)((long long)tc * ((a.R + kTile - 1) / kTile));
  if (rows == 1) {
    if (a.qt) quantize_kernel<X, AL, E5, false, true><<<grid, kQThreads, 0, st>>>(a, tc);
    else quantize_kernel<X, AL, E5, false, false><<<grid, kQThreads, 0, st>>>(a, tc);
  } else {
    if (a.qt) quantize_kernel<X, AL, E5, true, true><<<grid, kQThreads, 0, st>>>(a, tc);
    else quantize_kernel<X, AL, E5, true, false><<<grid, kQThreads, 0, st>>>(a, tc);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize(const dsv_rows& x, int R, int C, int rows, const dsv_rows& q, float* scale,
                            const dsv_rows& qt, float* scale_t, cudaStream_t st) {
  QuantArgs a;
  a.x = x.ptr;
  a.xs = x.stride;
  a.R = R;
  a.C = C;
  a.q = static_cast<uint8_t*>(q.ptr);
  a.qs = q.stride;
  a.scale = scale;
  a.qt = static_cast<uint8_t*>(qt.ptr);
  a.qts = qt.stride;
  a.scale_t = scale_t;
  const int size = x.type == DSV_F32 ? 4 : 2;
  // 16-byte loads: 8 columns lie inside a row or behind it
  const bool al = C % 8 == 0 && (reinterpret_cast<uintptr_t>(x.ptr) & 15u) == 0 && (x.stride * size) % 16 == 0;
  const bool e5 = q.type == DSV_E5M2;
  if (x.type == DSV_F32) {
    if (al) return e5 ? quant_t<float, true, true>(a, rows, st) : quant_t<float, true, false>(a, rows, st);
    return e5 ? quant_t<float, false, true>(a, rows, st) : quant_t<float, false, false>(a, rows, st);
  }
  if (al) return e5 ? quant_t<__nv_bfloat16, true, true>(a, rows, st) : quant_t<__nv_bfloat16, true, false>(a, rows, st);
  return e5 ? quant_t<__nv_bfloat16, false, true>(a, rows, st) : quant_t<__nv_bfloat16, false, false>(a, rows, st);
}

}  // namespace dsv
