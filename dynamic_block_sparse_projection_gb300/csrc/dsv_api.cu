// dsv_api.cu — the C ABI of libdsv: argument checks, TMA descriptors, dispatch.
//
// Every entry point validates its arguments on the host before any launch
// (returning DSV_ERR_INVALID_ARG / DSV_ERR_UNSUPPORTED and writing nothing),
// then enqueues its kernels on the caller's stream without synchronising
// (dsv_predict_topk_blocks also forks part of its work onto a library-owned
// side stream and joins it back with events).
#include <cudaTypedefs.h>
#include <math.h>
#include <stdint.h>

#include <mutex>

#include "dsv_launch.h"

namespace dsv {

// One error word per device: the first device-side error since the last clear.
static __device__ DeviceErr g_err_word;

namespace {

constexpr int kMaxDevices = 64;
constexpr unsigned long long kDefaultWaitNs = 1000000000ULL;

std::mutex g_mu;
DeviceErr* g_err_addr[kMaxDevices] = {};
unsigned long long g_limit_ns[kMaxDevices] = {};
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

dsv_status from_cuda(cudaError_t e) { return e == cudaSuccess ? DSV_OK : DSV_ERR_CUDA; }

// A second stream (and two events) per device for the fused predictor +
// top-k: the transposed lists of the heads whose rows are all selected are
// built there while the select kernel's last, partly filled wave runs on the
// caller's stream.  g_fork_mu keeps one call's record / wait / launch
// sequence on these objects from interleaving with another's.
struct ForkRes {
  cudaStream_t side = nullptr;
  cudaEvent_t main_done = nullptr, side_done = nullptr;
  int nsm = 0;
};
ForkRes g_fork[kMaxDevices];
std::mutex g_fork_mu;

cudaError_t fork_res(ForkRes** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_mu);
  ForkRes& f = g_fork[dev];
  if (f.side == nullptr) {
    ForkRes n;
    if ((e = cudaDeviceGetAttribute(&n.nsm, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    if ((e = cudaStreamCreateWithFlags(&n.side, cudaStreamNonBlocking)) != cudaSuccess) return e;
    if ((e = cudaEventCreateWithFlags(&n.main_done, cudaEventDisableTiming)) != cudaSuccess) return e;
    if ((e = cudaEventCreateWithFlags(&n.side_done, cudaEventDisableTiming)) != cudaSuccess) return e;
    f = n;
  }
  *out = &f;
  return cudaSuccess;
}

// Control block of the current device (error word address, wait limit).
cudaError_t current_ctl(Ctl* ctl) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_mu);
  if (g_err_addr[dev] == nullptr) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_err_word);
    if (e != cudaSuccess) return e;
    g_err_addr[dev] = static_cast<DeviceErr*>(p);
  }
  ctl->err = g_err_addr[dev];
  ctl->wait_limit_ns = g_limit_ns[dev] ? g_limit_ns[dev] : kDefaultWaitNs;
  return cudaSuccess;
}

cudaError_t get_encode(PFN_cuTensorMapEncodeTiled_v12000* out) {
  std::lock_guard<std::mutex> lock(g_mu);
  if (g_encode == nullptr) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || fn == nullptr) return cudaErrorNotSupported;
    g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }
  *out = g_encode;
  return cudaSuccess;
}

// 2D map over a [rows, d] bf16 tensor, box = [box_rows, 64 columns], 128-byte swizzle.
cudaError_t make_map(CUtensorMap* map, const void* base, long long rows, int d, int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc;
  cudaError_t e = get_encode(&enc);
  if (e != cudaSuccess) return e;
  cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)d * 2};
  cuuint32_t box[2] = {64u, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1u, 1u};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// 2D map over a [rows, 32] fp32 array, box = [32 columns, box_rows], 128-byte swizzle
// (the tf32 operand tiles of the fused predictor + top-k).
cudaError_t make_map_f32x32(CUtensorMap* map, const void* base, long long rows, int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc;
  cudaError_t e = get_encode(&enc);
  if (e != cudaSuccess) return e;
  cuuint64_t dims[2] = {32u, (cuuint64_t)rows};
  cuuint64_t strides[1] = {32u * 4u};
  cuuint32_t box[2] = {32u, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1u, 1u};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool al256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

// Common shape rules.  Returns DSV_OK, or the status to return.
dsv_status check_shape(const dsv_shape& s, bool need_r) {
  if (s.B < 0 || s.H < 0 || s.N < 0) return DSV_ERR_INVALID_ARG;
  if (s.block != 64 && s.block != 128) return DSV_ERR_UNSUPPORTED;
  if (s.d != 64 && s.d != 128) return DSV_ERR_UNSUPPORTED;
  if (s.N % s.block != 0) return DSV_ERR_INVALID_ARG;
  if (need_r && (s.r < 8 || s.r > 64 || s.r % 8 != 0)) return DSV_ERR_UNSUPPORTED;
  if (s.H > kMaxHeads) return DSV_ERR_UNSUPPORTED;
  if ((long long)s.B * s.H > 65535) return DSV_ERR_UNSUPPORTED;
  if ((long long)s.B * s.H * s.N >= (1LL << 31)) return DSV_ERR_UNSUPPORTED;
  return DSV_OK;
}

// 3D map over heads x tokens x d bf16 with the view's strides, box = [box_tok,
// box_heads, 64 columns]: the rows of a box come token by token, the heads of
// a token one behind the other.  128-byte swizzle.
cudaError_t make_map_view(CUtensorMap* map, const dsv_view& v, int heads, int tokens, int d, int box_heads,
                          int box_tok) {
  PFN_cuTensorMapEncodeTiled_v12000 enc;
  cudaError_t e = get_encode(&enc);
  if (e != cudaSuccess) return e;
  // the stride of a dimension of one element is never used: any valid one will do
  const long long hs = heads > 1 ? v.head_stride : d, ts = tokens > 1 ? v.token_stride : d;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
  cuuint64_t strides[2] = {(cuuint64_t)hs * 2, (cuuint64_t)ts * 2};
  cuuint32_t box[3] = {64u, (cuuint32_t)box_heads, (cuuint32_t)box_tok};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, v.ptr, dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// A view's strides: multiples of 8 elements (16 bytes) below 2^38, at least d
// along every dimension of more than one element.
constexpr long long kMaxStride = 1LL << 38;
bool stride_ok(long long stride, long long size, int d) {
  return size <= 1 || (stride >= d && stride < kMaxStride && stride % 8 == 0);
}
// The rows of an output must not overlap: with the dimensions sorted by
// stride, each stride spans the smaller dimensions.
bool disjoint(const long long* stride, const long long* size, int n, int d) {
  bool used[3] = {false, false, false};
  long long span = d;
  for (int k = 0; k < n; ++k) {
    int at = -1;
    for (int i = 0; i < n; ++i)
      if (!used[i] && size[i] > 1 && (at < 0 || stride[i] < stride[at])) at = i;
    if (at < 0) return true;
    if (stride[at] < span) return false;
    span = stride[at] * (size[at] - 1) + span;
    used[at] = true;
  }
  return true;
}
bool view_ok(const dsv_view& v, long long heads, long long tokens, int d, bool output) {
  if (!v.ptr || !al16(v.ptr)) return false;
  if (!stride_ok(v.head_stride, heads, d) || !stride_ok(v.token_stride, tokens, d)) return false;
  const long long st[2] = {v.head_stride, v.token_stride}, sz[2] = {heads, tokens};
  return !output || disjoint(st, sz, 2, d);
}
bool view4_ok(const dsv_view& v, long long B, long long H, long long N, int d, bool output) {
  if (!view_ok(v, H, N, d, false) || !stride_ok(v.batch_stride, B, d)) return false;
  const long long st[3] = {v.batch_stride, v.head_stride, v.token_stride}, sz[3] = {B, H, N};
  return !output || disjoint(st, sz, 3, d);
}

// The same rows as `a`, where both start at the same address.
bool same_or_apart(const dsv_view& a, const dsv_view& b, long long B, long long H, long long N) {
  if (a.ptr != b.ptr) return true;
  return (B <= 1 || a.batch_stride == b.batch_stride) && (H <= 1 || a.head_stride == b.head_stride) &&
         (N <= 1 || a.token_stride == b.token_stride);
}

// Packed attention: sizes, then whether a call has anything to do.
dsv_status check_packed(const dsv_packed& p) {
  if (p.S < 0 || p.H < 0 || p.Hkv < 0 || p.Tq < 0 || p.Tk < 0) return DSV_ERR_INVALID_ARG;
  if (p.d != 64 && p.d != 128) return DSV_ERR_UNSUPPORTED;
  if (p.H > kMaxHeads) return DSV_ERR_UNSUPPORTED;
  if (p.H == 0 || p.S == 0) return DSV_OK;
  if (p.Hkv == 0 || p.H % p.Hkv != 0) return DSV_ERR_INVALID_ARG;
  if (p.H / p.Hkv > 128) return DSV_ERR_UNSUPPORTED;
  // slots, work indexes and token coordinates stay inside 32 bits
  const long long q = packed_slots(p.Tq, 128 / (p.H / p.Hkv), p.S), k = packed_slots(p.Tk, 128, p.S);
  if ((long long)p.Tq + 128LL * p.S >= (1LL << 31) || (long long)p.Tk + 128LL * p.S >= (1LL << 31))
    return DSV_ERR_UNSUPPORTED;
  if (q * p.Hkv >= (1LL << 31) || k * p.Hkv >= (1LL << 31)) return DSV_ERR_UNSUPPORTED;
  return DSV_OK;
}
// Waits of a packed call: some last as long as a tile's whole stream of other
// tiles, so the limit grows with the longest possible one (10 us a tile, some
// ten times what it takes).
void widen_wait(Ctl* ctl, const dsv_packed& p) {
  const unsigned long long tiles = (unsigned long long)p.Tk / 128 + (unsigned long long)p.Tq / (128 / (p.H / p.Hkv)) + 2;
  ctl->wait_limit_ns += tiles * 10000ull;
}
bool no_queries(const dsv_packed& p) { return p.S == 0 || p.H == 0 || p.Tq == 0; }
bool no_keys(const dsv_packed& p) { return p.S == 0 || p.H == 0 || p.Tk == 0; }
float packed_scale(int d, float scale) { return (scale > 0.f && isfinite(scale)) ? scale : 1.0f / sqrtf((float)d); }

dsv_status check_rope(const dsv_rope& r) {
  if (r.B < 0 || r.H < 0 || r.N < 0) return DSV_ERR_INVALID_ARG;
  if (r.d != 64 && r.d != 128) return DSV_ERR_UNSUPPORTED;
  if (r.axes < 1 || r.axes > 4) return DSV_ERR_UNSUPPORTED;
  int sum = 0;
  for (int a = 0; a < r.axes; ++a) {
    if (r.section[a] < 2 || r.section[a] > r.d || r.section[a] % 2 != 0) return DSV_ERR_INVALID_ARG;
    sum += r.section[a];
  }
  if (sum > r.d) return DSV_ERR_INVALID_ARG;
  if (!(r.theta >= 1.0) || !isfinite(r.theta)) return DSV_ERR_INVALID_ARG;
  if (r.H > kMaxHeads || r.B > 65535) return DSV_ERR_UNSUPPORTED;
  if ((long long)r.B * r.H * (r.N / 16 + 1) >= (1LL << 31)) return DSV_ERR_UNSUPPORTED;
  if (r.N > INT32_MAX - 32) return DSV_ERR_UNSUPPORTED;   // token indexes of the last tile stay inside 32 bits
  return DSV_OK;
}
bool empty_rope(const dsv_rope& r) { return r.B == 0 || r.H == 0 || r.N == 0; }
bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Matrices of the calls behind the packed attention.
int size_of(int type) { return type == DSV_F32 ? 4 : type == DSV_BF16 ? 2 : 1; }
bool real_type(const dsv_rows& v) { return v.type == DSV_BF16 || v.type == DSV_F32; }
bool fp8_type(const dsv_rows& v) { return v.type == DSV_E4M3 || v.type == DSV_E5M2; }
bool rows_ok(const dsv_rows& v, long long rows, long long cols) {
  if (!v.ptr || reinterpret_cast<uintptr_t>(v.ptr) % size_of(v.type) != 0) return false;
  return rows <= 1 || (v.stride >= cols && v.stride < kMaxStride);
}
bool fp8_ok(const dsv_rows& v, long long rows, long long cols) {
  return fp8_type(v) && rows_ok(v, rows, cols) && al16(v.ptr) && (rows <= 1 || v.stride % 16 == 0);
}
// The same rows as `a`, where both start at the same address.
bool same_or_apart(const dsv_rows& a, const dsv_rows& b, long long rows) {
  return a.ptr != b.ptr || (a.type == b.type && (rows <= 1 || a.stride == b.stride));
}

dsv_status check_norm(const dsv_norm& p) {
  if (p.T < 0 || p.C < 0 || p.S < 0) return DSV_ERR_INVALID_ARG;
  if (p.T >= (1 << 30) || p.C < 1 || p.C > 16384 || p.S > 65535) return DSV_ERR_UNSUPPORTED;
  return DSV_OK;
}

// 2D map over a [rows, cols] matrix, box = [box_rows, 128 bytes], 128-byte swizzle.
cudaError_t make_map_rows(CUtensorMap* map, const dsv_rows& v, long long rows, long long cols, int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc;
  cudaError_t e = get_encode(&enc);
  if (e != cudaSuccess) return e;
  const int size = size_of(v.type);
  // the stride of a single row is never used: any valid one will do
  const long long stride = rows > 1 ? v.stride * size : (cols * size + 15) / 16 * 16;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)stride};
  cuuint32_t box[2] = {128u / size, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1u, 1u};
  const CUtensorMapDataType type = size == 4   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : size == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                               : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  CUresult r = enc(map, type, 2, v.ptr, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

bool empty(const dsv_shape& s) { return (long long)s.B * s.H * s.N == 0; }

float resolve_scale(const dsv_shape& s, float scale) {
  return (scale > 0.f && isfinite(scale)) ? scale : 1.0f / sqrtf((float)s.d);
}

// One thread waits on a barrier that nothing arrives at: phase 0 of a freshly
// initialised barrier never completes, so the bounded wait runs out, records
// DSV_ERR_TIMEOUT and returns.  Nothing else is in flight in this CTA.
__global__ void selftest_wait_kernel(Ctl ctl) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  mbar_init(&bar, 1);
  abort_flag = 0;
  fence_mbar_init();
  mbar_wait(&bar, 0, &abort_flag, ctl, DSV_SELFTEST_WAIT_ID);
}

}  // namespace
}  // namespace dsv

using namespace dsv;

extern "C" {

int32_t dsv_version(void) { return 10000; }


const char* dsv_status_string(dsv_status st) {
  switch (st) {
    case DSV_OK: return "ok";
    case DSV_ERR_INVALID_ARG: return "invalid argument";
    case DSV_ERR_UNSUPPORTED: return "unsupported size";
    case DSV_ERR_CUDA: return "CUDA error";
    case DSV_ERR_BAD_INDEX: return "out-of-range block index in a CSR list";
    case DSV_ERR_TIMEOUT: return "a kernel wait ran past its time limit";
    case DSV_ERR_INTERNAL: return "a kernel consistency check failed";
  }
  return "unknown status";
}

dsv_status dsv_set_wait_limit_ns(uint64_t limit_ns) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return DSV_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_mu);
  g_limit_ns[dev] = limit_ns;
  return DSV_OK;
}

dsv_status dsv_get_device_error(dsv_stream_t stream, uint32_t* info) {
  Ctl ctl;
  if (current_ctl(&ctl) != cudaSuccess) return DSV_ERR_CUDA;
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return DSV_ERR_CUDA;
  DeviceErr h{};
  if (cudaMemcpy(&h, ctl.err, sizeof(h), cudaMemcpyDeviceToHost) != cudaSuccess) return DSV_ERR_CUDA;
  if (info) *info = h.info;
  return static_cast<dsv_status>(h.code);
}

dsv_status dsv_selftest_wait_timeout(dsv_stream_t stream) {
  Ctl ctl;
  if (current_ctl(&ctl) != cudaSuccess) return DSV_ERR_CUDA;
  selftest_wait_kernel<<<1, 1, 0, reinterpret_cast<cudaStream_t>(stream)>>>(ctl);
  return from_cuda(cudaGetLastError());
}

dsv_status dsv_clear_device_error(dsv_stream_t stream) {
  Ctl ctl;
  if (current_ctl(&ctl) != cudaSuccess) return DSV_ERR_CUDA;
  return from_cuda(cudaMemsetAsync(ctl.err, 0, sizeof(DeviceErr), reinterpret_cast<cudaStream_t>(stream)));
}

size_t dsv_predict_workspace_bytes(dsv_shape s) {
  if (check_shape(s, true) != DSV_OK || empty(s)) return 0;
  return predict_ws_bytes(s);
}

dsv_status dsv_predict_scores(const void* Q, const void* K, const float* Wq, const float* Wk, dsv_shape s,
                              float* scores, void* workspace, size_t workspace_bytes, dsv_stream_t stream) {
  dsv_status v = check_shape(s, true);
  if (v != DSV_OK) return v;
  if (empty(s)) return DSV_OK;
  if (!Q || !K || !Wq || !Wk || !scores || !workspace) return DSV_ERR_INVALID_ARG;
  if (!al16(Q) || !al16(K) || !al16(Wq) || !al16(Wk) || !al16(scores) || !al256(workspace))
    return DSV_ERR_INVALID_ARG;
  if (workspace_bytes < predict_ws_bytes(s)) return DSV_ERR_INVALID_ARG;
  return from_cuda(launch_predict(Q, K, Wq, Wk, s, scores, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

size_t dsv_predict_max_workspace_bytes(dsv_shape s) {
  if (check_shape(s, true) != DSV_OK || empty(s)) return 0;
  return predict_max_ws_bytes(s);
}

dsv_status dsv_predict_scores_max(const void* Q, const void* K, const float* Wq, const float* Wk, dsv_shape s,
                                  float* scores, void* workspace, size_t workspace_bytes, dsv_stream_t stream) {
  dsv_status v = check_shape(s, true);
  if (v != DSV_OK) return v;
  if (empty(s)) return DSV_OK;
  if (!Q || !K || !Wq || !Wk || !scores || !workspace) return DSV_ERR_INVALID_ARG;
  if (!al16(Q) || !al16(K) || !al16(Wq) || !al16(Wk) || !al16(scores) || !al256(workspace))
    return DSV_ERR_INVALID_ARG;
  if (workspace_bytes < predict_max_ws_bytes(s)) return DSV_ERR_INVALID_ARG;
  Ctl ctl;
  if (current_ctl(&ctl) != cudaSuccess) return DSV_ERR_CUDA;
  return from_cuda(
      launch_predict_max(Q, K, Wq, Wk, s, scores, workspace, ctl, reinterpret_cast<cudaStream_t>(stream)));
}

size_t dsv_topk_workspace_bytes(dsv_shape s) {
  if (check_shape(s, false) != DSV_OK || empty(s)) return 0;
  return topk_ws_bytes(s);
}

dsv_status dsv_topk_blocks(const float* scores, dsv_shape s, const int32_t* k_per_head, int32_t* fwd_ptr,
                           int32_t* fwd_col, int32_t* bwd_ptr, int32_t* bwd_col, void* workspace,
                           size_t workspace_bytes, dsv_stream_t stream) {
  dsv_status v = check_shape(s, false);
  if (v != DSV_OK) return v;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!fwd_ptr || !bwd_ptr) return DSV_ERR_INVALID_ARG;
  if (empty(s)) {
    cudaError_t e = cudaMemsetAsync(fwd_ptr, 0, sizeof(int32_t), st);
    if (e == cudaSuccess) e = cudaMemsetAsync(bwd_ptr, 0, sizeof(int32_t), st);
    return from_cuda(e);
  }
  const int nb = s.N / s.block;
  if (nb > kMaxBlocksPerRow) return DSV_ERR_UNSUPPORTED;
  if (!scores || !k_per_head || !fwd_col || !bwd_col || !workspace) return DSV_ERR_INVALID_ARG;
  if (!al16(scores) || !al16(fwd_ptr) || !al16(fwd_col) || !al16(bwd_ptr) || !al16(bwd_col) || !al256(workspace))
    return DSV_ERR_INVALID_ARG;
  if (workspace_bytes < topk_ws_bytes(s)) return DSV_ERR_INVALID_ARG;
  HeadK hk;
  hk.kpre[0] = 0;
  for (int h = 0; h < s.H; ++h) {
    const int k = k_per_head[h];
    if (k < 1 || k > nb) return DSV_ERR_INVALID_ARG;
    hk.k[h] = k;
    hk.kpre[h + 1] = hk.kpre[h] + k;
  }
  for (int h = s.H; h < kMaxHeads; ++h) {
    hk.k[h] = 0;
    hk.kpre[h + 1] = hk.kpre[h];
  }
  const long long nnz = (long long)s.B * nb * hk.kpre[s.H];
  if (nnz > INT32_MAX) return DSV_ERR_UNSUPPORTED;
  return from_cuda(launch_topk(scores, s, hk, nnz, fwd_ptr, fwd_col, bwd_ptr, bwd_col, workspace, st));
}

size_t dsv_predict_topk_workspace_bytes(dsv_shape s) {
  if (check_shape(s, true) != DSV_OK || empty(s) || s.r > 32) return 0;
  return predict_ws_bytes(s) + split_tf32_bytes(s) + topk_ws_bytes(s);
}

dsv_status dsv_predict_topk_blocks(const void* Q, const void* K, const float* Wq, const float* Wk, dsv_shape s,
                                   const int32_t* k_per_head, int32_t* fwd_ptr, int32_t* fwd_col, int32_t* bwd_ptr,
                                   int32_t* bwd_col, float* scores, void* workspace, size_t workspace_bytes,
                                   dsv_stream_t stream) {
  dsv_status v = check_shape(s, true);
  if (v != DSV_OK) return v;
  if (s.r > 32) return DSV_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!fwd_ptr || !bwd_ptr) return DSV_ERR_INVALID_ARG;
  if (empty(s)) {
    cudaError_t e = cudaMemsetAsync(fwd_ptr, 0, sizeof(int32_t), st);
    if (e == cudaSuccess) e = cudaMemsetAsync(bwd_ptr, 0, sizeof(int32_t), st);
    return from_cuda(e);
  }
  const int nb = s.N / s.block;
  if (nb > kPredictTopkMaxBlocks) return DSV_ERR_UNSUPPORTED;
  if (!Q || !K || !Wq || !Wk || !k_per_head || !fwd_col || !bwd_col || !workspace) return DSV_ERR_INVALID_ARG;
  if (!al16(Q) || !al16(K) || !al16(Wq) || !al16(Wk) || !al16(fwd_ptr) || !al16(fwd_col) || !al16(bwd_ptr) ||
      !al16(bwd_col) || !al256(workspace) || (scores && !al16(scores)))
    return DSV_ERR_INVALID_ARG;
  if (workspace_bytes < predict_ws_bytes(s) + split_tf32_bytes(s) + topk_ws_bytes(s)) return DSV_ERR_INVALID_ARG;
  HeadK hk;
  hk.kpre[0] = 0;
  for (int h = 0; h < s.H; ++h) {
    const int k = k_per_head[h];
    if (k < 1 || k > nb) return DSV_ERR_INVALID_ARG;
    hk.k[h] = k;
    hk.kpre[h + 1] = hk.kpre[h] + k;
  }
  for (int h = s.H; h < kMaxHeads; ++h) {
    hk.k[h] = 0;
    hk.kpre[h + 1] = hk.kpre[h];
  }
  const long long nnz = (long long)s.B * nb * hk.kpre[s.H];
  if (nnz > INT32_MAX) return DSV_ERR_UNSUPPORTED;
  Ctl ctl;
  if (current_ctl(&ctl) != cudaSuccess) return DSV_ERR_CUDA;
  // workspace: pooled vectors | tf32 parts | top-k bitmask and transpose counts
  char* w = static_cast<char*>(workspace);
  const size_t rows = (size_t)s.B * s.H * nb;
  float* qp = reinterpret_cast<float*>(w);
  float* kp = reinterpret_cast<float*>(w + align256(rows * (size_t)s.r * sizeof(float)));
  float* split = reinterpret_cast<float*>(w + predict_ws_bytes(s));
  void* tws = w + predict_ws_bytes(s) + split_tf32_bytes(s);
  const size_t part = align256(rows * 32 * sizeof(float));
  PredictTopkMaps maps;
  const char* sp = reinterpret_cast<const char*>(split);
  if (make_map_f32x32(&maps.qh, sp, (long long)rows, 128) != cudaSuccess ||
      make_map_f32x32(&maps.ql, sp + part, (long long)rows, 128) != cudaSuccess ||
      make_map_f32x32(&maps.kh, sp + 2 * part, (long long)rows, 128) != cudaSuccess ||
      make_map_f32x32(&maps.kl, sp + 3 * part, (long long)rows, 128) != cudaSuccess)
    return DSV_ERR_CUDA;
  ForkRes* fr = nullptr;
  cudaError_t e = fork_res(&fr);
  if (e == cudaSuccess) e = launch_pool_project(Q, K, Wq, Wk, s, qp, kp, st, split, split_part_floats(s));
  if (e == cudaSuccess) e = launch_key_stats(kp, s, split, st);
  if (e != cudaSuccess) return from_cuda(e);
  uint32_t* mask = static_cast<uint32_t*>(tws);
  // The select kernel runs one CTA per SM; the items of a last, partly filled
  // wave go into a launch of their own, and the transposes of the heads done
  // before it run beside it on the side stream.
  const long long tiles = select_tiles(s), bhs = (long long)s.B * s.H, items = bhs * tiles;
  const long long tail = items % fr->nsm, n1 = items - tail, heads1 = n1 / tiles;
  if (tail == 0 || items < 2LL * fr->nsm || heads1 == 0) {
    e = launch_score_select(maps, s, hk, nnz, fwd_ptr, fwd_col, mask, scores, split, ctl, st);
    if (e == cudaSuccess) e = launch_topk_transpose(s, hk, nnz, bwd_ptr, bwd_col, tws, st);
    return from_cuda(e);
  }
  std::lock_guard<std::mutex> lock(g_fork_mu);
  e = launch_score_select(maps, s, hk, nnz, fwd_ptr, fwd_col, mask, scores, split, ctl, st, 0, n1);
  if (e == cudaSuccess) e = cudaEventRecord(fr->main_done, st);
  if (e == cudaSuccess) e = launch_score_select(maps, s, hk, nnz, fwd_ptr, fwd_col, mask, scores, split, ctl, st, n1, items);
  if (e == cudaSuccess) e = cudaStreamWaitEvent(fr->side, fr->main_done, 0);
  if (e == cudaSuccess) e = launch_topk_transpose(s, hk, nnz, bwd_ptr, bwd_col, tws, fr->side, 0, heads1);
  if (e == cudaSuccess) e = cudaEventRecord(fr->side_done, fr->side);
  if (e == cudaSuccess) e = launch_topk_transpose(s, hk, nnz, bwd_ptr, bwd_col, tws, st, heads1, -1);
  if (e == cudaSuccess) e = cudaStreamWaitEvent(st, fr->side_done, 0);
  return from_cuda(e);
}

dsv_status dsv_dispatch_heads(const int32_t* k_per_head, int32_t H, int32_t nb, const float* rho,
                              const float* ratio, int32_t n, int32_t* k_out, int32_t* dense_out) {
  if (!k_per_head || !rho || !ratio || !k_out || !dense_out || H < 1 || nb < 1 || n < 1) return DSV_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n; ++i) {
    if (!(rho[i] > 0.f && rho[i] <= 1.f) || !(ratio[i] > 0.f) || !isfinite(ratio[i])) return DSV_ERR_INVALID_ARG;
    if (i > 0 && !(rho[i] > rho[i - 1])) return DSV_ERR_INVALID_ARG;
  }
  for (int32_t h = 0; h < H; ++h)
    if (k_per_head[h] < 1 || k_per_head[h] > nb) return DSV_ERR_INVALID_ARG;
  for (int32_t h = 0; h < H; ++h) {
    const double x = (double)k_per_head[h] / (double)nb;
    double y;
    if (x <= rho[0]) {
      y = ratio[0];
    } else if (x >= rho[n - 1]) {
      y = ratio[n - 1];
    } else {
      int32_t i = 1;
      while (rho[i] < x) ++i;                     // rho[i-1] < x <= rho[i]
      const double t = (x - rho[i - 1]) / ((double)rho[i] - rho[i - 1]);
      y = ratio[i - 1] + t * ((double)ratio[i] - ratio[i - 1]);
    }
    const int dense = y >= 1.0 ? 1 : 0;
    dense_out[h] = dense;
    k_out[h] = dense ? nb : k_per_head[h];
  }
  return DSV_OK;
}

size_t dsv_topk_mass_workspace_bytes(dsv_shape s) {
  if (check_shape(s, false) != DSV_OK || empty(s)) return 0;
  return topk_mass_ws_bytes(s);
}

dsv_status dsv_topk_mass_blocks(const float* scores, dsv_shape s, float tau, float temperature, int32_t kmin,
                                int32_t kmax, int32_t* fwd_ptr, int32_t* fwd_col, int32_t* bwd_ptr, int32_t* bwd_col,
                                size_t col_capacity, void* workspace, size_t workspace_bytes, dsv_stream_t stream) {
  dsv_status v = check_shape(s, false);
  if (v != DSV_OK) return v;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!fwd_ptr || !bwd_ptr) return DSV_ERR_INVALID_ARG;
  if (!(tau > 0.f && tau <= 1.f) || !(temperature > 0.f) || !isfinite(temperature)) return DSV_ERR_INVALID_ARG;
  if (empty(s)) {
    cudaError_t e = cudaMemsetAsync(fwd_ptr, 0, sizeof(int32_t), st);
    if (e == cudaSuccess) e = cudaMemsetAsync(bwd_ptr, 0, sizeof(int32_t), st);
    return from_cuda(e);
  }
  const int nb = s.N / s.block;
  if (nb > kMaxBlocksPerRow) return DSV_ERR_UNSUPPORTED;
  if (kmin < 1 || kmin > kmax || kmax > nb) return DSV_ERR_INVALID_ARG;
  if (!scores || !fwd_col || !bwd_col || !workspace) return DSV_ERR_INVALID_ARG;
  if (!al16(scores) || !al16(fwd_ptr) || !al16(fwd_col) || !al16(bwd_ptr) || !al16(bwd_col) || !al256(workspace))
    return DSV_ERR_INVALID_ARG;
  if (workspace_bytes < topk_mass_ws_bytes(s)) return DSV_ERR_INVALID_ARG;
  const long long cap = (long long)s.B * s.H * nb * kmax;   // every row at most kmax entries
  if (cap > INT32_MAX) return DSV_ERR_UNSUPPORTED;
  if ((long long)col_capacity < cap) return DSV_ERR_INVALID_ARG;
  return from_cuda(
      launch_topk_mass(scores, s, tau, temperature, kmin, kmax, fwd_ptr, fwd_col, bwd_ptr, bwd_col, workspace, st));
}

dsv_status dsv_sparse_attn_fwd(const void* Q, const void* K, const void* V, dsv_shape s, const int32_t* fwd_ptr,
                               const int32_t* fwd_col, float softmax_scale, void* O, float* lse,
                               dsv_stream_t stream) {
  dsv_status v = check_shape(s, false);
  if (v != DSV_OK) return v;
  if (empty(s)) return DSV_OK;
  if (!Q || !K || !V || !fwd_ptr || !fwd_col || !O || !lse) return DSV_ERR_INVALID_ARG;
  if (!al16(Q) || !al16(K) || !al16(V) || !al16(O) || !al16(lse)) return DSV_ERR_INVALID_ARG;
  Ctl ctl;
  if (current_ctl(&ctl) != cudaSuccess) return DSV_ERR_CUDA;
  const long long rows = (long long)s.B * s.H * s.N;
  CUtensorMap tq, tk, tv;
  if (make_map(&tq, Q, rows, s.d, s.block) != cudaSuccess || make_map(&tk, K, rows, s.d, s.block) != cudaSuccess ||
      make_map(&tv, V, rows, s.d, s.block) != cudaSuccess)
    return DSV_ERR_CUDA;
  return from_cuda(launch_attn_fwd(tq, tk, tv, s, fwd_ptr, fwd_col, resolve_scale(s, softmax_scale), O, lse, ctl,
                                   reinterpret_cast<cudaStream_t>(stream)));
}

size_t dsv_attn_bwd_workspace_bytes(dsv_shape s) {
  if (check_shape(s, false) != DSV_OK || empty(s)) return 0;
  return attn_bwd_ws_bytes(s);
}

dsv_status dsv_sparse_attn_bwd(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                               const float* lse, dsv_shape s, const int32_t* fwd_ptr, const int32_t* fwd_col,
                               const int32_t* bwd_ptr, const int32_t* bwd_col, float softmax_scale, void* dQ,
                               void* dK, void* dV, void* workspace, size_t workspace_bytes, dsv_stream_t stream) {
  dsv_status v = check_shape(s, false);
  if (v != DSV_OK) return v;
  if (empty(s)) return DSV_OK;
  if (!Q || !K || !V || !O || !dO || !lse || !fwd_ptr || !fwd_col || !bwd_ptr || !bwd_col || !dQ || !dK || !dV ||
      !workspace)
    return DSV_ERR_INVALID_ARG;
  if (!al16(Q) || !al16(K) || !al16(V) || !al16(O) || !al16(dO) || !al16(lse) || !al16(dQ) || !al16(dK) ||
      !al16(dV) || !al256(workspace))
    return DSV_ERR_INVALID_ARG;
  if (workspace_bytes < attn_bwd_ws_bytes(s)) return DSV_ERR_INVALID_ARG;
  Ctl ctl;
  if (current_ctl(&ctl) != cudaSuccess) return DSV_ERR_CUDA;
  const long long rows = (long long)s.B * s.H * s.N;
  CUtensorMap tq, tk, tv, tdo;
  if (make_map(&tq, Q, rows, s.d, s.block) != cudaSuccess || make_map(&tk, K, rows, s.d, s.block) != cudaSuccess ||
      make_map(&tv, V, rows, s.d, s.block) != cudaSuccess || make_map(&tdo, dO, rows, s.d, s.block) != cudaSuccess)
    return DSV_ERR_CUDA;
  return from_cuda(launch_attn_bwd(Q, tq, tk, tv, tdo, O, dO, lse, s, fwd_ptr, fwd_col, bwd_ptr, bwd_col,
                                   resolve_scale(s, softmax_scale), dQ, dK, dV, workspace, ctl,
                                   reinterpret_cast<cudaStream_t>(stream)));
}

dsv_status dsv_cube_permute(const void* src, void* dst, dsv_shape s, int T, int Hl, int Wl, int ct, int cy, int cx,
                            int inverse, dsv_stream_t stream) {
  dsv_status v = check_shape(s, false);
  if (v != DSV_OK) return v;
  if (T <= 0 || Hl <= 0 || Wl <= 0 || ct <= 0 || cy <= 0 || cx <= 0) return DSV_ERR_INVALID_ARG;
  if ((long long)T * Hl * Wl != s.N || ct * cy * cx != s.block) return DSV_ERR_INVALID_ARG;
  if (T % ct != 0 || Hl % cy != 0 || Wl % cx != 0) return DSV_ERR_INVALID_ARG;
  if (inverse != 0 && inverse != 1) return DSV_ERR_INVALID_ARG;
  if (empty(s)) return DSV_OK;
  if (!src || !dst || !al16(src) || !al16(dst)) return DSV_ERR_INVALID_ARG;
  const size_t bytes = (size_t)s.B * s.H * s.N * s.d * 2;
  const char* a = static_cast<const char*>(src);
  const char* b = static_cast<const char*>(dst);
  if (a < b + bytes && b < a + bytes) return DSV_ERR_INVALID_ARG;   // overlapping buffers
  return from_cuda(launch_cube_permute(src, dst, s, T, Hl, Wl, ct, cy, cx, inverse,
                                       reinterpret_cast<cudaStream_t>(stream)));
}

dsv_status dsv_attn_bwd_preprocess(const void* O, const void* dO, const float* lse, dsv_shape s, void* workspace,
                                   size_t workspace_bytes, dsv_stream_t stream) {
  dsv_status v = check_shape(s, false);
  if (v != DSV_OK) return v;
  if (empty(s)) return DSV_OK;
  if (!O || !dO || !lse || !workspace) return DSV_ERR_INVALID_ARG;
  if (!al16(O) || !al16(dO) || !al16(lse) || !al256(workspace)) return DSV_ERR_INVALID_ARG;
  if (workspace_bytes < attn_bwd_ws_bytes(s)) return DSV_ERR_INVALID_ARG;
  return from_cuda(launch_attn_bwd_pre(O, dO, lse, s, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

dsv_status dsv_attn_bwd_dkdv(const void* Q, const void* K, const void* V, const void* dO, dsv_shape s,
                             const int32_t* bwd_ptr, const int32_t* bwd_col, float softmax_scale, void* dK, void* dV,
                             void* workspace, size_t workspace_bytes, dsv_stream_t stream) {
  dsv_status v = check_shape(s, false);
  if (v != DSV_OK) return v;
  if (empty(s)) return DSV_OK;
  if (!Q || !K || !V || !dO || !bwd_ptr || !bwd_col || !dK || !dV || !workspace) return DSV_ERR_INVALID_ARG;
  if (!al16(Q) || !al16(K) || !al16(V) || !al16(dO) || !al16(dK) || !al16(dV) || !al256(workspace))
    return DSV_ERR_INVALID_ARG;
  if (workspace_bytes < attn_bwd_ws_bytes(s)) return DSV_ERR_INVALID_ARG;
  Ctl ctl;
  if (current_ctl(&ctl) != cudaSuccess) return DSV_ERR_CUDA;
  const long long rows = (long long)s.B * s.H * s.N;
  CUtensorMap tq, tk, tv, tdo;
  if (make_map(&tq, Q, rows, s.d, s.block) != cudaSuccess || make_map(&tk, K, rows, s.d, s.block) != cudaSuccess ||
      make_map(&tv, V, rows, s.d, s.block) != cudaSuccess || make_map(&tdo, dO, rows, s.d, s.block) != cudaSuccess)
    return DSV_ERR_CUDA;
  return from_cuda(launch_attn_bwd_kv(tq, tk, tv, tdo, s, bwd_ptr, bwd_col, resolve_scale(s, softmax_scale), dK, dV,
                                      workspace, ctl, reinterpret_cast<cudaStream_t>(stream)));
}

dsv_status dsv_attn_bwd_dq(const void* Q, const void* K, const void* V, const void* dO, dsv_shape s,
                           const int32_t* fwd_ptr, const int32_t* fwd_col, float softmax_scale, void* dQ,
                           const void* workspace, size_t workspace_bytes, dsv_stream_t stream) {
  dsv_status v = check_shape(s, false);
  if (v != DSV_OK) return v;
  if (empty(s)) return DSV_OK;
  if (!Q || !K || !V || !dO || !fwd_ptr || !fwd_col || !dQ || !workspace) return DSV_ERR_INVALID_ARG;
  if (!al16(Q) || !al16(K) || !al16(V) || !al16(dO) || !al16(dQ) || !al256(workspace)) return DSV_ERR_INVALID_ARG;
  if (workspace_bytes < attn_bwd_ws_bytes(s)) return DSV_ERR_INVALID_ARG;
  Ctl ctl;
  if (current_ctl(&ctl) != cudaSuccess) return DSV_ERR_CUDA;
  const long long rows = (long long)s.B * s.H * s.N;
  CUtensorMap tq, tk, tv, tdo;
  if (make_map(&tq, Q, rows, s.d, s.block) != cudaSuccess || make_map(&tk, K, rows, s.d, s.block) != cudaSuccess ||
      make_map(&tv, V, rows, s.d, s.block) != cudaSuccess || make_map(&tdo, dO, rows, s.d, s.block) != cudaSuccess)
    return DSV_ERR_CUDA;
  return from_cuda(launch_attn_bwd_q(tq, tk, tv, tdo, s, fwd_ptr, fwd_col, resolve_scale(s, softmax_scale), dQ,
                                     workspace, ctl, reinterpret_cast<cudaStream_t>(stream)));
}

size_t dsv_packed_attn_fwd_workspace_bytes(dsv_packed p) {
  if (check_packed(p) != DSV_OK || no_queries(p) || no_keys(p)) return 0;
  return packed_fwd_ws_bytes(p);
}

dsv_status dsv_packed_attn_fwd(dsv_view Q, dsv_view K, dsv_view V, dsv_packed p, const int32_t* q_ptr,
                               const int32_t* k_ptr, int32_t causal, float softmax_scale, dsv_view O, float* lse,
                               void* workspace, size_t workspace_bytes, dsv_stream_t stream) {
  dsv_status v = check_packed(p);
  if (v != DSV_OK) return v;
  if (causal != 0 && causal != 1) return DSV_ERR_INVALID_ARG;
  if (no_queries(p)) return DSV_OK;
  if (!q_ptr || !k_ptr || !lse || !al4(q_ptr) || !al4(k_ptr) || !al4(lse)) return DSV_ERR_INVALID_ARG;
  if (!view_ok(Q, p.H, p.Tq, p.d, false) || !view_ok(O, p.H, p.Tq, p.d, true)) return DSV_ERR_INVALID_ARG;
  if (!no_keys(p) && (!view_ok(K, p.Hkv, p.Tk, p.d, false) || !view_ok(V, p.Hkv, p.Tk, p.d, false)))
    return DSV_ERR_INVALID_ARG;
  if (O.ptr == Q.ptr || O.ptr == K.ptr || O.ptr == V.ptr) return DSV_ERR_INVALID_ARG;
  const size_t need = dsv_packed_attn_fwd_workspace_bytes(p);
  if (need > 0 && (!workspace || !al256(workspace) || workspace_bytes < need)) return DSV_ERR_INVALID_ARG;
  Ctl ctl;
  if (current_ctl(&ctl) != cudaSuccess) return DSV_ERR_CUDA;
  widen_wait(&ctl, p);
  const int group = p.H / p.Hkv;
  CUtensorMap tq, tk, tv;
  if (make_map_view(&tq, Q, p.H, p.Tq, p.d, group, 128 / group) != cudaSuccess) return DSV_ERR_CUDA;
  if (no_keys(p)) {
    tk = tv = tq;                          // never loaded: no row has a key tile
  } else if (make_map_view(&tk, K, p.Hkv, p.Tk, p.d, 1, 128) != cudaSuccess ||
             make_map_view(&tv, V, p.Hkv, p.Tk, p.d, 1, 128) != cudaSuccess) {
    return DSV_ERR_CUDA;
  }
  return from_cuda(launch_packed_fwd(tq, tk, tv, p, q_ptr, k_ptr, causal, packed_scale(p.d, softmax_scale), O, lse,
                                     workspace, ctl, reinterpret_cast<cudaStream_t>(stream)));
}

size_t dsv_packed_attn_bwd_workspace_bytes(dsv_packed p) {
  if (check_packed(p) != DSV_OK || no_queries(p)) return 0;
  return packed_bwd_ws_bytes(p);
}

dsv_status dsv_packed_attn_bwd(dsv_view Q, dsv_view K, dsv_view V, dsv_view O, dsv_view dO, const float* lse,
                               dsv_packed p, const int32_t* q_ptr, const int32_t* k_ptr, int32_t causal,
                               float softmax_scale, dsv_view dQ, dsv_view dK, dsv_view dV, void* workspace,
                               size_t workspace_bytes, dsv_stream_t stream) {
  dsv_status v = check_packed(p);
  if (v != DSV_OK) return v;
  if (causal != 0 && causal != 1) return DSV_ERR_INVALID_ARG;
  // keys without any query head: their gradients are zeros that no kernel here would write
  if (p.S > 0 && p.H == 0 && p.Hkv > 0 && p.Tk > 0) return DSV_ERR_INVALID_ARG;
  const bool nq = no_queries(p), nk = no_keys(p);
  if (nq && nk) return DSV_OK;
  if (!q_ptr || !k_ptr || !al4(q_ptr) || !al4(k_ptr)) return DSV_ERR_INVALID_ARG;
  if (!nq) {
    if (!lse || !al4(lse)) return DSV_ERR_INVALID_ARG;
    if (!view_ok(Q, p.H, p.Tq, p.d, false) || !view_ok(O, p.H, p.Tq, p.d, false) ||
        !view_ok(dO, p.H, p.Tq, p.d, false) || !view_ok(dQ, p.H, p.Tq, p.d, true))
      return DSV_ERR_INVALID_ARG;
  }
  if (!nk && (!view_ok(K, p.Hkv, p.Tk, p.d, false) || !view_ok(V, p.Hkv, p.Tk, p.d, false) ||
              !view_ok(dK, p.Hkv, p.Tk, p.d, true) || !view_ok(dV, p.Hkv, p.Tk, p.d, true)))
    return DSV_ERR_INVALID_ARG;
  const void* const in[5] = {Q.ptr, K.ptr, V.ptr, O.ptr, dO.ptr};
  const void* const res[3] = {dQ.ptr, dK.ptr, dV.ptr};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 5; ++j)
      if (res[i] && res[i] == in[j]) return DSV_ERR_INVALID_ARG;
    if (res[i] && res[i] == res[(i + 1) % 3]) return DSV_ERR_INVALID_ARG;
  }
  const size_t need = dsv_packed_attn_bwd_workspace_bytes(p);
  if (need > 0 && (!workspace || !al256(workspace) || workspace_bytes < need)) return DSV_ERR_INVALID_ARG;
  Ctl ctl;
  if (current_ctl(&ctl) != cudaSuccess) return DSV_ERR_CUDA;
  widen_wait(&ctl, p);
  const int group = p.H / p.Hkv;
  PackedMaps m;
  if (!nq && (make_map_view(&m.Q, Q, p.H, p.Tq, p.d, group, 128 / group) != cudaSuccess ||
              make_map_view(&m.dO, dO, p.H, p.Tq, p.d, group, 128 / group) != cudaSuccess))
    return DSV_ERR_CUDA;
  if (!nk && (make_map_view(&m.K, K, p.Hkv, p.Tk, p.d, 1, 128) != cudaSuccess ||
              make_map_view(&m.V, V, p.Hkv, p.Tk, p.d, 1, 128) != cudaSuccess))
    return DSV_ERR_CUDA;
  // a side without tokens is never loaded
  if (nq) m.Q = m.dO = m.K;
  if (nk) m.K = m.V = m.Q;
  return from_cuda(launch_packed_bwd(m, p, q_ptr, k_ptr, causal, packed_scale(p.d, softmax_scale), O, dO, lse, dQ, dK,
                                     dV, workspace, ctl, reinterpret_cast<cudaStream_t>(stream)));
}

dsv_status dsv_rope_axes_fwd(dsv_view x, const int32_t* pos, int64_t pos_batch_stride, dsv_rope r,
                             const float* weight, float eps, dsv_view y, dsv_stream_t stream) {
  dsv_status v = check_rope(r);
  if (v != DSV_OK) return v;
  if (weight && (!(eps > 0.f) || !isfinite(eps) || !al4(weight))) return DSV_ERR_INVALID_ARG;
  if (empty_rope(r)) return DSV_OK;
  if (!pos || !al4(pos) || pos_batch_stride < 0) return DSV_ERR_INVALID_ARG;
  if (!view4_ok(x, r.B, r.H, r.N, r.d, false) || !view4_ok(y, r.B, r.H, r.N, r.d, true)) return DSV_ERR_INVALID_ARG;
  if (!same_or_apart(x, y, r.B, r.H, r.N)) return DSV_ERR_INVALID_ARG;
  return from_cuda(launch_rope_fwd(x, pos, pos_batch_stride, r, weight, eps, y, reinterpret_cast<cudaStream_t>(stream)));
}

size_t dsv_rope_axes_bwd_workspace_bytes(dsv_rope r) {
  if (check_rope(r) != DSV_OK || empty_rope(r)) return 0;
  return rope_bwd_ws_bytes(r);
}

dsv_status dsv_rope_axes_bwd(dsv_view dy, dsv_view x, const int32_t* pos, int64_t pos_batch_stride, dsv_rope r,
                             const float* weight, float eps, dsv_view dx, float* dweight, void* workspace,
                             size_t workspace_bytes, dsv_stream_t stream) {
  dsv_status v = check_rope(r);
  if (v != DSV_OK) return v;
  if (weight && (!(eps > 0.f) || !isfinite(eps) || !al4(weight) || !dweight || !al4(dweight)))
    return DSV_ERR_INVALID_ARG;
  if (empty_rope(r)) {                     // no rows: the sum over them is zero
    if (!weight) return DSV_OK;
    return from_cuda(cudaMemsetAsync(dweight, 0, (size_t)r.d * sizeof(float), reinterpret_cast<cudaStream_t>(stream)));
  }
  if (!pos || !al4(pos) || pos_batch_stride < 0) return DSV_ERR_INVALID_ARG;
  if (!view4_ok(dy, r.B, r.H, r.N, r.d, false) || !view4_ok(dx, r.B, r.H, r.N, r.d, true)) return DSV_ERR_INVALID_ARG;
  if (!same_or_apart(dy, dx, r.B, r.H, r.N)) return DSV_ERR_INVALID_ARG;
  if (weight) {
    if (!view4_ok(x, r.B, r.H, r.N, r.d, false) || !same_or_apart(x, dx, r.B, r.H, r.N)) return DSV_ERR_INVALID_ARG;
    if (!workspace || !al256(workspace) || workspace_bytes < rope_bwd_ws_bytes(r)) return DSV_ERR_INVALID_ARG;
  }
  return from_cuda(launch_rope_bwd(dy, x, pos, pos_batch_stride, r, weight, eps, dx, dweight, workspace,
                                   reinterpret_cast<cudaStream_t>(stream)));
}

dsv_status dsv_layer_norm_fwd(dsv_rows x, dsv_norm p, const int32_t* seq_ptr, const float* weight, const float* bias,
                              dsv_rows y, float* stats, dsv_stream_t stream) {
  dsv_status v = check_norm(p);
  if (v != DSV_OK) return v;
  if (!(p.eps > 0.f) || !isfinite(p.eps) || !al4(seq_ptr) || !al4(weight) || !al4(bias)) return DSV_ERR_INVALID_ARG;
  if ((bias && !weight) || (!seq_ptr && (p.S == 0 || p.T % p.S != 0))) return DSV_ERR_INVALID_ARG;
  if (p.T == 0 || p.S == 0) return DSV_OK;
  if (!real_type(x) || y.type != DSV_BF16 || !stats || !al4(stats)) return DSV_ERR_INVALID_ARG;
  if (!rows_ok(x, p.T, p.C) || !rows_ok(y, p.T, p.C) || !same_or_apart(x, y, p.T)) return DSV_ERR_INVALID_ARG;
  Ctl ctl;
  if (current_ctl(&ctl) != cudaSuccess) return DSV_ERR_CUDA;
  return from_cuda(
      launch_norm_fwd(x, p, seq_ptr, weight, bias, y, stats, ctl, reinterpret_cast<cudaStream_t>(stream)));
}

size_t dsv_layer_norm_bwd_workspace_bytes(dsv_norm p) {
  if (check_norm(p) != DSV_OK || p.T == 0 || p.S == 0) return 0;
  return norm_bwd_ws_bytes(p);
}

dsv_status dsv_layer_norm_bwd(dsv_rows dy, dsv_rows x, const float* stats, dsv_norm p, const int32_t* seq_ptr,
                              const float* weight, dsv_rows dx, float* dweight, float* dbias, void* workspace,
                              size_t workspace_bytes, dsv_stream_t stream) {
  dsv_status v = check_norm(p);
  if (v != DSV_OK) return v;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!al4(seq_ptr) || !al4(weight) || !al4(dweight) || !al4(dbias)) return DSV_ERR_INVALID_ARG;
  if ((weight && (!dweight || !dbias)) || (!seq_ptr && (p.S == 0 || p.T % p.S != 0))) return DSV_ERR_INVALID_ARG;
  if (!weight) dweight = dbias = nullptr;
  if (p.T == 0 || p.S == 0) {              // no rows: the sums over them are zero
    if (!weight || p.S == 0) return DSV_OK;
    const size_t bytes = (size_t)p.S * p.C * sizeof(float);
    cudaError_t e = cudaMemsetAsync(dweight, 0, bytes, st);
    if (e == cudaSuccess) e = cudaMemsetAsync(dbias, 0, bytes, st);
    return from_cuda(e);
  }
  if (!real_type(x) || dx.type != x.type || dy.type != DSV_BF16 || !stats || !al4(stats)) return DSV_ERR_INVALID_ARG;
  if (!rows_ok(x, p.T, p.C) || !rows_ok(dy, p.T, p.C) || !rows_ok(dx, p.T, p.C)) return DSV_ERR_INVALID_ARG;
  if (!same_or_apart(x, dx, p.T) || !same_or_apart(dy, dx, p.T)) return DSV_ERR_INVALID_ARG;
  if (weight && (!workspace || !al256(workspace) || workspace_bytes < norm_bwd_ws_bytes(p))) return DSV_ERR_INVALID_ARG;
  Ctl ctl;
  if (current_ctl(&ctl) != cudaSuccess) return DSV_ERR_CUDA;
  return from_cuda(launch_norm_bwd(dy, x, stats, p, seq_ptr, weight, dx, dweight, dbias, workspace, ctl, st));
}

dsv_status dsv_quantize_fp8(dsv_rows x, int32_t R, int32_t C, int32_t rows, dsv_rows q, float* scale, dsv_rows qt,
                            float* scale_t, dsv_stream_t stream) {
  if (R < 0 || C < 0 || (rows != 1 && rows != 128)) return DSV_ERR_INVALID_ARG;
  if (R >= INT32_MAX - 128 || C >= INT32_MAX - 128) return DSV_ERR_UNSUPPORTED;
  if (((long long)R + 127) / 128 * (((long long)C + 127) / 128) > INT32_MAX) return DSV_ERR_UNSUPPORTED;
  if (R == 0 || C == 0) return DSV_OK;
  if (!real_type(x) || !rows_ok(x, R, C) || !fp8_ok(q, R, C) || !scale || !al4(scale)) return DSV_ERR_INVALID_ARG;
  if (qt.ptr && (!fp8_ok(qt, C, R) || qt.type != q.type || !scale_t || !al4(scale_t) || qt.ptr == q.ptr))
    return DSV_ERR_INVALID_ARG;
  if (q.ptr == x.ptr || qt.ptr == x.ptr) return DSV_ERR_INVALID_ARG;
  return from_cuda(launch_quantize(x, R, C, rows, q, scale, qt, scale_t, reinterpret_cast<cudaStream_t>(stream)));
}

dsv_status dsv_matmul_fp8(dsv_rows a, const float* a_scale, dsv_rows b, const float* b_scale, dsv_matmul p, dsv_rows c,
                          dsv_stream_t stream) {
  if (p.M < 0 || p.N < 0 || p.K < 0) return DSV_ERR_INVALID_ARG;
  if ((p.a_rows != 1 && p.a_rows != 128) || (p.b_rows != 1 && p.b_rows != 128)) return DSV_ERR_INVALID_ARG;
  if (p.accumulate != 0 && p.accumulate != 1) return DSV_ERR_INVALID_ARG;
  const int most = INT32_MAX - 256;
  if (p.M > most || p.N > most || p.K > most) return DSV_ERR_UNSUPPORTED;
  if (((long long)p.M + 127) / 128 * (((long long)p.N + 127) / 128) > INT32_MAX) return DSV_ERR_UNSUPPORTED;
  if (p.M == 0 || p.N == 0) return DSV_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!real_type(c) || !rows_ok(c, p.M, p.N) || (p.accumulate && c.type != DSV_F32)) return DSV_ERR_INVALID_ARG;
  if (p.K == 0) {                          // the sum over nothing
    if (p.accumulate) return DSV_OK;
    const size_t size = (size_t)size_of(c.type), width = (size_t)p.N * size;
    return from_cuda(cudaMemset2DAsync(c.ptr, p.M > 1 ? (size_t)c.stride * size : width, 0, width, (size_t)p.M, st));
  }
  if (!fp8_ok(a, p.M, p.K) || !fp8_ok(b, p.N, p.K)) return DSV_ERR_INVALID_ARG;
  if (!a_scale || !b_scale || !al4(a_scale) || !al4(b_scale)) return DSV_ERR_INVALID_ARG;
  if (c.ptr == a.ptr || c.ptr == b.ptr) return DSV_ERR_INVALID_ARG;
  Ctl ctl;
  if (current_ctl(&ctl) != cudaSuccess) return DSV_ERR_CUDA;
  CUtensorMap ta, tb, tc;
  int box_a, box_b;
  matmul_boxes(p, &box_a, &box_b);
  if (make_map_rows(&ta, a, p.M, p.K, box_a) != cudaSuccess || make_map_rows(&tb, b, p.N, p.K, box_b) != cudaSuccess)
    return DSV_ERR_CUDA;
  const bool copies = !p.accumulate && al16(c.ptr) && (p.M == 1 || c.stride * size_of(c.type) % 16 == 0);
  if (copies && make_map_rows(&tc, c, p.M, p.N, 32) != cudaSuccess) return DSV_ERR_CUDA;
  return from_cuda(launch_matmul_fp8(ta, tb, copies ? &tc : nullptr, p, a.type == DSV_E5M2, b.type == DSV_E5M2, a_scale,
                                     b_scale, c, ctl, st));
}

}  // extern "C"
