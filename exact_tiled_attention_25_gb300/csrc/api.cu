// The C ABI: argument validation, device checks, tensor maps, status word.
#include <cmath>
#include <cstring>
#include <mutex>
#include <string>

#include "common.h"
#include "rope.h"
#include "sm103_prims.cuh"

namespace attn {

namespace {

thread_local std::string g_last_error;

// One status word per device; kernels record the first internal error here.
__device__ int g_device_status;

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    cudaDriverEntryPointQueryResult q;
    void* f = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
  });
  return fn;
}

constexpr int kMaxDevices = 64;
int g_arch_ok[kMaxDevices];   // 0 unknown, 1 ok, 2 wrong arch (a property of the device)
std::mutex g_dev_mutex;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Pure argument checks: no CUDA call is made here, so they also run on a
// machine without a GPU.
attn_status_t check_shape(int B, int H, int N, int d, int causal) {
  if (B < 1 || H < 1 || N < 1) return fail(ATTN_ERR_INVALID_ARG, "B, H and N must be >= 1");
  if (d != 64 && d != 128 && d != 256)
    return fail(ATTN_ERR_INVALID_ARG, "d must be 64, 128 or 256");
  if (causal != 0 && causal != 1) return fail(ATTN_ERR_INVALID_ARG, "causal must be 0 or 1");
  const double elems = static_cast<double>(B) * H * N * d;
  if (elems >= 2147483648.0) return fail(ATTN_ERR_INVALID_ARG, "B*H*N*d must be < 2^31");
  return ATTN_OK;
}

attn_status_t check_heads(int H, int H_kv) {
  if (H_kv < 1 || H_kv > H || H % H_kv != 0)
    return fail(ATTN_ERR_INVALID_ARG, "H_kv must divide H (1 <= H_kv <= H)");
  return ATTN_OK;
}

// A packed batch: B sequences, the longest max_seqlen tokens, total tokens.
attn_status_t check_packed(int B, int max_seqlen, int total, int H, int d, int causal) {
  if (B < 1 || H < 1 || max_seqlen < 1 || total < 1)
    return fail(ATTN_ERR_INVALID_ARG, "B, H, max_seqlen and total must be >= 1");
  if (d != 64 && d != 128 && d != 256)
    return fail(ATTN_ERR_INVALID_ARG, "d must be 64, 128 or 256");
  if (causal != 0 && causal != 1) return fail(ATTN_ERR_INVALID_ARG, "causal must be 0 or 1");
  if (static_cast<double>(total) * H * d >= 2147483648.0)
    return fail(ATTN_ERR_INVALID_ARG, "total*H*d must be < 2^31");
  if (static_cast<double>(B) * H * (max_seqlen + 127) / 128 * 128 >= 2147483648.0)
    return fail(ATTN_ERR_INVALID_ARG, "B*H*max_seqlen too large");
  return ATTN_OK;
}

attn_status_t check_ptrs(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs) {
    if (p == nullptr) return fail(ATTN_ERR_INVALID_ARG, "null tensor pointer");
    if (!aligned16(p)) return fail(ATTN_ERR_INVALID_ARG, "tensor pointer not 16-byte aligned");
  }
  return ATTN_OK;
}

attn_status_t check_dtype(attn_dtype_t dtype) {
  if (dtype != ATTN_BF16 && dtype != ATTN_FP16)
    return fail(ATTN_ERR_INVALID_ARG, "dtype must be ATTN_BF16 or ATTN_FP16");
  return ATTN_OK;
}

attn_status_t check_ints(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (p == nullptr || (reinterpret_cast<uintptr_t>(p) & 3u) != 0)
      return fail(ATTN_ERR_INVALID_ARG, "integer arrays must be non-null and 4-byte aligned");
  return ATTN_OK;
}

// Rows of 16-bit values: heads >= 1 of d values, strides in elements that keep
// every row 16-byte aligned.  An output's strides are positive.
attn_status_t check_row_strides(std::initializer_list<long long> strides, bool output) {
  for (long long x : strides)
    if (x < (output ? 1 : 0) || (x & 7) != 0)
      return fail(ATTN_ERR_INVALID_ARG,
                  "strides must be non-negative (of outputs: positive) multiples of 8 elements");
  return ATTN_OK;
}

attn_status_t check_rope(const float* cos, const float* sin, int d, int rot_dim, int max_pos, int interleaved) {
  if (rot_dim < 16 || rot_dim > d || rot_dim % 16 != 0)
    return fail(ATTN_ERR_INVALID_ARG, "rot_dim must be a multiple of 16 in [16, d]");
  if (max_pos < 1) return fail(ATTN_ERR_INVALID_ARG, "the rotary tables need max_pos >= 1 rows");
  if (interleaved != 0 && interleaved != 1)
    return fail(ATTN_ERR_INVALID_ARG, "interleaved must be 0 or 1");
  return check_ptrs({cos, sin});
}

attn_status_t check_page_size(int page_size, int least) {
  if (page_size < least || page_size > 65536 || (page_size & (page_size - 1)) != 0)
    return fail(ATTN_ERR_INVALID_ARG,
                "page_size must be a power of two in [" + std::to_string(least) + ", 65536]");
  return ATTN_OK;
}

attn_status_t check_scale(float s) {
  if (!(s > 0.f) || !std::isfinite(s))
    return fail(ATTN_ERR_INVALID_ARG, "softmax_scale must be positive and finite");
  return ATTN_OK;
}

}  // namespace

// Device check: compute capability 10.3, cached per device ordinal (the
// architecture does not change with the context).
attn_status_t check_device() {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail_cuda(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(ATTN_ERR_CUDA, "device ordinal out of range");
  std::lock_guard<std::mutex> lock(g_dev_mutex);
  if (g_arch_ok[dev] == 0) {
    int major = 0, minor = 0;
    e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (e != cudaSuccess) return fail_cuda(e, "cudaDeviceGetAttribute");
    e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    if (e != cudaSuccess) return fail_cuda(e, "cudaDeviceGetAttribute");
    g_arch_ok[dev] = (major == 10 && minor == 3) ? 1 : 2;
  }
  if (g_arch_ok[dev] != 1)
    return fail(ATTN_ERR_ARCH, "this library runs on compute capability 10.3 (GB300) only");
  return ATTN_OK;
}

attn_status_t fail(attn_status_t code, const std::string& msg) {
  g_last_error = msg;
  return code;
}

attn_status_t fail_cuda(cudaError_t err, const char* what) {
  g_last_error = std::string(what) + ": " + cudaGetErrorName(err) + " (" +
                 cudaGetErrorString(err) + ")";
  return ATTN_ERR_CUDA;
}

// Looked up on every call rather than cached per device ordinal, so the
// address always belongs to the current context (a cached one would go stale
// after cudaDeviceReset or under another context on the same device).
int* device_status_word() {
  void* p = nullptr;
  if (cudaGetSymbolAddress(&p, g_device_status) != cudaSuccess) return nullptr;
  return static_cast<int*>(p);
}

attn_status_t make_tmap_3d(CUtensorMap* map, const void* base, int elem_bytes, uint64_t inner,
                           uint64_t rows, uint64_t planes, uint32_t box_inner,
                           uint32_t box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  cuuint64_t dims[3] = {inner, rows, planes};
  cuuint64_t strides[2] = {inner * elem_bytes, inner * rows * elem_bytes};
  cuuint32_t box[3] = {box_inner, box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUtensorMapDataType dt = elem_bytes == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                           : elem_bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16
                                             : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  CUresult r = enc(map, dt, 3, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled failed with CUresult " + std::to_string(r));
  return ATTN_OK;
}

attn_status_t make_tmap_fp4(CUtensorMap* map, const void* base, uint64_t rows, uint64_t heads, uint64_t pages,
                            uint64_t row_bytes, uint64_t head_bytes, uint64_t page_bytes, uint32_t box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  cuuint64_t dims[4] = {128, rows, heads, pages};
  cuuint64_t strides[3] = {row_bytes, head_bytes, page_bytes};
  cuuint32_t box[4] = {128, box_rows, 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 4, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled (4-bit) failed with CUresult " + std::to_string(r));
  return ATTN_OK;
}

attn_status_t make_tmap_4d(CUtensorMap* map, const void* base, int elem_bytes, uint64_t inner,
                           uint64_t rows, uint64_t heads, uint64_t batches, uint64_t row_bytes,
                           uint64_t head_bytes, uint64_t batch_bytes, uint32_t box_inner,
                           uint32_t box_rows, uint32_t box_heads) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  cuuint64_t dims[4] = {inner, rows, heads, batches};
  cuuint64_t strides[3] = {row_bytes, head_bytes, batch_bytes};
  cuuint32_t box[4] = {box_inner, box_rows, box_heads, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUtensorMapDataType dt = elem_bytes == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                           : elem_bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16
                                             : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  CUresult r = enc(map, dt, 4, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled (4-D) failed with CUresult " + std::to_string(r));
  return ATTN_OK;
}

attn_status_t set_smem(const void* kernel, int bytes) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return fail_cuda(e, "cudaFuncSetAttribute(max dynamic shared memory)");
  return ATTN_OK;
}

// One thread waits on a barrier that nothing arrives on, through the same
// bounded wait every kernel uses; the wait gives up after limit_ns and the
// kernel records the timeout in the status word and returns.
__global__ void selftest_wait_kernel(int* status, uint64_t limit_ns) {
  __shared__ __align__(8) uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x != 0) return;
  abort_flag = 0;
  mbar_init(&bar, 1);
  fence_mbar_init();
  const Abort ab{&abort_flag, status};
  mbar_wait_limit(&bar, 0, ab, kDevTimeoutSelftest, limit_ns);
}

}  // namespace attn

using namespace attn;

extern "C" {

const char* attn_status_string(attn_status_t s) {
  switch (s) {
    case ATTN_OK: return "ok";
    case ATTN_ERR_INVALID_ARG: return "invalid argument";
    case ATTN_ERR_UNSUPPORTED: return "unsupported shape or mode";
    case ATTN_ERR_ARCH: return "device is not compute capability 10.3";
    case ATTN_ERR_CUDA: return "CUDA error";
    case ATTN_ERR_TIMEOUT: return "a kernel wait exceeded its time limit";
  }
  return "unknown status";
}

const char* attn_last_error(void) { return g_last_error.c_str(); }

size_t attn_bwd_workspace_size(int B, int H, int N, int d) {
  if (B < 1 || H < 1 || N < 1 || d < 1) return 0;
  return bwd_workspace_layout(B, H, N, d).total;
}

attn_status_t attn_fwd_gqa(const void* q, const void* k, const void* v, void* o, float* lse,
                           int B, int H, int H_kv, int N, int d, int causal, float softmax_scale,
                           attn_dtype_t dtype, cudaStream_t stream) {
  g_last_error.clear();
  attn_status_t s;
  if ((s = check_shape(B, H, N, d, causal)) != ATTN_OK) return s;
  if ((s = check_heads(H, H_kv)) != ATTN_OK) return s;
  if ((s = check_ptrs({q, k, v, o, lse})) != ATTN_OK) return s;
  if ((s = check_scale(softmax_scale)) != ATTN_OK) return s;
  if (dtype != ATTN_BF16 && dtype != ATTN_FP16)
    return fail(ATTN_ERR_INVALID_ARG, "dtype must be ATTN_BF16 or ATTN_FP16");
  if ((s = check_device()) != ATTN_OK) return s;
  FwdParams p{q, k, v, o, lse, B, H, N, d, H_kv, nullptr, 0, causal, softmax_scale,
              dtype == ATTN_FP16 ? 1 : 0};
  return launch_fwd(p, stream);
}

attn_status_t attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                       int H, int N, int d, int causal, float softmax_scale, attn_dtype_t dtype,
                       cudaStream_t stream) {
  return attn_fwd_gqa(q, k, v, o, lse, B, H, H, N, d, causal, softmax_scale, dtype, stream);
}

attn_status_t attn_fwd_schedule(const void* q, const void* k, const void* v, void* o, float* lse,
                                int B, int H, int N, int d, int causal, float softmax_scale,
                                attn_dtype_t dtype, int schedule, cudaStream_t stream) {
  g_last_error.clear();
  attn_status_t s;
  if ((s = check_shape(B, H, N, d, causal)) != ATTN_OK) return s;
  if ((s = check_ptrs({q, k, v, o, lse})) != ATTN_OK) return s;
  if ((s = check_scale(softmax_scale)) != ATTN_OK) return s;
  if (dtype != ATTN_BF16 && dtype != ATTN_FP16)
    return fail(ATTN_ERR_INVALID_ARG, "dtype must be ATTN_BF16 or ATTN_FP16");
  if (schedule < 0 || schedule > (ATTN_SCHED_ONE_TILE | ATTN_SCHED_EAGER_RESCALE))
    return fail(ATTN_ERR_INVALID_ARG, "schedule must combine ATTN_SCHED_* flags");
  if (dtype != ATTN_BF16 || d == 256)
    return fail(ATTN_ERR_UNSUPPORTED, "schedule variants: bfloat16, d = 64 or 128");
  if ((s = check_device()) != ATTN_OK) return s;
  FwdParams p{q, k, v, o, lse, B, H, N, d, H, nullptr, 0, causal, softmax_scale, 0};
  return launch_fwd_sched(p, schedule, stream);
}

attn_status_t attn_fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse,
                              const int* cu_seqlens, int B, int max_seqlen, int total, int H,
                              int H_kv, int d, int causal, float softmax_scale,
                              attn_dtype_t dtype, cudaStream_t stream) {
  g_last_error.clear();
  attn_status_t s;
  if ((s = check_packed(B, max_seqlen, total, H, d, causal)) != ATTN_OK) return s;
  if ((s = check_heads(H, H_kv)) != ATTN_OK) return s;
  if ((s = check_ptrs({q, k, v, o, lse})) != ATTN_OK) return s;
  if (cu_seqlens == nullptr || (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) != 0)
    return fail(ATTN_ERR_INVALID_ARG, "cu_seqlens must be a non-null, 4-byte aligned device array");
  if ((s = check_scale(softmax_scale)) != ATTN_OK) return s;
  if (dtype != ATTN_BF16 && dtype != ATTN_FP16)
    return fail(ATTN_ERR_INVALID_ARG, "dtype must be ATTN_BF16 or ATTN_FP16");
  if ((s = check_device()) != ATTN_OK) return s;
  FwdParams p{q, k, v, o, lse, B, H, max_seqlen, d, H_kv, cu_seqlens, total, causal,
              softmax_scale, dtype == ATTN_FP16 ? 1 : 0};
  return launch_fwd(p, stream);
}

// Shared by the backward entry points after their own shape checks.
static attn_status_t bwd_common(const void* q, const void* k, const void* v, const void* o,
                                const void* dout, const float* lse, void* dq, void* dk, void* dv,
                                void* workspace, size_t workspace_bytes, size_t workspace_need,
                                const BwdWorkspace& w, int B, int H, int H_kv, int N, int d,
                                const int* cu_seqlens, int total, int causal,
                                float softmax_scale, attn_dtype_t dtype, cudaStream_t stream) {
  attn_status_t s;
  if ((s = check_ptrs({q, k, v, o, dout, lse, dq, dk, dv, workspace})) != ATTN_OK) return s;
  if ((s = check_scale(softmax_scale)) != ATTN_OK) return s;
  if (dtype != ATTN_BF16 && dtype != ATTN_FP16)
    return fail(ATTN_ERR_INVALID_ARG, "dtype must be ATTN_BF16 or ATTN_FP16");
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(ATTN_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (workspace_bytes < workspace_need)
    return fail(ATTN_ERR_INVALID_ARG, "workspace smaller than the workspace-size query returns");
  if (d == 256) return fail(ATTN_ERR_UNSUPPORTED, "the backward pass supports d = 64 and 128");
  if ((s = check_device()) != ATTN_OK) return s;
  char* ws = static_cast<char*>(workspace);
  BwdParams p{q,  k,  v,  o,  dout, lse, dq, dk, dv, reinterpret_cast<float*>(ws + w.dq_acc),
              reinterpret_cast<float*>(ws + w.lse2), reinterpret_cast<float*>(ws + w.delta),
              B,  H,  N,  d,  H_kv, cu_seqlens, total, causal, softmax_scale,
              dtype == ATTN_FP16 ? 1 : 0};
  return launch_bwd(p, stream);
}

attn_status_t attn_bwd_gqa(const void* q, const void* k, const void* v, const void* o,
                           const void* dout, const float* lse, void* dq, void* dk, void* dv,
                           void* workspace, size_t workspace_bytes, int B, int H, int H_kv, int N,
                           int d, int causal, float softmax_scale, attn_dtype_t dtype,
                           cudaStream_t stream) {
  g_last_error.clear();
  attn_status_t s;
  if ((s = check_shape(B, H, N, d, causal)) != ATTN_OK) return s;
  if ((s = check_heads(H, H_kv)) != ATTN_OK) return s;
  return bwd_common(q, k, v, o, dout, lse, dq, dk, dv, workspace, workspace_bytes,
                    attn_bwd_workspace_size(B, H, N, d), bwd_workspace_layout(B, H, N, d), B, H,
                    H_kv, N, d, nullptr, 0, causal, softmax_scale, dtype, stream);
}

attn_status_t attn_bwd(const void* q, const void* k, const void* v, const void* o,
                       const void* dout, const float* lse, void* dq, void* dk, void* dv,
                       void* workspace, size_t workspace_bytes, int B, int H, int N, int d,
                       int causal, float softmax_scale, attn_dtype_t dtype,
                       cudaStream_t stream) {
  return attn_bwd_gqa(q, k, v, o, dout, lse, dq, dk, dv, workspace, workspace_bytes, B, H, H, N,
                      d, causal, softmax_scale, dtype, stream);
}

size_t attn_bwd_varlen_workspace_size(int B, int max_seqlen, int total, int H, int d) {
  if (B < 1 || max_seqlen < 1 || total < 1 || H < 1 || d < 1) return 0;
  return bwd_workspace_layout_packed(B, max_seqlen, total, H, d).total;
}

attn_status_t attn_bwd_varlen(const void* q, const void* k, const void* v, const void* o,
                              const void* dout, const float* lse, void* dq, void* dk, void* dv,
                              void* workspace, size_t workspace_bytes, const int* cu_seqlens,
                              int B, int max_seqlen, int total, int H, int H_kv, int d,
                              int causal, float softmax_scale, attn_dtype_t dtype,
                              cudaStream_t stream) {
  g_last_error.clear();
  attn_status_t s;
  if ((s = check_packed(B, max_seqlen, total, H, d, causal)) != ATTN_OK) return s;
  if ((s = check_heads(H, H_kv)) != ATTN_OK) return s;
  if (cu_seqlens == nullptr || (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) != 0)
    return fail(ATTN_ERR_INVALID_ARG, "cu_seqlens must be a non-null, 4-byte aligned device array");
  return bwd_common(q, k, v, o, dout, lse, dq, dk, dv, workspace, workspace_bytes,
                    attn_bwd_varlen_workspace_size(B, max_seqlen, total, H, d),
                    bwd_workspace_layout_packed(B, max_seqlen, total, H, d), B, H, H_kv,
                    max_seqlen, d, cu_seqlens, total, causal, softmax_scale, dtype, stream);
}

attn_status_t attn_fp8_quantize(const float* q, const float* k, const float* v,
                                const float* hadamard_signs, uint8_t* q8, uint8_t* k8,
                                uint8_t* v8, float* q_descale, float* k_descale,
                                float* v_descale, int B, int H, int N, int d, int per_tensor,
                                cudaStream_t stream) {
  return attn_fp8_quantize_gqa(q, k, v, hadamard_signs, q8, k8, v8, q_descale, k_descale,
                               v_descale, B, H, H, N, d, per_tensor, stream);
}

// Shared by the fixed-length pre-pass entry points (float32 or bfloat16 inputs).
static attn_status_t fp8_quantize_common(const void* q, const void* k, const void* v,
                                         const float* hadamard_signs, uint8_t* q8, uint8_t* k8,
                                         uint8_t* v8, float* q_descale, float* k_descale,
                                         float* v_descale, int B, int H, int H_kv, int N, int d,
                                         int per_tensor, int in_bf16, cudaStream_t stream);

attn_status_t attn_fp8_quantize_gqa(const float* q, const float* k, const float* v,
                                    const float* hadamard_signs, uint8_t* q8, uint8_t* k8,
                                    uint8_t* v8, float* q_descale, float* k_descale,
                                    float* v_descale, int B, int H, int H_kv, int N, int d,
                                    int per_tensor, cudaStream_t stream) {
  return fp8_quantize_common(q, k, v, hadamard_signs, q8, k8, v8, q_descale, k_descale, v_descale,
                             B, H, H_kv, N, d, per_tensor, 0, stream);
}

attn_status_t attn_fp8_quantize_bf16(const void* q, const void* k, const void* v,
                                     const float* hadamard_signs, uint8_t* q8, uint8_t* k8,
                                     uint8_t* v8, float* q_descale, float* k_descale,
                                     float* v_descale, int B, int H, int H_kv, int N, int d,
                                     int per_tensor, cudaStream_t stream) {
  return fp8_quantize_common(q, k, v, hadamard_signs, q8, k8, v8, q_descale, k_descale, v_descale,
                             B, H, H_kv, N, d, per_tensor, 1, stream);
}

static attn_status_t fp8_quantize_common(const void* q, const void* k, const void* v,
                                         const float* hadamard_signs, uint8_t* q8, uint8_t* k8,
                                         uint8_t* v8, float* q_descale, float* k_descale,
                                         float* v_descale, int B, int H, int H_kv, int N, int d,
                                         int per_tensor, int in_bf16, cudaStream_t stream) {
  g_last_error.clear();
  attn_status_t s;
  if ((s = check_shape(B, H, N, d, 0)) != ATTN_OK) return s;
  if ((s = check_heads(H, H_kv)) != ATTN_OK) return s;
  if ((s = check_ptrs({q, k, v, q8, k8, v8, q_descale, k_descale, v_descale})) != ATTN_OK)
    return s;
  if (per_tensor != 0 && per_tensor != 1)
    return fail(ATTN_ERR_INVALID_ARG, "per_tensor must be 0 or 1");
  if (per_tensor && hadamard_signs)
    return fail(ATTN_ERR_INVALID_ARG, "the per-tensor comparator takes no Hadamard signs");
  if (hadamard_signs && !aligned16(hadamard_signs))
    return fail(ATTN_ERR_INVALID_ARG, "hadamard_signs not 16-byte aligned");
  if (d != 128) return fail(ATTN_ERR_UNSUPPORTED, "the FP8 path supports d = 128");
  if ((s = check_device()) != ATTN_OK) return s;
  Fp8QuantParams p{{q, k, v}, {q8, k8, v8}, {q_descale, k_descale, v_descale}, hadamard_signs,
                   B, H, N, d, per_tensor, nullptr, nullptr, H_kv, nullptr, 0, in_bf16};
  return launch_fp8_quantize(p, stream);
}

attn_status_t attn_fp8_quantize_varlen(const float* q, const float* k, const float* v,
                                       const float* hadamard_signs, uint8_t* q8, uint8_t* k8,
                                       uint8_t* v8, float* q_descale, float* k_descale,
                                       float* v_descale, const int* cu_seqlens, int B,
                                       int max_seqlen, int total, int H, int H_kv, int d,
                                       cudaStream_t stream) {
  g_last_error.clear();
  attn_status_t s;
  if ((s = check_packed(B, max_seqlen, total, H, d, 0)) != ATTN_OK) return s;
  if ((s = check_heads(H, H_kv)) != ATTN_OK) return s;
  if ((s = check_ptrs({q, k, v, q8, k8, v8, q_descale, k_descale, v_descale})) != ATTN_OK)
    return s;
  if (cu_seqlens == nullptr || (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) != 0)
    return fail(ATTN_ERR_INVALID_ARG, "cu_seqlens must be a non-null, 4-byte aligned device array");
  if (hadamard_signs && !aligned16(hadamard_signs))
    return fail(ATTN_ERR_INVALID_ARG, "hadamard_signs not 16-byte aligned");
  if (d != 128) return fail(ATTN_ERR_UNSUPPORTED, "the FP8 path supports d = 128");
  if ((s = check_device()) != ATTN_OK) return s;
  Fp8QuantParams p{{q, k, v}, {q8, k8, v8}, {q_descale, k_descale, v_descale}, hadamard_signs,
                   B, H, max_seqlen, d, 0, nullptr, nullptr, H_kv, cu_seqlens, total};
  return launch_fp8_quantize(p, stream);
}

attn_status_t attn_fp8_quantize_rope(const float* q, const float* k, const float* v,
                                     const float* rope_cos, const float* rope_sin,
                                     const float* hadamard_signs, uint8_t* q8, uint8_t* k8,
                                     uint8_t* v8, float* q_descale, float* k_descale,
                                     float* v_descale, int B, int H, int N, int d,
                                     cudaStream_t stream) {
  g_last_error.clear();
  attn_status_t s;
  if ((s = check_shape(B, H, N, d, 0)) != ATTN_OK) return s;
  if ((s = check_ptrs({q, k, v, rope_cos, rope_sin, q8, k8, v8, q_descale, k_descale,
                       v_descale})) != ATTN_OK)
    return s;
  if (hadamard_signs && !aligned16(hadamard_signs))
    return fail(ATTN_ERR_INVALID_ARG, "hadamard_signs not 16-byte aligned");
  if (d != 128) return fail(ATTN_ERR_UNSUPPORTED, "the FP8 path supports d = 128");
  if ((s = check_device()) != ATTN_OK) return s;
  Fp8QuantParams p{{q, k, v}, {q8, k8, v8}, {q_descale, k_descale, v_descale}, hadamard_signs,
                   B, H, N, d, 0, rope_cos, rope_sin};
  return launch_fp8_quantize(p, stream);
}

attn_status_t attn_fp8_quantize_ex(const void* q, const void* k, const void* v, int input_bf16,
                                   const float* rope_cos, const float* rope_sin,
                                   const float* hadamard_signs, uint8_t* q8, uint8_t* k8,
                                   uint8_t* v8, float* q_descale, float* k_descale,
                                   float* v_descale, const int* cu_seqlens, int B, int N,
                                   int total, int H, int H_kv, int d, int per_tensor,
                                   cudaStream_t stream) {
  g_last_error.clear();
  attn_status_t s;
  if (input_bf16 != 0 && input_bf16 != 1)
    return fail(ATTN_ERR_INVALID_ARG, "input_bf16 must be 0 or 1");
  if (cu_seqlens) {
    if ((s = check_packed(B, N, total, H, d, 0)) != ATTN_OK) return s;
    if (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u)
      return fail(ATTN_ERR_INVALID_ARG, "cu_seqlens must be 4-byte aligned");
  } else {
    if ((s = check_shape(B, H, N, d, 0)) != ATTN_OK) return s;
  }
  if ((s = check_heads(H, H_kv)) != ATTN_OK) return s;
  if ((s = check_ptrs({q, k, v, q8, k8, v8, q_descale, k_descale, v_descale})) != ATTN_OK)
    return s;
  if ((rope_cos == nullptr) != (rope_sin == nullptr))
    return fail(ATTN_ERR_INVALID_ARG, "give both rope_cos and rope_sin, or neither");
  if (rope_cos && (!aligned16(rope_cos) || !aligned16(rope_sin)))
    return fail(ATTN_ERR_INVALID_ARG, "rope tables must be 16-byte aligned");
  if (hadamard_signs && !aligned16(hadamard_signs))
    return fail(ATTN_ERR_INVALID_ARG, "hadamard_signs not 16-byte aligned");
  if (per_tensor != 0 && per_tensor != 1)
    return fail(ATTN_ERR_INVALID_ARG, "per_tensor must be 0 or 1");
  if (per_tensor && (hadamard_signs || rope_cos || cu_seqlens))
    return fail(ATTN_ERR_INVALID_ARG,
                "the per-tensor comparator takes fixed-length inputs without Hadamard or rotation");
  if (d != 128) return fail(ATTN_ERR_UNSUPPORTED, "the FP8 path supports d = 128");
  if ((s = check_device()) != ATTN_OK) return s;
  Fp8QuantParams p{{q, k, v}, {q8, k8, v8}, {q_descale, k_descale, v_descale}, hadamard_signs,
                   B, H, N, d, per_tensor, rope_cos, rope_sin, H_kv, cu_seqlens,
                   cu_seqlens ? total : 0, input_bf16};
  return launch_fp8_quantize(p, stream);
}

size_t attn_decode_workspace_size(int B, int H, int H_kv, int n_q, int d, int max_seqlen) {
  if (B < 1 || H < 1 || H_kv < 1 || n_q < 1 || d < 1 || max_seqlen < 1) return 0;
  return decode_workspace_bytes(B, H, H_kv, n_q, d, max_seqlen);
}

attn_status_t attn_decode_paged(const void* q, const void* k_cache, const void* v_cache,
                                const int* block_table, const int* seq_lens, void* o, float* lse,
                                void* workspace, size_t workspace_bytes, int B, int H, int H_kv,
                                int n_q, int d, int num_pages, int page_size, int max_pages,
                                int max_seqlen, int causal, float softmax_scale,
                                attn_dtype_t dtype, cudaStream_t stream) {
  g_last_error.clear();
  attn_status_t s;
  if (B < 1 || H < 1 || n_q < 1 || num_pages < 1 || max_pages < 1 || max_seqlen < 1)
    return fail(ATTN_ERR_INVALID_ARG, "B, H, n_q, num_pages, max_pages and max_seqlen must be >= 1");
  if ((s = check_heads(H, H_kv)) != ATTN_OK) return s;
  if (d != 64 && d != 128) return fail(ATTN_ERR_INVALID_ARG, "decode supports d = 64 and 128");
  if (causal != 0 && causal != 1) return fail(ATTN_ERR_INVALID_ARG, "causal must be 0 or 1");
  if ((H / H_kv) * n_q > 128)
    return fail(ATTN_ERR_UNSUPPORTED, "(H / H_kv) * n_q must be <= 128 (one query tile)");
  if (page_size < 8 || page_size > 65536 || (page_size & (page_size - 1)) != 0)
    return fail(ATTN_ERR_INVALID_ARG, "page_size must be a power of two in [8, 65536]");
  if (static_cast<long long>(max_pages) * page_size > 2147483647LL ||
      static_cast<double>(num_pages) * page_size * H_kv * d >= 9.0e15)
    return fail(ATTN_ERR_INVALID_ARG, "cache too large");
  if (static_cast<double>(B) * H * n_q * d >= 2147483648.0)
    return fail(ATTN_ERR_INVALID_ARG, "B*H*n_q*d must be < 2^31");
  if ((s = check_ptrs({q, k_cache, v_cache, o, lse, workspace})) != ATTN_OK) return s;
  if (!block_table || !seq_lens || (reinterpret_cast<uintptr_t>(block_table) & 3u) ||
      (reinterpret_cast<uintptr_t>(seq_lens) & 3u))
    return fail(ATTN_ERR_INVALID_ARG, "block_table and seq_lens must be non-null, 4-byte aligned");
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(ATTN_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (workspace_bytes < attn_decode_workspace_size(B, H, H_kv, n_q, d, max_seqlen))
    return fail(ATTN_ERR_INVALID_ARG, "workspace smaller than attn_decode_workspace_size()");
  if ((s = check_scale(softmax_scale)) != ATTN_OK) return s;
  if (dtype != ATTN_BF16 && dtype != ATTN_FP16)
    return fail(ATTN_ERR_INVALID_ARG, "dtype must be ATTN_BF16 or ATTN_FP16");
  if ((s = check_device()) != ATTN_OK) return s;
  const DecodeSplits sp = decode_splits(B, H_kv, max_seqlen);
  const size_t rows = static_cast<size_t>(B) * H * n_q * sp.splits;
  char* ws = static_cast<char*>(workspace);
  DecodeParams p{q, k_cache, v_cache, block_table, seq_lens, o, lse,
                 reinterpret_cast<float*>(ws),
                 reinterpret_cast<float*>(ws + align_up(rows * d * sizeof(float), 256)),
                 B, H, H_kv, n_q, d, num_pages, page_size, max_pages, max_seqlen, causal,
                 softmax_scale, dtype == ATTN_FP16 ? 1 : 0};
  return launch_decode(p, stream);
}

attn_status_t attn_decode_paged_fp8(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                    const float* k_descale, const float* v_descale,
                                    const float* hadamard_signs, const int* block_table,
                                    const int* seq_lens, void* o, float* lse, void* workspace,
                                    size_t workspace_bytes, int B, int H, int H_kv, int n_q, int d,
                                    int num_pages, int page_size, int max_pages, int max_seqlen,
                                    int causal, float softmax_scale, attn_dtype_t dtype,
                                    cudaStream_t stream) {
  g_last_error.clear();
  attn_status_t s;
  if (B < 1 || H < 1 || n_q < 1 || num_pages < 1 || max_pages < 1 || max_seqlen < 1)
    return fail(ATTN_ERR_INVALID_ARG, "B, H, n_q, num_pages, max_pages and max_seqlen must be >= 1");
  if ((s = check_heads(H, H_kv)) != ATTN_OK) return s;
  if (d != 128) return fail(ATTN_ERR_UNSUPPORTED, "the FP8 decode supports d = 128");
  if (causal != 0 && causal != 1) return fail(ATTN_ERR_INVALID_ARG, "causal must be 0 or 1");
  if ((H / H_kv) * n_q > 128)
    return fail(ATTN_ERR_UNSUPPORTED, "(H / H_kv) * n_q must be <= 128 (one query tile)");
  if (page_size < 16 || page_size > 65536 || (page_size & (page_size - 1)) != 0)
    return fail(ATTN_ERR_INVALID_ARG, "page_size must be a power of two in [16, 65536] for an FP8 cache");
  if (static_cast<long long>(max_pages) * page_size > 2147483647LL ||
      static_cast<double>(num_pages) * page_size * H_kv * d >= 9.0e15)
    return fail(ATTN_ERR_INVALID_ARG, "cache too large");
  if (static_cast<double>(B) * H * n_q * d >= 2147483648.0)
    return fail(ATTN_ERR_INVALID_ARG, "B*H*n_q*d must be < 2^31");
  if ((s = check_ptrs({q, k_cache, v_cache, o, lse, workspace, k_descale, v_descale})) != ATTN_OK)
    return s;
  if (hadamard_signs && (reinterpret_cast<uintptr_t>(hadamard_signs) & 15u))
    return fail(ATTN_ERR_INVALID_ARG, "hadamard_signs must be 16-byte aligned");
  if (!block_table || !seq_lens || (reinterpret_cast<uintptr_t>(block_table) & 3u) ||
      (reinterpret_cast<uintptr_t>(seq_lens) & 3u))
    return fail(ATTN_ERR_INVALID_ARG, "block_table and seq_lens must be non-null, 4-byte aligned");
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(ATTN_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (workspace_bytes < attn_decode_workspace_size(B, H, H_kv, n_q, d, max_seqlen))
    return fail(ATTN_ERR_INVALID_ARG, "workspace smaller than attn_decode_workspace_size()");
  if ((s = check_scale(softmax_scale)) != ATTN_OK) return s;
  if (dtype != ATTN_BF16 && dtype != ATTN_FP16)
    return fail(ATTN_ERR_INVALID_ARG, "dtype must be ATTN_BF16 or ATTN_FP16");
  if ((s = check_device()) != ATTN_OK) return s;
  const DecodeSplits sp = decode_splits(B, H_kv, max_seqlen);
  const size_t rows = static_cast<size_t>(B) * H * n_q * sp.splits;
  char* ws = static_cast<char*>(workspace);
  DecodeParams p{q, k_cache, v_cache, block_table, seq_lens, o, lse,
                 reinterpret_cast<float*>(ws),
                 reinterpret_cast<float*>(ws + align_up(rows * d * sizeof(float), 256)),
                 B, H, H_kv, n_q, d, num_pages, page_size, max_pages, max_seqlen, causal,
                 softmax_scale, dtype == ATTN_FP16 ? 1 : 0,
                 1, k_descale, v_descale, hadamard_signs};
  return launch_decode(p, stream);
}

attn_status_t attn_fwd_fp8(const uint8_t* q8, const uint8_t* k8, const uint8_t* v8,
                           const float* q_descale, const float* k_descale,
                           const float* v_descale, void* o, float* lse, int B, int H, int N,
                           int d, int causal, float softmax_scale, cudaStream_t stream) {
  return attn_fwd_fp8_gqa(q8, k8, v8, q_descale, k_descale, v_descale, o, lse, B, H, H, N, d,
                          causal, softmax_scale, stream);
}

attn_status_t attn_fwd_fp8_schedule(const uint8_t* q8, const uint8_t* k8, const uint8_t* v8,
                                    const float* q_descale, const float* k_descale,
                                    const float* v_descale, void* o, float* lse, int B, int H,
                                    int N, int d, int causal, float softmax_scale, int schedule,
                                    cudaStream_t stream) {
  g_last_error.clear();
  attn_status_t s;
  if ((s = check_shape(B, H, N, d, causal)) != ATTN_OK) return s;
  if ((s = check_ptrs({q8, k8, v8, o, lse})) != ATTN_OK) return s;
  if (!q_descale || !k_descale || !v_descale)
    return fail(ATTN_ERR_INVALID_ARG, "null descale pointer");
  if ((s = check_scale(softmax_scale)) != ATTN_OK) return s;
  // 0, ATTN_SCHED_EXP2_NONE, or ATTN_SCHED_EXP2_POLY with an optional share of 1..4
  // eighths in bits 8..11
  const int eighths = (schedule >> 8) & 15;
  if (schedule != 0 && schedule != ATTN_SCHED_EXP2_NONE &&
      ((schedule & ~(15 << 8)) != ATTN_SCHED_EXP2_POLY || eighths > 4))
    return fail(ATTN_ERR_INVALID_ARG,
                "schedule must be 0, ATTN_SCHED_EXP2_NONE, ATTN_SCHED_EXP2_POLY or "
                "ATTN_SCHED_EXP2_EIGHTHS(1..4)");
  if (d != 128) return fail(ATTN_ERR_UNSUPPORTED, "the FP8 path supports d = 128");
  if ((s = check_device()) != ATTN_OK) return s;
  Fp8FwdParams p{q8, k8, v8, q_descale, k_descale, v_descale, o, lse, B, H, N, d, causal,
                 softmax_scale, H};
  // the kernels count the share in sixteenths
  p.exp2_poly = schedule == 0 ? -1 : schedule == ATTN_SCHED_EXP2_NONE ? 0 : 2 * (eighths == 0 ? 2 : eighths);
  return launch_fwd_fp8(p, stream);
}

attn_status_t attn_selftest_exp2(const float* x, float* y_poly, float* y_mufu, long long n,
                                 cudaStream_t stream) {
  g_last_error.clear();
  attn_status_t s;
  if (n < 1 || n > (1ll << 30)) return fail(ATTN_ERR_INVALID_ARG, "n must be in [1, 2^30]");
  if (!x || !y_poly || !y_mufu) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
  if ((s = check_device()) != ATTN_OK) return s;
  return launch_exp2_selftest(x, y_poly, y_mufu, n, stream);
}

attn_status_t attn_fwd_fp8_varlen(const uint8_t* q8, const uint8_t* k8, const uint8_t* v8,
                                  const float* q_descale, const float* k_descale,
                                  const float* v_descale, void* o, float* lse,
                                  const int* cu_seqlens, int B, int max_seqlen, int total, int H,
                                  int H_kv, int d, int causal, float softmax_scale,
                                  cudaStream_t stream) {
  g_last_error.clear();
  attn_status_t s;
  if ((s = check_packed(B, max_seqlen, total, H, d, causal)) != ATTN_OK) return s;
  if ((s = check_heads(H, H_kv)) != ATTN_OK) return s;
  if ((s = check_ptrs({q8, k8, v8, o, lse})) != ATTN_OK) return s;
  if (!q_descale || !k_descale || !v_descale)
    return fail(ATTN_ERR_INVALID_ARG, "null descale pointer");
  if (cu_seqlens == nullptr || (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) != 0)
    return fail(ATTN_ERR_INVALID_ARG, "cu_seqlens must be a non-null, 4-byte aligned device array");
  if ((s = check_scale(softmax_scale)) != ATTN_OK) return s;
  if (d != 128) return fail(ATTN_ERR_UNSUPPORTED, "the FP8 path supports d = 128");
  if ((s = check_device()) != ATTN_OK) return s;
  Fp8FwdParams p{q8, k8, v8, q_descale, k_descale, v_descale, o, lse, B, H, max_seqlen, d, causal,
                 softmax_scale, H_kv, cu_seqlens, total};
  return launch_fwd_fp8(p, stream);
}

attn_status_t attn_fwd_fp8_gqa(const uint8_t* q8, const uint8_t* k8, const uint8_t* v8,
                               const float* q_descale, const float* k_descale,
                               const float* v_descale, void* o, float* lse, int B, int H,
                               int H_kv, int N, int d, int causal, float softmax_scale,
                               cudaStream_t stream) {
  g_last_error.clear();
  attn_status_t s;
  if ((s = check_shape(B, H, N, d, causal)) != ATTN_OK) return s;
  if ((s = check_heads(H, H_kv)) != ATTN_OK) return s;
  if ((s = check_ptrs({q8, k8, v8, o, lse})) != ATTN_OK) return s;
  if (!q_descale || !k_descale || !v_descale)
    return fail(ATTN_ERR_INVALID_ARG, "null descale pointer");
  if ((s = check_scale(softmax_scale)) != ATTN_OK) return s;
  if (d != 128) return fail(ATTN_ERR_UNSUPPORTED, "the FP8 path supports d = 128");
  if ((s = check_device()) != ATTN_OK) return s;
  Fp8FwdParams p{q8, k8, v8, q_descale, k_descale, v_descale, o, lse, B, H, N, d, causal,
                 softmax_scale, H_kv};
  return launch_fwd_fp8(p, stream);
}

// Shape checks shared by the cross-attention entry points.
static attn_status_t check_cross(int B, int H, int H_kv, int N_q, int N_k, int d, const int* kv_lens) {
  attn_status_t s;
  if (N_k < 1) return fail(ATTN_ERR_INVALID_ARG, "N_k must be >= 1");
  if ((s = check_shape(B, H, N_q, d, 0)) != ATTN_OK) return s;
  if ((s = check_heads(H, H_kv)) != ATTN_OK) return s;
  if (static_cast<double>(B) * H_kv * N_k * d >= 2147483648.0)
    return fail(ATTN_ERR_INVALID_ARG, "B*H_kv*N_k*d must be < 2^31");
  if (B > 65535 || H > 65535) return fail(ATTN_ERR_UNSUPPORTED, "grid dimension limit exceeded");
  if (reinterpret_cast<uintptr_t>(kv_lens) & 3u)
    return fail(ATTN_ERR_INVALID_ARG, "kv_lens must be 4-byte aligned");
  return ATTN_OK;
}

size_t attn_cross_workspace_size(int B, int H, int H_kv, int N_q, int N_k, int d) {
  if (B < 1 || H < 1 || H_kv < 1 || H % H_kv != 0 || N_q < 1 || N_k < 1 || d < 1) return 0;
  return cross_workspace_bytes(H, H_kv, N_q, d, cross_plan(B, H, H_kv, N_q, N_k, d));
}

attn_status_t attn_cross_fwd(const void* q, const void* k, const void* v, const int* kv_lens, void* o,
                             float* lse, void* workspace, size_t workspace_bytes, int B, int H, int H_kv,
                             int N_q, int N_k, int d, float softmax_scale, attn_dtype_t dtype,
                             cudaStream_t stream) {
  g_last_error.clear();
  attn_status_t s;
  if ((s = check_cross(B, H, H_kv, N_q, N_k, d, kv_lens)) != ATTN_OK) return s;
  if ((s = check_ptrs({q, k, v, o, lse})) != ATTN_OK) return s;
  if ((s = check_scale(softmax_scale)) != ATTN_OK) return s;
  if ((s = check_dtype(dtype)) != ATTN_OK) return s;
  const CrossPlan plan = cross_plan(B, H, H_kv, N_q, N_k, d);
  const size_t need = cross_workspace_bytes(H, H_kv, N_q, d, plan);
  if (need > 0) {
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
      return fail(ATTN_ERR_INVALID_ARG, "workspace must be non-null and 256-byte aligned");
    if (workspace_bytes < need)
      return fail(ATTN_ERR_INVALID_ARG, "workspace smaller than attn_cross_workspace_size()");
  }
  if ((s = check_device()) != ATTN_OK) return s;
  FwdParams p{q, k, v, o, lse, B, H, N_q, d, H_kv, nullptr, 0, 0, softmax_scale,
              dtype == ATTN_FP16 ? 1 : 0, N_k, kv_lens};
  return plan.ctas > 0 ? launch_cross_rows(p, plan, workspace, stream) : launch_cross_fwd(p, stream);
}

size_t attn_cross_bwd_workspace_size(int B, int H, int N_q, int N_k, int d) {
  if (B < 1 || H < 1 || N_q < 1 || N_k < 1 || d < 1) return 0;
  return cross_bwd_plan(B, H, N_q, N_k, d).total;
}

attn_status_t attn_cross_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout,
                             const float* lse, const int* kv_lens, void* dq, void* dk, void* dv,
                             void* workspace, size_t workspace_bytes, int B, int H, int H_kv, int N_q,
                             int N_k, int d, float softmax_scale, attn_dtype_t dtype,
                             cudaStream_t stream) {
  g_last_error.clear();
  attn_status_t s;
  if ((s = check_cross(B, H, H_kv, N_q, N_k, d, kv_lens)) != ATTN_OK) return s;
  if ((s = check_ptrs({q, k, v, o, dout, lse, dq, dk, dv, workspace})) != ATTN_OK) return s;
  if ((s = check_scale(softmax_scale)) != ATTN_OK) return s;
  if ((s = check_dtype(dtype)) != ATTN_OK) return s;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(ATTN_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  const CrossBwdPlan plan = cross_bwd_plan(B, H, N_q, N_k, d);
  if (workspace_bytes < plan.total)
    return fail(ATTN_ERR_INVALID_ARG, "workspace smaller than attn_cross_bwd_workspace_size()");
  if (d == 256) return fail(ATTN_ERR_UNSUPPORTED, "the backward pass supports d = 64 and 128");
  if (plan.steps > 2147483647LL) return fail(ATTN_ERR_UNSUPPORTED, "over 2^31 tile pairs");
  if ((s = check_device()) != ATTN_OK) return s;
  char* ws = static_cast<char*>(workspace);
  BwdParams p{q, k, v, o, dout, lse, dq, dk, dv, reinterpret_cast<float*>(ws + plan.w.dq_acc),
              reinterpret_cast<float*>(ws + plan.w.lse2), reinterpret_cast<float*>(ws + plan.w.delta),
              B, H, N_q, d, H_kv, nullptr, 0, 0, softmax_scale, dtype == ATTN_FP16 ? 1 : 0, N_k, kv_lens};
  return launch_cross_bwd(p, reinterpret_cast<float*>(ws + plan.part), plan.ctas, stream);
}

attn_status_t attn_rope_table(float* rope_cos, float* rope_sin, long long n, int rot_dim, double base,
                              double factor, long long orig_len, double low, double high,
                              double attn_factor, long long first, cudaStream_t stream) {
  g_last_error.clear();
  attn_status_t s;
  if (rot_dim < 16 || rot_dim > 256 || rot_dim % 16 != 0)
    return fail(ATTN_ERR_INVALID_ARG, "rot_dim must be a multiple of 16 in [16, 256]");
  if (n < 1 || first < 0 || first > 2147483647LL || n > 2147483647LL || first + n > 2147483648LL)
    return fail(ATTN_ERR_INVALID_ARG, "positions first .. first + n - 1 must lie in [0, 2^31)");
  if (!(base > 1.0) || !std::isfinite(base)) return fail(ATTN_ERR_INVALID_ARG, "base must be finite and > 1");
  if (!(factor >= 1.0) || !std::isfinite(factor))
    return fail(ATTN_ERR_INVALID_ARG, "factor must be finite and >= 1");
  if (orig_len < 0 || orig_len > 2147483647LL)
    return fail(ATTN_ERR_INVALID_ARG, "orig_len must lie in [0, 2^31)");
  if (orig_len > 0 && (!(low >= 0.0) || !(high > low) || !std::isfinite(high)))
    return fail(ATTN_ERR_INVALID_ARG, "0 <= low < high, in turns of the original context");
  if (!(attn_factor > 0.0) || !std::isfinite(attn_factor))
    return fail(ATTN_ERR_INVALID_ARG, "attn_factor must be positive and finite");
  if ((s = check_ptrs({rope_cos, rope_sin})) != ATTN_OK) return s;
  if ((s = check_device()) != ATTN_OK) return s;
  return launch_rope_table(rope_cos, rope_sin, n, rot_dim, base, factor, orig_len, low, high, attn_factor,
                           first, stream);
}

attn_status_t attn_rope(const void* q, void* q_out, const void* k, void* k_out, const float* rope_cos,
                        const float* rope_sin, const int* positions, int B, int N, int H, int H_kv, int d,
                        int rot_dim, int max_pos, const long long* q_strides, const long long* q_out_strides,
                        const long long* k_strides, const long long* k_out_strides, int interleaved,
                        int inverse, attn_dtype_t dtype, cudaStream_t stream) {
  g_last_error.clear();
  attn_status_t s;
  if ((s = check_shape(B, H, N, d, 0)) != ATTN_OK) return s;
  if (H_kv < 0 || static_cast<double>(B) * H_kv * N * d >= 2147483648.0)
    return fail(ATTN_ERR_INVALID_ARG, "H_kv must be >= 0 (0: no k) and B*H_kv*N*d < 2^31");
  if ((s = check_rope(rope_cos, rope_sin, d, rot_dim, max_pos, interleaved)) != ATTN_OK) return s;
  if (inverse != 0 && inverse != 1) return fail(ATTN_ERR_INVALID_ARG, "inverse must be 0 or 1");
  if ((s = check_dtype(dtype)) != ATTN_OK) return s;
  if ((s = check_ptrs({q, q_out})) != ATTN_OK) return s;
  if (H_kv > 0 && (s = check_ptrs({k, k_out})) != ATTN_OK) return s;
  if (reinterpret_cast<uintptr_t>(positions) & 3u)
    return fail(ATTN_ERR_INVALID_ARG, "positions must be 4-byte aligned");
  RopeKParams p{};
  auto put = [&](int t, const void* src, void* dst, int heads, const long long* si, const long long* so) {
    const long long row = d, head = static_cast<long long>(N) * d, batch = head * heads;
    p.src[t] = static_cast<const uint16_t*>(src);
    p.dst[t] = static_cast<uint16_t*>(dst);
    p.heads[t] = heads;
    p.sb[t] = si ? si[0] : batch, p.sh[t] = si ? si[1] : head, p.st[t] = si ? si[2] : row;
    p.db[t] = so ? so[0] : batch, p.dh[t] = so ? so[1] : head, p.dt[t] = so ? so[2] : row;
    attn_status_t r = check_row_strides({p.sb[t], p.sh[t], p.st[t]}, false);
    return r != ATTN_OK ? r : check_row_strides({p.db[t], p.dh[t], p.dt[t]}, true);
  };
  if ((s = put(0, q, q_out, H, q_strides, q_out_strides)) != ATTN_OK) return s;
  if (H_kv > 0 && (s = put(1, k, k_out, H_kv, k_strides, k_out_strides)) != ATTN_OK) return s;
  if ((s = check_device()) != ATTN_OK) return s;
  p.rotated = 2;
  p.cos = rope_cos, p.sin = rope_sin, p.positions = positions;
  p.B = B, p.N = N, p.d = d, p.rot = rot_dim, p.max_pos = max_pos, p.inverse = inverse;
  return launch_rope(p, dtype == ATTN_FP16, interleaved, stream);
}

attn_status_t attn_block_tables(int* block_table, const int* old_lens, const int* new_lens,
                                const int* free_pages, int* seq_lens, int* cu_seqlens, long long* slots,
                                int* positions, int* used, int B, int max_pages, int n_free, int page_size,
                                int capacity, cudaStream_t stream) {
  g_last_error.clear();
  attn_status_t s;
  if (B < 1 || max_pages < 1 || n_free < 0 || capacity < 0)
    return fail(ATTN_ERR_INVALID_ARG, "B and max_pages must be >= 1, n_free and capacity >= 0");
  if ((s = check_page_size(page_size, 8)) != ATTN_OK) return s;
  if (static_cast<long long>(max_pages) * page_size > 2147483647LL)
    return fail(ATTN_ERR_INVALID_ARG, "max_pages * page_size must be < 2^31");
  if ((s = check_ints({block_table, old_lens, new_lens, seq_lens, cu_seqlens, used})) != ATTN_OK) return s;
  if (n_free > 0 && (s = check_ints({free_pages})) != ATTN_OK) return s;
  if (capacity > 0) {
    if ((s = check_ints({positions})) != ATTN_OK) return s;
    if (slots == nullptr || (reinterpret_cast<uintptr_t>(slots) & 7u) != 0)
      return fail(ATTN_ERR_INVALID_ARG, "slots must be non-null and 8-byte aligned");
  }
  // every block reads the inputs while others write
  struct Range {
    const void* p;
    size_t bytes;
  };
  const size_t b4 = 4 * static_cast<size_t>(B), cap = static_cast<size_t>(capacity);
  const Range ins[] = {{old_lens, b4}, {new_lens, b4}, {free_pages, 4 * static_cast<size_t>(n_free)}};
  const Range outs[] = {{block_table, b4 * max_pages}, {seq_lens, b4}, {cu_seqlens, b4 + 4}, {slots, 8 * cap},
                        {positions, 4 * cap}, {used, 4}};
  for (const Range& o : outs)
    for (const Range& i : ins) {
      const uintptr_t x = reinterpret_cast<uintptr_t>(o.p), y = reinterpret_cast<uintptr_t>(i.p);
      if (o.bytes > 0 && i.bytes > 0 && x < y + i.bytes && y < x + o.bytes)
        return fail(ATTN_ERR_INVALID_ARG, "outputs (block_table, seq_lens, ...) must not overlap old_lens, new_lens or free_pages");
    }
  if ((s = check_device()) != ATTN_OK) return s;
  return launch_block_tables({block_table, old_lens, new_lens, free_pages, seq_lens, cu_seqlens, slots,
                              positions, used, B, max_pages, n_free, page_size, capacity},
                             stream);
}

// Checks and parameters shared by the two cache appends: rows of new tokens
// [total, heads, d] with {token, head} strides, q [total, H, d] optional.
static attn_status_t append_common(RopeKParams* p, const void* q, void* q_out, const void* k, const void* v,
                                   const void* k_cache, const void* v_cache, const float* rope_cos,
                                   const float* rope_sin, int total, int H, int H_kv, int d, int rot_dim,
                                   int max_pos, int num_pages, int page_size, const long long* q_strides,
                                   const long long* k_strides, const long long* v_strides, int interleaved,
                                   attn_dtype_t dtype) {
  attn_status_t s;
  if (total < 0 || H < 0 || H_kv < 1 || num_pages < 1)
    return fail(ATTN_ERR_INVALID_ARG, "total and H must be >= 0, H_kv and num_pages >= 1");
  if (d != 64 && d != 128 && d != 256) return fail(ATTN_ERR_INVALID_ARG, "d must be 64, 128 or 256");
  if (static_cast<double>(num_pages) * page_size * H_kv * d >= 9.0e15)
    return fail(ATTN_ERR_INVALID_ARG, "cache too large");
  if (static_cast<double>(total) * (H > H_kv ? H : H_kv) * d >= 2147483648.0)
    return fail(ATTN_ERR_INVALID_ARG, "total*H*d must be < 2^31");
  if (interleaved != 0 && interleaved != 1)
    return fail(ATTN_ERR_INVALID_ARG, "interleaved must be 0 or 1");
  if ((s = check_dtype(dtype)) != ATTN_OK) return s;
  if ((s = check_ptrs({k_cache, v_cache})) != ATTN_OK) return s;
  if (total > 0 && (s = check_ptrs({k, v})) != ATTN_OK) return s;
  if ((rope_cos == nullptr) != (rope_sin == nullptr))
    return fail(ATTN_ERR_INVALID_ARG, "give both rope_cos and rope_sin, or neither");
  if (rope_cos && (s = check_rope(rope_cos, rope_sin, d, rot_dim, max_pos, interleaved)) != ATTN_OK) return s;
  if (H > 0) {
    if (!rope_cos) return fail(ATTN_ERR_INVALID_ARG, "q is only rotated: it needs rope_cos and rope_sin");
    if (total > 0 && (s = check_ptrs({q, q_out})) != ATTN_OK) return s;
  }
  auto put = [&](int t, const void* src, int heads, const long long* strides) {
    p->src[t] = static_cast<const uint16_t*>(src);
    p->heads[t] = heads;
    p->st[t] = strides ? strides[0] : static_cast<long long>(heads) * d;
    p->sh[t] = strides ? strides[1] : d;
    return check_row_strides({p->st[t], p->sh[t]}, false);
  };
  if (H > 0 && (s = put(0, q, H, q_strides)) != ATTN_OK) return s;
  if ((s = put(1, k, H_kv, k_strides)) != ATTN_OK) return s;
  if ((s = put(2, v, H_kv, v_strides)) != ATTN_OK) return s;
  p->dst[0] = static_cast<uint16_t*>(q_out);
  p->dh[0] = d, p->dt[0] = static_cast<long long>(H) * d;
  p->rotated = rope_cos ? 2 : 0;
  p->cos = rope_cos, p->sin = rope_sin;
  p->B = 1, p->N = total, p->d = d, p->rot = rope_cos ? rot_dim : 0, p->max_pos = max_pos;
  return ATTN_OK;
}

attn_status_t attn_cache_append(const void* q, void* q_out, const void* k, const void* v, void* k_cache,
                                void* v_cache, const long long* slots, const float* rope_cos,
                                const float* rope_sin, const int* positions, int total, int H, int H_kv,
                                int d, int rot_dim, int max_pos, int num_pages, int page_size,
                                const long long* q_strides, const long long* k_strides,
                                const long long* v_strides, int interleaved, attn_dtype_t dtype,
                                cudaStream_t stream) {
  g_last_error.clear();
  attn_status_t s;
  if ((s = check_page_size(page_size, 8)) != ATTN_OK) return s;
  RopeKParams p{};
  if ((s = append_common(&p, q, q_out, k, v, k_cache, v_cache, rope_cos, rope_sin, total, H, H_kv, d,
                         rot_dim, max_pos, num_pages, page_size, q_strides, k_strides, v_strides,
                         interleaved, dtype)) != ATTN_OK)
    return s;
  if (total > 0) {
    if (slots == nullptr || (reinterpret_cast<uintptr_t>(slots) & 7u) != 0)
      return fail(ATTN_ERR_INVALID_ARG, "slots must be non-null and 8-byte aligned");
    if (rope_cos && (s = check_ints({positions})) != ATTN_OK) return s;
  }
  if ((s = check_device()) != ATTN_OK) return s;
  if (total == 0) return ATTN_OK;
  p.dst[1] = static_cast<uint16_t*>(k_cache);
  p.dst[2] = static_cast<uint16_t*>(v_cache);
  p.positions = positions;
  p.slots = slots;
  p.num_slots = static_cast<long long>(num_pages) * page_size;
  return launch_rope(p, dtype == ATTN_FP16, interleaved, stream);
}

attn_status_t attn_cache_append_fp8(const void* q, void* q_out, const void* k, const void* v,
                                    uint8_t* k_cache, uint8_t* v_cache, float* k_descale, float* v_descale,
                                    const int* block_table, const int* seq_lens, const int* cu_seqlens,
                                    const float* rope_cos, const float* rope_sin,
                                    const float* hadamard_signs, int B, int total, int H, int H_kv, int d,
                                    int rot_dim, int max_pos, int num_pages, int page_size, int max_pages,
                                    const long long* q_strides, const long long* k_strides,
                                    const long long* v_strides, int interleaved, attn_dtype_t dtype,
                                    cudaStream_t stream) {
  g_last_error.clear();
  attn_status_t s;
  if (B < 1 || max_pages < 1) return fail(ATTN_ERR_INVALID_ARG, "B and max_pages must be >= 1");
  if ((s = check_page_size(page_size, 16)) != ATTN_OK) return s;
  if (static_cast<long long>(max_pages) * page_size > 2147483647LL)
    return fail(ATTN_ERR_INVALID_ARG, "max_pages * page_size must be < 2^31");
  RopeKParams p{};
  if ((s = append_common(&p, q, q_out, k, v, k_cache, v_cache, rope_cos, rope_sin, total, H, H_kv, d,
                         rot_dim, max_pos, num_pages, page_size, q_strides, k_strides, v_strides,
                         interleaved, dtype)) != ATTN_OK)
    return s;
  if (d != 128) return fail(ATTN_ERR_UNSUPPORTED, "the FP8 cache supports d = 128");
  if ((s = check_ptrs({k_descale, v_descale})) != ATTN_OK) return s;
  if (hadamard_signs && !aligned16(hadamard_signs))
    return fail(ATTN_ERR_INVALID_ARG, "hadamard_signs not 16-byte aligned");
  if ((s = check_ints({block_table, seq_lens, cu_seqlens})) != ATTN_OK) return s;
  if ((s = check_device()) != ATTN_OK) return s;
  if (total == 0) return ATTN_OK;
  const AppendFp8Params a{k, v, p.st[1], p.sh[1], p.st[2], p.sh[2], k_cache, v_cache, k_descale, v_descale,
                          block_table, seq_lens, cu_seqlens, rope_cos, rope_sin, hadamard_signs, nullptr,
                          B, total, H_kv, num_pages, page_size, max_pages, p.rot, max_pos};
  p.heads[1] = p.heads[2] = 0;
  p.cu_seqlens = cu_seqlens;
  p.seq_lens = seq_lens;
  p.requests = B;
  return launch_append_fp8(a, p, dtype == ATTN_FP16, interleaved, stream);
}

// Sizes of a paged cache that are shared by the calls below.
static attn_status_t check_cache(int num_pages, int page_size, int H_kv, int d, int B, int max_pages, int least_page) {
  attn_status_t s;
  if (B < 1 || max_pages < 1 || num_pages < 1 || H_kv < 1)
    return fail(ATTN_ERR_INVALID_ARG, "B, max_pages, num_pages and H_kv must be >= 1");
  if ((s = check_page_size(page_size, least_page)) != ATTN_OK) return s;
  if (static_cast<long long>(max_pages) * page_size > 2147483647LL)
    return fail(ATTN_ERR_INVALID_ARG, "max_pages * page_size must be < 2^31");
  if (static_cast<double>(num_pages) * page_size * H_kv * d >= 9.0e15)
    return fail(ATTN_ERR_INVALID_ARG, "cache too large");
  return ATTN_OK;
}

attn_status_t attn_cache_append_fp4(const void* q, void* q_out, const void* k, const void* v,
                                    uint8_t* k_cache, uint8_t* v_cache, void* k_descale, void* v_descale,
                                    const long long* slots, const float* rope_cos, const float* rope_sin,
                                    const int* positions, const float* hadamard_signs, int total, int H,
                                    int H_kv, int d, int rot_dim, int max_pos, int num_pages, int page_size,
                                    const long long* q_strides, const long long* k_strides,
                                    const long long* v_strides, int interleaved, attn_dtype_t dtype,
                                    cudaStream_t stream) {
  g_last_error.clear();
  attn_status_t s;
  if ((s = check_page_size(page_size, 16)) != ATTN_OK) return s;
  RopeKParams p{};
  if ((s = append_common(&p, q, q_out, k, v, k_cache, v_cache, rope_cos, rope_sin, total, H, H_kv, d,
                         rot_dim, max_pos, num_pages, page_size, q_strides, k_strides, v_strides,
                         interleaved, dtype)) != ATTN_OK)
    return s;
  if (d == 256) return fail(ATTN_ERR_UNSUPPORTED, "the 4-bit cache supports d = 64 and 128");
  if ((s = check_ptrs({k_descale, v_descale})) != ATTN_OK) return s;
  if (hadamard_signs && !aligned16(hadamard_signs))
    return fail(ATTN_ERR_INVALID_ARG, "hadamard_signs not 16-byte aligned");
  if (total > 0) {
    if (slots == nullptr || (reinterpret_cast<uintptr_t>(slots) & 7u) != 0)
      return fail(ATTN_ERR_INVALID_ARG, "slots must be non-null and 8-byte aligned");
    if (rope_cos && (s = check_ints({positions})) != ATTN_OK) return s;
  }
  if ((s = check_device()) != ATTN_OK) return s;
  if (total == 0) return ATTN_OK;
  const AppendFp4Params a{k, v, p.st[1], p.sh[1], p.st[2], p.sh[2], k_cache, v_cache,
                          static_cast<uint16_t*>(k_descale), static_cast<uint16_t*>(v_descale), slots, positions,
                          rope_cos, rope_sin, hadamard_signs, total, H_kv, num_pages, page_size, p.rot, max_pos};
  p.heads[1] = p.heads[2] = 0;
  p.positions = positions;
  return launch_append_fp4(a, p, d, dtype == ATTN_FP16, interleaved, stream);
}

size_t attn_decode_fp4_workspace_size(int B, int H, int H_kv, int n_q, int d, int max_seqlen) {
  if (B < 1 || H < 1 || H_kv < 1 || H % H_kv != 0 || n_q < 1 || d < 1 || max_seqlen < 1 ||
      (d != 64 && d != 128) || static_cast<long long>(H / H_kv) * n_q > 128)
    return 0;
  return fp4_decode_workspace_bytes(fp4_decode_plan(B, H, H_kv, n_q, d, max_seqlen), d);
}

attn_status_t attn_decode_paged_fp4(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                    const void* k_descale, const void* v_descale, const float* hadamard_signs,
                                    const int* block_table, const int* seq_lens, void* o, float* lse,
                                    void* workspace, size_t workspace_bytes, int B, int H, int H_kv, int n_q,
                                    int d, int num_pages, int page_size, int max_pages, int max_seqlen,
                                    int causal, float softmax_scale, attn_dtype_t dtype,
                                    cudaStream_t stream) {
  g_last_error.clear();
  attn_status_t s;
  if (H < 1 || n_q < 1 || max_seqlen < 1)
    return fail(ATTN_ERR_INVALID_ARG, "H, n_q and max_seqlen must be >= 1");
  if ((s = check_cache(num_pages, page_size, H_kv, d, B, max_pages, 16)) != ATTN_OK) return s;
  if ((s = check_heads(H, H_kv)) != ATTN_OK) return s;
  if (d != 64 && d != 128) return fail(ATTN_ERR_UNSUPPORTED, "the 4-bit decode supports d = 64 and 128");
  if (causal != 0 && causal != 1) return fail(ATTN_ERR_INVALID_ARG, "causal must be 0 or 1");
  if (static_cast<long long>(H / H_kv) * n_q > 128)
    return fail(ATTN_ERR_UNSUPPORTED, "(H / H_kv) * n_q must be <= 128");
  if (static_cast<double>(B) * H * n_q * d >= 2147483648.0)
    return fail(ATTN_ERR_INVALID_ARG, "B*H*n_q*d must be < 2^31");
  if (static_cast<double>(B) * H_kv * ((H / H_kv * n_q + 15) / 16) * (static_cast<double>(max_pages) * page_size / 128 + 8.0) >=
      2147483648.0)
    return fail(ATTN_ERR_UNSUPPORTED,
                "B * H_kv * ceil((H / H_kv) * n_q / 16) * (max_pages * page_size / 128 + 8) must be < 2^31");
  if ((s = check_ptrs({q, k_cache, v_cache, o, lse, workspace, k_descale, v_descale})) != ATTN_OK) return s;
  if (((reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache)) & 31u) != 0)
    return fail(ATTN_ERR_INVALID_ARG, "k_cache and v_cache must be 32-byte aligned");
  if (hadamard_signs && !aligned16(hadamard_signs))
    return fail(ATTN_ERR_INVALID_ARG, "hadamard_signs not 16-byte aligned");
  if ((s = check_ints({block_table, seq_lens})) != ATTN_OK) return s;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(ATTN_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (workspace_bytes < attn_decode_fp4_workspace_size(B, H, H_kv, n_q, d, max_seqlen))
    return fail(ATTN_ERR_INVALID_ARG, "workspace smaller than attn_decode_fp4_workspace_size()");
  if ((s = check_scale(softmax_scale)) != ATTN_OK) return s;
  if ((s = check_dtype(dtype)) != ATTN_OK) return s;
  if ((s = check_device()) != ATTN_OK) return s;
  return launch_decode_fp4({q, k_cache, v_cache, static_cast<const uint16_t*>(k_descale),
                            static_cast<const uint16_t*>(v_descale), hadamard_signs, block_table, seq_lens, o, lse,
                            workspace, B, H, H_kv, n_q, d, num_pages, page_size, max_pages, max_seqlen, causal,
                            softmax_scale, dtype == ATTN_FP16 ? 1 : 0},
                           stream);
}

// The three forms of reading back; bits: 16, 8 or 4 per stored value.
static attn_status_t cache_read(const void* k_cache, const void* v_cache, const void* k_descale,
                                const void* v_descale, const float* signs, const int* block_table,
                                const int* seq_lens, const int* first, const int* cu_seqlens, void* k_out,
                                void* v_out, int B, int n, int H_kv, int d, int num_pages, int page_size,
                                int max_pages, int bits, attn_dtype_t dtype, cudaStream_t stream) {
  attn_status_t s;
  if (n < 0) return fail(ATTN_ERR_INVALID_ARG, "n must be >= 0");
  if ((s = check_cache(num_pages, page_size, H_kv, d, B, max_pages, bits == 16 ? 8 : 16)) != ATTN_OK) return s;
  if (d != 64 && d != 128 && d != 256) return fail(ATTN_ERR_INVALID_ARG, "d must be 64, 128 or 256");
  if (bits == 8 && d != 128) return fail(ATTN_ERR_UNSUPPORTED, "the FP8 cache supports d = 128");
  if (bits == 4 && d == 256) return fail(ATTN_ERR_UNSUPPORTED, "the 4-bit cache supports d = 64 and 128");
  if (static_cast<double>(cu_seqlens ? 1 : B) * n * H_kv * d >= 9.0e15)
    return fail(ATTN_ERR_INVALID_ARG, "output too large");
  if ((s = check_dtype(dtype)) != ATTN_OK) return s;
  if ((s = check_ptrs({k_cache, v_cache})) != ATTN_OK) return s;
  if (bits < 16 && (s = check_ptrs({k_descale, v_descale})) != ATTN_OK) return s;
  if (n > 0 && (s = check_ptrs({k_out, v_out})) != ATTN_OK) return s;
  if (signs && !aligned16(signs)) return fail(ATTN_ERR_INVALID_ARG, "hadamard_signs not 16-byte aligned");
  if ((s = check_ints({block_table, seq_lens})) != ATTN_OK) return s;
  if (first && (s = check_ints({first})) != ATTN_OK) return s;
  if (cu_seqlens && (s = check_ints({cu_seqlens})) != ATTN_OK) return s;
  // blocks read the caches and the rest while others write
  const size_t rows = static_cast<size_t>(num_pages) * page_size * H_kv, out_bytes = (cu_seqlens ? 1ull : B) * n * H_kv * d * 2;
  const size_t scales = bits == 16 ? 0 : bits == 8 ? 4ull * num_pages * H_kv : 2 * rows, b4 = 4 * static_cast<size_t>(B);
  struct Range {
    const void* p;
    size_t bytes;
  };
  const Range all[] = {{k_out, out_bytes}, {v_out, out_bytes}, {k_cache, rows * d * bits / 8}, {v_cache, rows * d * bits / 8},
                       {k_descale, scales}, {v_descale, scales}, {signs, signs ? 4ull * d : 0}, {block_table, b4 * max_pages},
                       {seq_lens, b4}, {first, first ? b4 : 0}, {cu_seqlens, cu_seqlens ? b4 + 4 : 0}};
  for (int i = 0; i < 2; ++i)
    for (int k = i + 1; k < 11; ++k) {
      const uintptr_t x = reinterpret_cast<uintptr_t>(all[i].p), y = reinterpret_cast<uintptr_t>(all[k].p);
      if (all[i].bytes > 0 && all[k].bytes > 0 && x < y + all[k].bytes && y < x + all[i].bytes)
        return fail(ATTN_ERR_INVALID_ARG, "k_out and v_out must not overlap each other or the inputs");
    }
  if ((s = check_device()) != ATTN_OK) return s;
  if (n == 0) return ATTN_OK;
  return launch_cache_read({k_cache, v_cache, k_descale, v_descale, signs, block_table, seq_lens, first, cu_seqlens,
                            k_out, v_out, B, n, H_kv, num_pages, page_size, max_pages},
                           bits, d, dtype == ATTN_FP16, stream);
}

attn_status_t attn_cache_read(const void* k_cache, const void* v_cache, const int* block_table,
                              const int* seq_lens, const int* first, const int* cu_seqlens, void* k_out,
                              void* v_out, int B, int n, int H_kv, int d, int num_pages, int page_size,
                              int max_pages, attn_dtype_t dtype, cudaStream_t stream) {
  g_last_error.clear();
  return cache_read(k_cache, v_cache, nullptr, nullptr, nullptr, block_table, seq_lens, first, cu_seqlens, k_out, v_out,
                    B, n, H_kv, d, num_pages, page_size, max_pages, 16, dtype, stream);
}

attn_status_t attn_cache_read_fp8(const uint8_t* k_cache, const uint8_t* v_cache, const float* k_descale,
                                  const float* v_descale, const float* hadamard_signs, const int* block_table,
                                  const int* seq_lens, const int* first, const int* cu_seqlens, void* k_out,
                                  void* v_out, int B, int n, int H_kv, int d, int num_pages, int page_size,
                                  int max_pages, attn_dtype_t dtype, cudaStream_t stream) {
  g_last_error.clear();
  return cache_read(k_cache, v_cache, k_descale, v_descale, hadamard_signs, block_table, seq_lens, first, cu_seqlens,
                    k_out, v_out, B, n, H_kv, d, num_pages, page_size, max_pages, 8, dtype, stream);
}

attn_status_t attn_cache_read_fp4(const uint8_t* k_cache, const uint8_t* v_cache, const void* k_descale,
                                  const void* v_descale, const float* hadamard_signs, const int* block_table,
                                  const int* seq_lens, const int* first, const int* cu_seqlens, void* k_out,
                                  void* v_out, int B, int n, int H_kv, int d, int num_pages, int page_size,
                                  int max_pages, attn_dtype_t dtype, cudaStream_t stream) {
  g_last_error.clear();
  return cache_read(k_cache, v_cache, k_descale, v_descale, hadamard_signs, block_table, seq_lens, first, cu_seqlens,
                    k_out, v_out, B, n, H_kv, d, num_pages, page_size, max_pages, 4, dtype, stream);
}

attn_status_t attn_merge(const void* o_a, const float* lse_a, const void* o_b, const float* lse_b, void* o,
                         float* lse, int B, int H, int N, int d, int packed, attn_dtype_t dtype,
                         cudaStream_t stream) {
  g_last_error.clear();
  attn_status_t s;
  if ((s = check_shape(B, H, N, d, 0)) != ATTN_OK) return s;
  if (packed != 0 && packed != 1) return fail(ATTN_ERR_INVALID_ARG, "packed must be 0 or 1");
  if (packed && B != 1) return fail(ATTN_ERR_INVALID_ARG, "a packed batch has B = 1");
  if ((s = check_dtype(dtype)) != ATTN_OK) return s;
  if ((s = check_ptrs({o_a, o_b, o, lse_a, lse_b, lse})) != ATTN_OK) return s;
  const size_t rows = static_cast<size_t>(B) * H * N;
  struct Range {
    const void* p;
    size_t bytes;
  };
  // a result may be an input's own memory, whole, or none of it
  const Range ins[] = {{o_a, rows * d * 2}, {o_b, rows * d * 2}, {lse_a, rows * 4}, {lse_b, rows * 4}};
  const Range outs[] = {{o, rows * d * 2}, {lse, rows * 4}};
  for (int i = 0; i < 2; ++i)
    for (int k = 0; k < 4; ++k) {
      const uintptr_t x = reinterpret_cast<uintptr_t>(outs[i].p), y = reinterpret_cast<uintptr_t>(ins[k].p);
      if (x < y + ins[k].bytes && y < x + outs[i].bytes && !(x == y && i == k / 2))
        return fail(ATTN_ERR_INVALID_ARG, "o and lse must be an input's o or lse, or not overlap the inputs");
    }
  {
    const uintptr_t x = reinterpret_cast<uintptr_t>(o), y = reinterpret_cast<uintptr_t>(lse);
    if (x < y + outs[1].bytes && y < x + outs[0].bytes)
      return fail(ATTN_ERR_INVALID_ARG, "o and lse must not overlap");
  }
  if ((s = check_device()) != ATTN_OK) return s;
  return launch_merge({o_a, lse_a, o_b, lse_b, o, lse, static_cast<long long>(rows), H, N, packed}, d,
                      dtype == ATTN_FP16, stream);
}

attn_status_t attn_selftest_wait_timeout(unsigned limit_us, cudaStream_t stream) {
  g_last_error.clear();
  attn_status_t s;
  if (limit_us < 1 || limit_us > 1000000)
    return fail(ATTN_ERR_INVALID_ARG, "limit_us must be in [1, 1000000]");
  if ((s = check_device()) != ATTN_OK) return s;
  int* status = device_status_word();
  if (!status) return fail(ATTN_ERR_CUDA, "status word unavailable");
  selftest_wait_kernel<<<1, 32, 0, stream>>>(status, static_cast<uint64_t>(limit_us) * 1000ull);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail_cuda(e, "self-test launch");
  return ATTN_OK;
}

attn_status_t attn_get_device_status(cudaStream_t stream) {
  g_last_error.clear();
  attn_status_t s;
  if ((s = check_device()) != ATTN_OK) return s;
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return fail_cuda(e, "cudaStreamSynchronize");
  int* word = device_status_word();
  if (!word) return fail(ATTN_ERR_CUDA, "status word unavailable");
  int value = 0;
  e = cudaMemcpy(&value, word, sizeof(int), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return fail_cuda(e, "reading the status word");
  if (value == 0) return ATTN_OK;
  const int zero = 0;
  e = cudaMemcpy(word, &zero, sizeof(int), cudaMemcpyHostToDevice);
  if (e != cudaSuccess) return fail_cuda(e, "clearing the status word");
  static const char* roles[] = {"?",        "load",   "mma",
                                "softmax",  "epilogue", "reduce",
                                "shared-memory alignment", "self-test"};
  const int role = (value >> 8) & 0xF;
  if (value == kDevBadSeqlens)
    return fail(ATTN_ERR_INVALID_ARG,
                "cu_seqlens inconsistent (an entry outside [0, total], decreasing, or a sequence "
                "longer than max_seqlen), a kv_lens entry outside [0, N_k], or a decode seq_lens / "
                "block_table entry out of range; "
                "those sequences or pages were skipped");
  if (value == kDevBadTables)
    return fail(ATTN_ERR_INVALID_ARG,
                "request lengths, free pages, slots, table entries or positions that do not fit the "
                "block table, the cache or the rotary tables; those tokens were skipped, rows of "
                "positions past the rotary tables written unrotated");
  return fail(ATTN_ERR_TIMEOUT, std::string("kernel wait timed out in role ") +
                                    (role < 8 ? roles[role] : "?") + " (code " +
                                    std::to_string(value) + ")");
}

}  // extern "C"
