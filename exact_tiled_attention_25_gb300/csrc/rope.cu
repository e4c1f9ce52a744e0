// Rotary position embedding: the rotation of Q and K rows, and the tables of
// cosines and sines it reads, stretched for long contexts.
//
// "FlashAttention-3: Hopper Asynchrony and FP8 Attention", section "FP8 accuracy
// controls", fuses the rotation with the Hadamard transform of the FP8 pre-pass
// (fp8.cu) and leaves its definition to the caller's tables; this is the same
// rotation for the 16-bit kernels, forward and inverse.
#include "common.h"
#include "rope.cuh"

namespace attn {
namespace {

template <bool FP16, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeKParams p) {
  rope_block<FP16, INTERLEAVED>(p, blockIdx.x, blockIdx.y);
}

// Table row r holds position p = first + r.  Frequency theta_i = base^(-2i/rot)
// makes r_i = orig_len * theta_i / (2 pi) turns within the original context; it
// is kept where r_i >= high, divided by `factor` where r_i <= low, and blended
// linearly in r_i between (interpolation "by parts", section 3.2 of "YaRN:
// Efficient Context Window Extension of Large Language Models",
// arXiv:2309.00071); orig_len = 0 divides every frequency (position
// interpolation, arXiv:2306.15595).  The angle p * theta reaches 1e6 rad, where
// a float32 angle would be off by 0.06, so theta and the angle are float64,
// reduced to [-pi, pi] before the float32 sine and cosine.
// Bound: the writes, 8 bytes per entry; the float64 work is one product, one
// rounding and one fused multiply-add per entry, the power one per column.
__global__ void __launch_bounds__(256)
    rope_table_kernel(float* __restrict__ cos_out, float* __restrict__ sin_out, long long n, int half,
                      double base, double factor, double orig_len, double low, double high,
                      float attn_factor, long long first, int rows_per_block) {
  const int cols = min(half, 256);
  const int lanes = 256 / cols;                     // rows written at a time
  const int i0 = threadIdx.x % cols;
  const int sub = threadIdx.x / cols;
  if (sub >= lanes) return;
  const long long r0 = static_cast<long long>(blockIdx.x) * rows_per_block;
  const long long r1 = r0 + rows_per_block < n ? r0 + rows_per_block : n;
  for (int i = i0; i < half; i += cols) {
    double theta = pow(base, -static_cast<double>(i) / half);
    double keep = 0.0;
    if (orig_len > 0.0) {
      keep = (orig_len * theta * 0.15915494309189533577 - low) / (high - low);
      keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
    }
    theta *= keep + (1.0 - keep) / factor;
    for (long long r = r0 + sub; r < r1; r += lanes) {
      const double a = static_cast<double>(first + r) * theta;
      const double turns = rint(a * 0.15915494309189533577);
      const float x = static_cast<float>(fma(turns, -6.28318530717958647693, a));
      float sn, cs;
      sincosf(x, &sn, &cs);
      cos_out[r * half + i] = cs * attn_factor;
      sin_out[r * half + i] = sn * attn_factor;
    }
  }
}

}  // namespace

attn_status_t launch_rope(RopeKParams p, int fp16, int interleaved, cudaStream_t stream) {
  p.status = device_status_word();
  if (!p.status) return fail(ATTN_ERR_CUDA, "status word unavailable");
  const RopeGrid g = rope_grid(&p);
  if (g.columns > 2147483647LL || g.chunks > 65535)
    return fail(ATTN_ERR_UNSUPPORTED, "grid dimension limit exceeded");
  const dim3 grid(static_cast<unsigned>(g.columns), g.chunks);
  if (fp16) {
    if (interleaved) rope_kernel<true, true><<<grid, kRopeThreads, 0, stream>>>(p);
    else rope_kernel<true, false><<<grid, kRopeThreads, 0, stream>>>(p);
  } else {
    if (interleaved) rope_kernel<false, true><<<grid, kRopeThreads, 0, stream>>>(p);
    else rope_kernel<false, false><<<grid, kRopeThreads, 0, stream>>>(p);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail_cuda(e, "rotary kernel launch");
  return ATTN_OK;
}

attn_status_t launch_rope_table(float* cos_out, float* sin_out, long long n, int rot, double base,
                                double factor, long long orig_len, double low, double high,
                                double attn_factor, long long first, cudaStream_t stream) {
  // a block computes its columns' powers once, for up to 64 rows
  long long rows = (n + 152 * 8 - 1) / (152 * 8);
  rows = rows < 8 ? 8 : rows > 64 ? 64 : rows;
  const long long blocks = (n + rows - 1) / rows;
  if (blocks > 2147483647LL) return fail(ATTN_ERR_UNSUPPORTED, "grid dimension limit exceeded");
  rope_table_kernel<<<static_cast<unsigned>(blocks), 256, 0, stream>>>(
      cos_out, sin_out, n, rot / 2, base, factor, static_cast<double>(orig_len), low, high,
      static_cast<float>(attn_factor), first, static_cast<int>(rows));
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail_cuda(e, "rotary table launch");
  return ATTN_OK;
}

}  // namespace attn
