// Two partial attentions of the same queries over disjoint keys, joined by their
// log-sum-exps:  L = log(e^La + e^Lb),  O = e^(La - L) Oa + e^(Lb - L) Ob.
//
// A row's d / 8 threads (16 bytes of each output) are lanes of one warp and read the two
// log-sum-exps before one of them stores L, so the results may replace either input.
// Bound: DRAM, 6 d + 12 bytes a row: 262,144 rows of d = 128 take 30.7 us (6.7 TB/s), 2048 rows 1.8.
#include <cmath>

#include "common.h"
#include "rope.cuh"

namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 2;          // rows of a thread, loaded before the first is stored

struct Weights {
  float a, b, lse;
};
// A part without keys (L = -inf) has weight 0; two of them give O = 0 and L = -inf.
__device__ __forceinline__ Weights weights(float la, float lb) {
  const float m = fmaxf(la, lb);
  if (m == -INFINITY && la == lb) return {0.f, 0.f, -INFINITY};
  const float ea = expf(la - m), eb = expf(lb - m), sum = ea + eb;
  return {__fdividef(ea, sum), __fdividef(eb, sum), m + logf(sum)};
}

// Rows are counted in the outputs' order: (b, h, n), or packed (token, h) with log-sum-exps
// [H, tokens].
template <int D, bool FP16, bool PACKED>
__global__ void __launch_bounds__(kThreads)
    merge_kernel(const uint4* oa, const float* la, const uint4* ob, const float* lb, uint4* o, float* lse,
                 long long rows, int H, long long tokens) {
  constexpr int L = D / 8;
  const int u = threadIdx.x % L;
  const long long r0 = static_cast<long long>(blockIdx.x) * (kThreads / L * kRows) + threadIdx.x / L;
  wait_for_previous_kernel();
  uint4 a[kRows], b[kRows];
  float xa[kRows], xb[kRows];
  long long at[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const long long r = r0 + k * (kThreads / L);
    a[k] = b[k] = make_uint4(0u, 0u, 0u, 0u);
    xa[k] = xb[k] = -INFINITY;
    at[k] = 0;
    if (r >= rows) continue;
    at[k] = PACKED ? (r % H) * tokens + r / H : r;
    a[k] = __ldcg(oa + r * L + u);
    b[k] = __ldcg(ob + r * L + u);
    xa[k] = __ldcg(la + at[k]);
    xb[k] = __ldcg(lb + at[k]);
  }
  __syncwarp();
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const long long r = r0 + k * (kThreads / L);
    if (r >= rows) continue;
    const Weights w = weights(xa[k], xb[k]);
    float fa[8], fb[8], x[8];
    unpack16<FP16>(a[k], fa);
    unpack16<FP16>(b[k], fb);
    // what an empty part holds does not matter; of another, however small its weight, infinities and NaN show
    const bool has_a = xa[k] != -INFINITY, has_b = xb[k] != -INFINITY;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (has_a ? w.a * fa[i] : 0.f) + (has_b ? w.b * fb[i] : 0.f);
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = FP16 ? cvt_pack_f16(x[2 * i], x[2 * i + 1]) : cvt_pack_bf16(x[2 * i], x[2 * i + 1]);
    o[r * L + u] = make_uint4(p[0], p[1], p[2], p[3]);
    if (u == 0) lse[at[k]] = w.lse;
  }
}

template <int D, bool FP16>
attn_status_t launch_t(const MergeParams& p, cudaStream_t stream) {
  constexpr int per_block = kThreads / (D / 8) * kRows;
  const long long blocks = (p.rows + per_block - 1) / per_block;
  if (blocks > 2147483647LL) return fail(ATTN_ERR_UNSUPPORTED, "grid dimension limit exceeded");
  auto kern = p.packed ? merge_kernel<D, FP16, true> : merge_kernel<D, FP16, false>;
  const cudaError_t e = launch_dependent(
      kern, dim3(static_cast<unsigned>(blocks)), kThreads, 0, stream, 0, static_cast<const uint4*>(p.o_a), p.lse_a,
      static_cast<const uint4*>(p.o_b), p.lse_b, static_cast<uint4*>(p.o), p.lse, p.rows, p.H, p.tokens);
  return e == cudaSuccess ? ATTN_OK : fail_cuda(e, "merge kernel launch");
}

}  // namespace

attn_status_t launch_merge(const MergeParams& p, int d, int fp16, cudaStream_t stream) {
  switch (d) {
    case 64: return fp16 ? launch_t<64, true>(p, stream) : launch_t<64, false>(p, stream);
    case 128: return fp16 ? launch_t<128, true>(p, stream) : launch_t<128, false>(p, stream);
  }
  return fp16 ? launch_t<256, true>(p, stream) : launch_t<256, false>(p, stream);
}

}  // namespace attn
