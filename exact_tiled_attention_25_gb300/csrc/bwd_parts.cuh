// Pieces of the backward pass that bwd.cu and cross_bwd.cu share: the tile
// configuration and the pre-pass.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.h"
#include "sm103_prims.cuh"

namespace attn {
namespace {

constexpr int kSmemLimit = 232448;
constexpr float kLog2e = 1.4426950408889634f;

__host__ __device__ constexpr int cmin(int a, int b) { return a < b ? a : b; }

template <int D>
struct BwdCfg {
  static constexpr int BM = 128;                 // query rows per step
  static constexpr int BN = 128;                 // keys per CTA
  static constexpr int CH = D / 64;              // 128-byte chunks per row
  static constexpr int CHUNK = 128 * 128;        // one 128-row x 128-byte chunk
  static constexpr int TILE = 128 * D * 2;       // a K, V, Q or dO tile
  // Q_i (with its row vectors) and dO_i have rings of their own: Q_i is read
  // by S^T(i) early and dK late, dO_i only by dP^T(i) and dV.  At d = 128 one
  // dO slot is all that fits next to the dQ staging buffers.
  static constexpr int NQS = 2;                  // Q ring slots
  static constexpr int NDS = (D == 128) ? 1 : 2; // dO ring slots
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = TILE;
  static constexpr int OFF_Q = 2 * TILE;
  static constexpr int OFF_DO = OFF_Q + NQS * TILE;
  static constexpr int OFF_DS = OFF_DO + NDS * TILE;      // dS^T, 128 keys x 128 queries
  // dQ staging: one 32-query x 32-column float32 box (4 KB, 128-byte swizzle)
  // per reduce warp, handed to a TMA reduce-add into the float32 accumulator
  static constexpr int STG_BOX = 32 * 32 * 4;
  static constexpr int OFF_STG = OFF_DS + 2 * CHUNK;
  static constexpr int OFF_LD = OFF_STG + 8 * STG_BOX;    // per Q slot: L*log2e[128], D[128]
  static constexpr int OFF_BAR = OFF_LD + NQS * 1024;
  static constexpr int NEED = OFF_BAR + 256;
  static constexpr int SMEM_BYTES = cmin(kSmemLimit, NEED + 1024);
  static constexpr int SLACK = SMEM_BYTES - NEED;   // room to align the base to 1024
  // TMEM columns: S^T/P^T [0,128), dP^T/dS^T [128,256), dV, dK.  At d = 128
  // there is no room left, so dQ reuses the dP^T columns (after dK has read
  // dS^T there); at d = 64 dQ has its own columns.  dQ is stored with one
  // query per TMEM lane.
  static constexpr bool DQ_IN_DP = (D == 128);
  static constexpr uint32_t S_COL = 0;
  static constexpr uint32_t DP_COL = 128;
  static constexpr uint32_t DV_COL = 256;
  static constexpr uint32_t DK_COL = 256 + D;
  static constexpr uint32_t DQ_COL = DQ_IN_DP ? DP_COL : 256 + 2 * D;
  // Warps 0-7: two compute warpgroups (one per half of the 128 query columns);
  // warps 8-15: two reduce warpgroups (one per half of dQ's columns);
  // warp 16: TMA producer; warp 17: MMA issuer.
  static constexpr int THREADS = 576;
  static constexpr int LOAD_WARP = 16;
  static constexpr int MMA_WARP = 17;
  // Packed 16-bit P^T / dS^T of query half h sit in columns [64 h, 64 h + 32) of
  // the S^T / dP^T region, inside the half's own fp32 columns, so each
  // warpgroup overwrites only scores it has already read.
  __host__ __device__ static constexpr uint32_t half_col(int kk) {
    return 64u * static_cast<uint32_t>(kk / 4) + 8u * static_cast<uint32_t>(kk % 4);
  }
  static_assert(DQ_COL + D <= 512 && DK_COL + D <= 512, "TMEM overflow");
  static_assert(SLACK >= 0, "shared memory overflow");
  static_assert(OFF_STG % 1024 == 0, "staging boxes need 1024-byte alignment (swizzle atoms)");
};

// Sequence b of a packed batch: first token and length, or false when its
// offsets do not fit (outside [0, total], decreasing, or longer than max_len).
__device__ __forceinline__ bool packed_seq(const int* cu, int b, int total, int max_len, int& s0,
                                           int& len) {
  s0 = cu[b];
  const int e = cu[b + 1];
  if (s0 < 0 || e < s0 || e > total || e - s0 > max_len) return false;
  len = e - s0;
  return true;
}

// ------------------------------------------------------------------ prep ----
// One group of D/8 lanes per row; each lane holds 8 consecutive elements.
// Rows of O, dO and dQ are [B, H, N, d] or, for a packed batch (PACKED),
// [total, H, d] with LSE [H, total].
// CHAINED: a dependent launch, so O, dO and the LSE, which the kernel before may have
// written, are read past the L1 cache; the main kernel may start its prologue meanwhile.
template <int D, bool FP16, bool PACKED, bool CHAINED = false>
__global__ void __launch_bounds__(256)
    bwd_prep_kernel(const uint16_t* __restrict__ o, const uint16_t* __restrict__ dout,
                    const float* __restrict__ lse, float* __restrict__ lse2,
                    float* __restrict__ delta, float* __restrict__ dq_acc, int N, int Npad,
                    long long total_rows_pad, int H, const int* __restrict__ cu_seqlens,
                    int total) {
  if constexpr (CHAINED) {
    wait_for_previous_kernel();
    release_dependents();
  }
  constexpr int L = D / 8;
  constexpr int ROWS_PER_WARP = 32 / L;
  const int lane = threadIdx.x & 31;
  const int sub = lane / L;
  const int li = lane % L;
  const long long warp_global = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) / 32;
  const long long prow = warp_global * ROWS_PER_WARP + sub;   // padded row index
  if (prow >= total_rows_pad) return;
  const long long bh = prow / Npad;
  const int n = static_cast<int>(prow - bh * Npad);
  int len = N;
  long long row, lrow;     // row of O / dO / dQ, index into LSE
  if constexpr (PACKED) {
    const int b = static_cast<int>(bh / H), h = static_cast<int>(bh % H);
    int s0 = 0;
    if (!packed_seq(cu_seqlens, b, total, N, s0, len)) len = 0;   // reported by the main kernel
    row = (static_cast<long long>(s0) + n) * H + h;
    lrow = static_cast<long long>(h) * total + s0 + n;
  } else {
    row = bh * N + n;
    lrow = row;
  }
  float acc = 0.f;
  if (n < len) {
    const uint4* const ao = reinterpret_cast<const uint4*>(o + row * D) + li;
    const uint4* const bo = reinterpret_cast<const uint4*>(dout + row * D) + li;
    const uint4 a = CHAINED ? __ldcg(ao) : *ao;
    const uint4 b = CHAINED ? __ldcg(bo) : *bo;
    const uint32_t av[4] = {a.x, a.y, a.z, a.w};
    const uint32_t bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float2 fa, fb;
      if (FP16) {
        fa = __half22float2(*reinterpret_cast<const __half2*>(&av[e]));
        fb = __half22float2(*reinterpret_cast<const __half2*>(&bv[e]));
      } else {
        fa = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&av[e]));
        fb = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&bv[e]));
      }
      acc = fmaf(fa.x, fb.x, acc);
      acc = fmaf(fa.y, fb.y, acc);
    }
    float4* z = reinterpret_cast<float4*>(dq_acc + row * D) + 2 * li;
    z[0] = make_float4(0.f, 0.f, 0.f, 0.f);
    z[1] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll
  for (int off = L / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
  if (li == 0) {
    // stored negated so the main kernel adds them with packed f32x2 FMAs
    delta[prow] = (n < len) ? -acc : 0.f;
    lse2[prow] = (n < len) ? -(CHAINED ? __ldcg(lse + lrow) : lse[lrow]) * kLog2e : -INFINITY;
  }
}

}  // namespace
}  // namespace attn
