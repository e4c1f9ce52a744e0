// Host-side internals shared by the kernel translation units and the C ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <string>

#include "../../include/attn_gb300.h"

namespace attn {

// Record a detail message for attn_last_error() and return `code`.
attn_status_t fail(attn_status_t code, const std::string& msg);
attn_status_t fail_cuda(cudaError_t err, const char* what);

// Device address of the status word in the current context (nullptr if the
// lookup fails).
int* device_status_word();

// Compute capability 10.3 check of the current device (ATTN_ERR_ARCH if not).
attn_status_t check_device();

// 3-D tensor map over a contiguous [planes][rows][inner] array with a
// (box_inner x box_rows x 1) box and 128-byte swizzle.  elem_bytes is 1 or 2
// (raw bytes / 16-bit words), or 4 (float32, the type a reduce-add needs).
attn_status_t make_tmap_3d(CUtensorMap* map, const void* base, int elem_bytes, uint64_t inner,
                           uint64_t rows, uint64_t planes, uint32_t box_inner,
                           uint32_t box_rows);

// 4-D map over {d, rows, heads, batches} with byte strides for rows, heads and
// batches (each a multiple of 16); box {box_inner, box_rows, box_heads, 1},
// 128-byte swizzle.  Covers [B, H, N, d] and packed [total, H, d] alike.
attn_status_t make_tmap_4d(CUtensorMap* map, const void* base, int elem_bytes, uint64_t inner,
                           uint64_t rows, uint64_t heads, uint64_t batches, uint64_t row_bytes,
                           uint64_t head_bytes, uint64_t batch_bytes, uint32_t box_inner,
                           uint32_t box_rows, uint32_t box_heads = 1);

// Launch a kernel that may start before the stream's previous kernel has ended (it
// calls wait_for_previous_kernel() before it uses that one's results), in clusters of
// `cluster` blocks when that is given.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t stream,
                             int cluster, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Opt a kernel into more than 48 KB of dynamic shared memory (once per kernel).
attn_status_t set_smem(const void* kernel, int bytes);

struct FwdParams {
  const void* q;
  const void* k;
  const void* v;
  void* o;
  float* lse;
  int B, H, N, d;     // N: sequence length, or the longest one of a packed batch
  int H_kv;           // key/value heads (H % H_kv == 0)
  const int* cu_seqlens;   // device [B + 1] for a packed batch, else nullptr
  int total;          // tokens of a packed batch (cu_seqlens[B])
  int causal;
  float scale;
  int fp16;   // 0 = bf16, 1 = fp16
  int N_k = 0;                     // cross attention: keys per sequence (N counts queries)
  const int* kv_lens = nullptr;    // cross attention: device [B] keys seen, or nullptr (all N_k)
};

struct BwdParams {
  const void* q;
  const void* k;
  const void* v;
  const void* o;
  const void* dout;
  const float* lse;
  void* dq;
  void* dk;
  void* dv;
  float* dq_acc;   // float32 scratch in dQ's layout
  float* lse2;     // [B, H, Npad] float32 scratch: -LSE * log2(e), -inf padding
  float* delta;    // [B, H, Npad] float32 scratch: -rowsum(dO * O), 0 padding
  int B, H, N, d;  // N: sequence length, or the longest one of a packed batch
  int H_kv;        // key/value heads (H % H_kv == 0)
  const int* cu_seqlens;   // device [B + 1] for a packed batch, else nullptr
  int total;       // tokens of a packed batch
  int causal;
  float scale;
  int fp16;
  int N_k = 0;                     // cross attention, as in FwdParams
  const int* kv_lens = nullptr;
};

struct Fp8QuantParams {
  const void* src[3];                // float32, or bfloat16 when in_bf16
  uint8_t* dst[3];
  float* descale[3];
  const float* signs;
  int B, H, N, d;
  int per_tensor;
  const float* rope_cos = nullptr;   // [N, d/2] rotary tables (block mode), or nullptr
  const float* rope_sin = nullptr;
  int H_kv = 0;                      // heads of K and V (0: H)
  const int* cu_seqlens = nullptr;   // packed batch: device [B + 1] offsets (N = longest)
  int total = 0;                     // packed batch: tokens
  int in_bf16 = 0;                   // inputs are bfloat16 (block and per-tensor modes)
};

struct Fp8FwdParams {
  const uint8_t* q8;
  const uint8_t* k8;
  const uint8_t* v8;
  const float* q_descale;
  const float* k_descale;
  const float* v_descale;
  void* o;
  float* lse;
  int B, H, N, d;
  int causal;
  float scale;
  int H_kv;   // heads of K and V (H % H_kv == 0)
  const int* cu_seqlens = nullptr;   // packed batch: device [B + 1] offsets (N = longest)
  int total = 0;                     // packed batch: tokens
  int exp2_poly = -1;                // sixteenths of the exponentials on the FMA pipe (0, 1, 2, 4, 6, 8); -1: the library's choice
};

attn_status_t launch_fwd(const FwdParams& p, cudaStream_t stream);
// exp2_poly2 and ex2.approx on the same n inputs (diagnostic).
attn_status_t launch_exp2_selftest(const float* x, float* y_poly, float* y_mufu, long long n,
                                   cudaStream_t stream);
// Schedule variants of the forward kernel (ATTN_SCHED_* flags), for measurement.
attn_status_t launch_fwd_sched(const FwdParams& p, int sched, cudaStream_t stream);
// Persistent forward (cluster launch control) for packed causal batches.
attn_status_t launch_fwd_persistent(const FwdParams& p, cudaStream_t stream);
attn_status_t launch_bwd(const BwdParams& p, cudaStream_t stream);
// Cross attention (N_k keys): one query tile pair per CTA, and its backward on `ctas`
// CTAs with `part` for their partial dK and dV.
attn_status_t launch_cross_fwd(const FwdParams& p, cudaStream_t stream);
attn_status_t launch_cross_bwd(const BwdParams& p, float* part, int ctas, cudaStream_t stream);
attn_status_t launch_fp8_quantize(const Fp8QuantParams& p, cudaStream_t stream);
attn_status_t launch_fwd_fp8(const Fp8FwdParams& p, cudaStream_t stream);

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Backward scratch layout: dQ accumulator, then L*log2(e) and D, each padded
// to a multiple of 128 rows per head; every part 256-byte aligned.
struct BwdWorkspace {
  size_t dq_acc, lse2, delta, total;
};
// dq_rows: rows of d floats in the dQ accumulator; rows_pad: entries of each
// padded row vector.
inline BwdWorkspace bwd_workspace_layout_rows(size_t dq_rows, size_t rows_pad, int d) {
  const size_t rows = dq_rows;
  BwdWorkspace w;
  w.dq_acc = 0;
  w.lse2 = align_up(rows * d * sizeof(float), 256);
  w.delta = w.lse2 + align_up(rows_pad * sizeof(float), 256);
  w.total = w.delta + align_up(rows_pad * sizeof(float), 256);
  return w;
}

inline BwdWorkspace bwd_workspace_layout(int B, int H, int N, int d) {
  return bwd_workspace_layout_rows(static_cast<size_t>(B) * H * N,
                                   static_cast<size_t>(B) * H * ((static_cast<size_t>(N) + 127) / 128 * 128), d);
}

// A packed batch: dQ accumulator [total, H, d]; row vectors padded per (b, h)
// to the longest sequence.
inline BwdWorkspace bwd_workspace_layout_packed(int B, int max_seqlen, int total, int H, int d) {
  return bwd_workspace_layout_rows(static_cast<size_t>(total) * H,
                                   static_cast<size_t>(B) * H *
                                       ((static_cast<size_t>(max_seqlen) + 127) / 128 * 128), d);
}

// Paged decode (few new query tokens per sequence against a paged cache).
struct DecodeParams {
  const void* q;            // [B, H, n_q, d]
  const void* k_cache;      // [num_pages, page_size, H_kv, d]
  const void* v_cache;
  const int* block_table;   // [B, max_pages]
  const int* seq_lens;      // [B]
  void* o;                  // [B, H, n_q, d]
  float* lse;               // [B, H, n_q]
  float* o_part;            // workspace: [B, H, n_q, splits, d] float32
  float* lse_part;          // workspace: [B, H, n_q, splits] float32
  int B, H, H_kv, n_q, d;
  int num_pages, page_size, max_pages, max_seqlen;
  int causal;
  float scale;
  int fp16;
  // e4m3 cache (d = 128): codes in k_cache / v_cache, one float32 descale per
  // (physical page, key/value head), optional key-transform signs
  int fp8 = 0;
  const float* k_descale = nullptr;   // [num_pages, H_kv]
  const float* v_descale = nullptr;
  const float* signs = nullptr;       // [d] of +-1, or nullptr
};

// Key-range splits of a decode call, each a whole number of 128-key tiles.
// One CTA runs per SM at a time, so the split size minimises the modelled time
// ceil(CTAs / 152) waves x (tiles per CTA + about 1.5 tiles of per-CTA start-up
// and drain), trading the last wave's idle SMs against start-up costs.
struct DecodeSplits {
  int splits, tiles_per_split;
};
inline DecodeSplits decode_splits(int B, int H_kv, int max_seqlen) {
  const int ntiles = (max_seqlen + 127) / 128;
  const long long base = static_cast<long long>(B) * H_kv;
  int best_tps = ntiles;
  double best = 1e300;
  for (int tps = 1; tps <= ntiles; ++tps) {
    const long long splits = (ntiles + tps - 1) / tps;
    if (tps > 1 && (ntiles + tps - 2) / (tps - 1) == splits) continue;   // same split count
    const long long waves = (base * splits + 151) / 152;
    const double cost = static_cast<double>(waves) * (tps + 1.5);
    if (cost < best) {
      best = cost;
      best_tps = tps;
    }
  }
  return {(ntiles + best_tps - 1) / best_tps, best_tps};
}

inline size_t decode_workspace_bytes(int B, int H, int H_kv, int n_q, int d, int max_seqlen) {
  const DecodeSplits sp = decode_splits(B, H_kv, max_seqlen);
  const size_t rows = static_cast<size_t>(B) * H * n_q * sp.splits;
  return align_up(rows * d * sizeof(float), 256) + align_up(rows * sizeof(float), 256);
}

attn_status_t launch_decode(const DecodeParams& p, cudaStream_t stream);

// How a cross-attention forward runs.  ctas > 0: the rows kernel (cross.cu) on tiles of
// 128 query rows of one key/value head (its G * N_q rows together), that many CTAs
// sharing the tiles of all keys, or in clusters of `cluster` CTAs, one for each
// query tile's keys; ctas = 0: the forward kernel (fwd.cu), one CTA per 256 query rows of
// one query head with all keys.
struct CrossPlan {
  int ctas, qtiles, cluster;
};
constexpr int kCrossMaxB = 2048;   // batch entries of the rows kernel (8 bytes of shared memory each)
// The smallest of three modelled times, in microseconds, fitted to the kernels at d = 64
// and 128, N_k = 512 .. 4096 and N_q = 1 .. 1024 (bfloat16, K and V in L2):
//  forward: waves of 152 CTAs x (3.5 + 1.4 or 1.55 per key tile), a tenth more per
//           tile when both of a CTA's query tiles are in use;
//  shared:  a start and a merge, the tiles of one CTA's share, and 2 or more for
//           every segment it finishes (its output leaves tensor memory row by row);
//  cluster: waves of the clusters that run at a time (they do not fill every SM: 152, 76,
//           46, 36, 28, 23, 15 and 15 of 1 to 8 CTAs) x (a start, one CTA's tiles of its
//           segment and their merge).
// 16 heads, N_k = 4096, d = 128: N_q = 1: 51 us (forward), 17 (rows); 512: 56, 44;
// 1024: 57, 74.  8 x 16 heads, N_k = 512: N_q = 1: 10, 13.
inline CrossPlan cross_plan(int B, int H, int H_kv, int N_q, int N_k, int d) {
  if (d > 128) return {0, 0, 0};
  const long long rows = static_cast<long long>(H / H_kv) * N_q;
  const long long qtiles = (rows + 127) / 128, ktiles = (N_k + 127) / 128;
  const long long segs = static_cast<long long>(B) * H_kv * qtiles, tiles = segs * ktiles;
  const long long fwd_ctas = static_cast<long long>(B) * H * ((N_q + 255) / 256);
  const double fwd = static_cast<double>((fwd_ctas + 151) / 152) *
                     (3.5 + ktiles * (d == 64 ? 1.4 : 1.55) * (N_q > 128 ? 1.1 : 1.0));
  const bool few = rows <= 16;
  const double share = static_cast<double>((tiles + 151) / 152), ends = static_cast<double>((segs + 151) / 152);
  const double shared = d == 64 ? 9.0 + share * (few ? 0.75 : 0.95) + ends * (few ? 0.3 : 2.0)
                                : (few ? 10.0 : 12.0) + share * (few ? 1.0 : 1.16) + ends * (few ? 0.3 : 2.7);
  if (tiles > 2147483647LL || H_kv * qtiles > 2147483647LL || segs > 2147483647LL / 8) return {0, 0, 0};
  CrossPlan plan{0, static_cast<int>(qtiles), 0};
  double best = fwd;
  if (shared < best && B <= kCrossMaxB) {
    best = shared;
    plan.ctas = static_cast<int>(tiles < 152 ? tiles : 152);
  }
  constexpr int at_a_time[9] = {0, 152, 76, 46, 36, 28, 23, 15, 15};
  for (int c = 1; c <= 8; ++c) {
    const double waves = static_cast<double>((segs + at_a_time[c] - 1) / at_a_time[c]);
    const double t = waves * (d == 64 ? (few ? 6.5 : 8.5) + (ktiles + c - 1) / c * (few ? 0.75 : 0.95)
                                      : (few ? 7.5 : 10.7) + (ktiles + c - 1) / c * (few ? 1.0 : 1.16));
    if (t < best) {
      best = t;
      plan.cluster = c;
      plan.ctas = static_cast<int>(segs * c);
    }
  }
  return plan;
}
// The rows kernel's float32 partial O and log-sum-exps, two per CTA.
inline size_t cross_workspace_bytes(int H, int H_kv, int N_q, int d, const CrossPlan& plan) {
  if (plan.ctas <= 1 || plan.cluster > 0) return 0;
  const size_t seg = static_cast<size_t>(H / H_kv) * N_q;
  const size_t rows = 2ull * plan.ctas * (seg < 128 ? seg : 128);
  return align_up(rows * d * sizeof(float), 256) + align_up(rows * sizeof(float), 256);
}
attn_status_t launch_cross_rows(const FwdParams& p, const CrossPlan& plan, void* workspace,
                                cudaStream_t stream);

// The cross-attention backward's CTAs, sharing the steps of all key tiles (a step: a key
// tile with a query tile of one query head), and its scratch: the backward's, then
// two float32 pairs of dV and dK tiles per CTA.
struct CrossBwdPlan {
  long long steps;      // with every key seen
  int ctas;
  BwdWorkspace w;
  size_t part, total;   // byte offset of the pairs, bytes of all
};
inline CrossBwdPlan cross_bwd_plan(int B, int H, int N_q, int N_k, int d) {
  CrossBwdPlan c;
  c.steps = static_cast<long long>(B) * H * ((N_q + 127) / 128) * ((N_k + 127) / 128);
  c.ctas = static_cast<int>(c.steps < 152 ? c.steps : 152);
  c.w = bwd_workspace_layout(B, H, N_q, d);
  c.part = c.w.total;
  c.total = c.part + 2ull * c.ctas * 2 * 128 * d * sizeof(float);
  return c;
}

}  // namespace attn
