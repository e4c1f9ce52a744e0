// Backward of cross attention: N_q query rows against N_k keys of another length,
// kv_lens[b] of them seen (cross.cu and fwd.cu compute the forward).
//
// The formulas and the step are those of the self-attention backward (bwd.cu): for a
// key tile j and a query tile i, S^T and dP^T on the tensor cores, P^T and dS^T in the
// compute warps, then dV += P^T dO_i, dK += dS^T Q_i, and dQ_i += dS K_j added to a
// float32 accumulator by TMA.  What differs is how the steps are dealt out.
//
//  * A segment is a key tile of one key/value head and batch entry with all its
//    steps: the query tiles of every query head that shares it.  All segments have
//    equally many.  Their steps stand in one line, and CTA c of C (one per SM) takes
//    an even share.  One CTA per segment, as in the self-attention pass, would
//    leave a short encoder or few key/value heads on a handful of SMs, and the key
//    tiles of two long ones in a last, half-empty wave (B = 2, H = 16, H_kv = 4, N_q =
//    8192, N_k = 4096 with a quarter of the second entry's keys unseen, d = 128: 1003 us
//    so, 803 shared, both with the 16-bit P below).
//  * Step n of a segment that starts when its CTA has done t steps is query step (t + n)
//    mod the segment's steps: CTAs on the same heads read the same Q and dO tiles at
//    about the same time, from L2.  (In each segment's own order they read them
//    from HBM, 1245 us for the shape above.)
//  * A segment inside one share is finished there.  One that crosses shares leaves
//    float32 partial dK and dV, at most two per CTA, which a last kernel adds in
//    the order of the CTAs, so dK and dV do not depend on timing.  The same kernel
//    converts dQ and clears dK and dV behind the keys.
//  * Rows of K and V behind kv_lens[b] may hold anything, NaN included.  The compute
//    warps zero them in shared memory before a segment's first product: then S = dP =
//    0 there, and P is set to 0 as for rows past the tensor.
//
// P is rounded to 16 bits for dV = P^T dO; dS takes it in 24 (64 float32 values per
// thread and the packed ones do not fit the 96 registers that 18 warps leave), so dQ and
// dK carry the rounding of dS and their own: relative 0.0024 in bfloat16, 0.0017 of it
// the output's.  With the 16-bit P for both, as in bwd.cu: 0.0029, and 1 to 2 % less time.
#include <cmath>

#include "bwd_parts.cuh"

namespace attn {
namespace {

struct XBars {
  uint64_t kv_full;
  uint64_t kv_clean;       // rows of K and V behind the keys are zeroed (with kv_lens)
  uint64_t q_full[2];
  uint64_t q_empty[2];
  uint64_t do_full[2];
  uint64_t do_empty[2];
  uint64_t s_full;
  uint64_t dp_full;
  uint64_t p_ready;
  uint64_t ds_ready;
  uint64_t dq_full;
  uint64_t dq_free;
  uint64_t dkv_full;
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  int kv_items, q_items, do_items;   // loads issued (for draining after an abort)
  int start[2];                      // the share's first segment: batch entry, segment of it
};
// the barrier area's first 256 bytes; the prologue's warp sums lie in the staging
// buffers, which nothing uses yet
static_assert(sizeof(XBars) <= 256, "barrier area overflow");

struct XBwdKParams {
  void* dk;
  void* dv;
  float* part;          // [2 C][dV, dK][128][D] float32
  const float* lse2;    // -L * log2(e), [B * H][Npad], -inf padding
  const float* delta;   // -rowsum(dO * O), [B * H][Npad], 0 padding
  const int* kv_lens;   // [B], or nullptr
  int* status;
  int B, N, Npad, Nk, H, H_kv, group;
  float scale;
  float scale_log2;
};

__device__ __forceinline__ int seen_keys(const int* kv_lens, int b, int Nk) {
  if (!kv_lens) return Nk;
  const int n = __ldg(kv_lens + b);
  return n < 0 || n > Nk ? 0 : n;
}

// CTAs that get a share of `segs` segments of nsteps steps, of the grid's `ctas`.
// Loading a segment's K and V, its first step's latency and its output cost about
// kPartSteps steps (8 us), and shares that cross segments pay that at least twice.
// So with fewer segments than CTAs every segment may be cut into m equal parts, one
// CTA each; otherwise, or where even shares of all CTAs come out ahead, all of them.
// (31 tiles x 4 heads, 12 steps each, d = 64: one part each 27 us, even shares 32.)
constexpr int kPartSteps = 5;
__device__ __forceinline__ int share_count(int segs, int nsteps, int ctas) {
  const int m = min(ctas / max(segs, 1), nsteps);
  if (m == 0) return ctas;
  const long long T = static_cast<long long>(segs) * nsteps;
  const int even = static_cast<int>((T + ctas - 1) / ctas);
  const int even_cost = even + kPartSteps * ((even + nsteps - 1) / nsteps + 1);
  return (nsteps + m - 1) / m + kPartSteps <= even_cost ? segs * m : ctas;
}

// First step of CTA c's share of T steps; at most T CTAs get one.
__device__ __forceinline__ int step_share(int c, int C, int T) {
  C = min(C, T);
  return c >= C ? T : static_cast<int>(static_cast<long long>(c) * T / C);
}

// A walk over the parts of segments in a share.
struct Walk {
  const int* kv_lens;
  int B, Nk, H_kv, nsteps;
  int b, keys, y;   // batch entry, the keys it sees, segment of it (head-major)
  int n0;           // step of the segment
  int left;         // steps of the share from here on
  int done;         // steps of the share before
  int rot;          // query step of the segment's step 0
  __device__ __forceinline__ int ktiles() const { return (keys + 127) / 128; }
  __device__ __forceinline__ int take() const { return min(nsteps - n0, left); }
  __device__ __forceinline__ int head() const { return y / ktiles(); }
  __device__ __forceinline__ int tile() const { return y % ktiles(); }
  // query step of the part's first step
  __device__ __forceinline__ int first() const { return (rot + n0) % nsteps; }
  __device__ __forceinline__ void next(int n) {
    left -= n;
    done += n;
    rot = done % nsteps;
    n0 = 0;
    if (++y == ktiles() * H_kv) {
      y = 0;
      do {
        keys = ++b < B ? seen_keys(kv_lens, b, Nk) : 1;
      } while (keys == 0);
    }
  }
};

template <int D, bool FP16>
__global__ void __launch_bounds__(BwdCfg<D>::THREADS, 1)
    cross_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                     const __grid_constant__ CUtensorMap tmDQ, const XBwdKParams kp) {
  using C = BwdCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
  if (pad > static_cast<uint32_t>(C::SLACK)) {
    // Cannot place the swizzled tiles: report and leave before touching anything.
    if (threadIdx.x == 0) atomicCAS(kp.status, 0, kDevSmemMisaligned);
    wait_for_previous_kernel();
    return;
  }
  uint8_t* smem = smem_raw + pad;
  XBars& bars = *reinterpret_cast<XBars*>(smem + C::OFF_BAR);

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const int nQ = (kp.N + C::BM - 1) / C::BM;
  const int nsteps = kp.group * nQ;

  if (threadIdx.x == 0) {
    mbar_init(&bars.kv_full, 1);
    mbar_init(&bars.kv_clean, 256);
    for (int s = 0; s < C::NQS; ++s) {
      mbar_init(&bars.q_full[s], 1);
      mbar_init(&bars.q_empty[s], 1);
    }
    for (int s = 0; s < C::NDS; ++s) {
      mbar_init(&bars.do_full[s], 1);
      mbar_init(&bars.do_empty[s], 1);
    }
    mbar_init(&bars.s_full, 1);
    mbar_init(&bars.dp_full, 1);
    mbar_init(&bars.p_ready, 256);
    mbar_init(&bars.ds_ready, 256);
    mbar_init(&bars.dq_full, 1);
    mbar_init(&bars.dq_free, 256);
    mbar_init(&bars.dkv_full, 1);
    mbar_init(&bars.drain, 1);
    bars.abort_flag = 0;
    bars.kv_items = bars.q_items = bars.do_items = 0;
    bars.start[0] = kp.B;
    bars.start[1] = 0;
    fence_mbar_init();
  }
  if (warp == C::MMA_WARP) {
    tmem_alloc(&bars.tmem_base, 512);
    tmem_relinquish();
  }
  // Key tiles of the batch entries before each thread's own, and of all: the steps'
  // count T, and the segment in which this CTA's share starts.
  int* warp_sum = reinterpret_cast<int*>(smem + C::OFF_STG);
  const int per = (kp.B + C::THREADS - 1) / C::THREADS;
  const int b0 = min(static_cast<int>(threadIdx.x) * per, kp.B), b1 = min(b0 + per, kp.B);
  int sum = 0;
  for (int b = b0; b < b1; ++b) {
    if (kp.kv_lens && blockIdx.x == 0) {
      const int n = __ldg(kp.kv_lens + b);
      if (n < 0 || n > kp.Nk) atomicCAS(kp.status, 0, kDevBadSeqlens);
    }
    sum += (seen_keys(kp.kv_lens, b, kp.Nk) + C::BN - 1) / C::BN;
  }
  int scan = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += t;
  }
  if (lane == 31) warp_sum[warp] = scan;
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  int base = scan - sum, all = 0;
  for (int w = 0; w < C::THREADS / 32; ++w) {
    if (w < warp) base += warp_sum[w];
    all += warp_sum[w];
  }
  const int T = all * kp.H_kv * nsteps;
  const int ctas = share_count(all * kp.H_kv, nsteps, gridDim.x);
  const int g0 = step_share(blockIdx.x, ctas, T);
  const int total = step_share(blockIdx.x + 1, ctas, T) - g0;        // steps of this CTA
  const int seg0 = g0 / nsteps;                                      // its first segment
  release_dependents();
  if (total > 0 && seg0 >= base * kp.H_kv && seg0 < (base + sum) * kp.H_kv) {
    int at = base, b = b0;
    while (true) {
      const int n = (seen_keys(kp.kv_lens, b, kp.Nk) + C::BN - 1) / C::BN;
      if (seg0 < (at + n) * kp.H_kv) break;
      at += n;
      ++b;
    }
    bars.start[0] = b;
    bars.start[1] = seg0 - at * kp.H_kv;
  }
  wait_for_previous_kernel();      // row vectors, and the dQ accumulator's zeros
  __syncthreads();
  const uint32_t tmem = bars.tmem_base;
  const Abort ab{&bars.abort_flag, kp.status};
  Walk w{kp.kv_lens, kp.B, kp.Nk, kp.H_kv, nsteps, bars.start[0], 1, bars.start[1], g0 - seg0 * nsteps, total, 0, 0};
  if (total > 0) {
    w.keys = seen_keys(kp.kv_lens, w.b, kp.Nk);
    // the CTA in whose share the first segment starts: the last c with c T / C <= start
    const long long start = static_cast<long long>(seg0) * nsteps;
    const int C0 = min(ctas, T);
    const int c0 = static_cast<int>(((start + 1) * C0 - 1) / T);
    w.rot = static_cast<int>(start - step_share(c0, C0, T)) % nsteps;
  }

  // Every barrier's phase below follows the CTA's own count of steps (n) or of
  // parts, over all its parts.
  if (warp == C::LOAD_WARP) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tmap(&tmQ);
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
      prefetch_tmap(&tmDO);
      int n = 0, nd = 0;                   // Q and dO loads issued
      bool ok = true;
      for (int part = 0; ok && w.left > 0; ++part) {
        const int take = w.take(), hk = w.head(), j = w.tile(), bhk = w.b * kp.H_kv + hk;
        // K_j and V_j, once every product of the part before has read its own
        if (part >= 1 && !mbar_wait(&bars.dkv_full, (part - 1) & 1, ab, kDevTimeoutLoad)) break;
        mbar_arrive_expect_tx(&bars.kv_full, 2 * C::TILE);
#pragma unroll
        for (int c = 0; c < C::CH; ++c) {
          tma_load_3d(smem + C::OFF_K + c * C::CHUNK, &tmK, &bars.kv_full, c * 64, j * C::BN, bhk);
          tma_load_3d(smem + C::OFF_V + c * C::CHUNK, &tmV, &bars.kv_full, c * 64, j * C::BN, bhk);
        }
        bars.kv_items = part + 1;
        int h = w.first() / nQ, i = w.first() % nQ;      // query head of the group, query tile
        const int plane0 = w.b * kp.H + hk * kp.group;
        for (int s = 0; s < take; ++s, ++n, (++i == nQ) ? (i = 0, (++h == kp.group) ? (h = 0) : 0) : 0) {
          // Q_i with its row vectors -L*log2(e) and -D into Q slot n % NQS
          {
            const int st = n % C::NQS;
            const int use = n / C::NQS;
            if (use >= 1 && !mbar_wait(&bars.q_empty[st], (use - 1) & 1, ab, kDevTimeoutLoad)) {
              ok = false;
              break;
            }
            uint8_t* sq = smem + C::OFF_Q + st * C::TILE;
            float* sld = reinterpret_cast<float*>(smem + C::OFF_LD + st * 1024);
            mbar_arrive_expect_tx(&bars.q_full[st], C::TILE + 1024);
#pragma unroll
            for (int c = 0; c < C::CH; ++c)
              tma_load_3d(sq + c * C::CHUNK, &tmQ, &bars.q_full[st], c * 64, i * C::BM, plane0 + h);
            const size_t roff = static_cast<size_t>(plane0 + h) * kp.Npad + static_cast<size_t>(i) * C::BM;
            bulk_load(sld, kp.lse2 + roff, 512, &bars.q_full[st]);
            bulk_load(sld + 128, kp.delta + roff, 512, &bars.q_full[st]);
            bars.q_items = n + 1;
          }
          // dO_i into dO slot n % NDS
          {
            const int st = n % C::NDS;
            const int use = n / C::NDS;
            if (use >= 1 && !mbar_wait(&bars.do_empty[st], (use - 1) & 1, ab, kDevTimeoutLoad)) {
              ok = false;
              break;
            }
            uint8_t* sdo = smem + C::OFF_DO + st * C::TILE;
            mbar_arrive_expect_tx(&bars.do_full[st], C::TILE);
#pragma unroll
            for (int c = 0; c < C::CH; ++c)
              tma_load_3d(sdo + c * C::CHUNK, &tmDO, &bars.do_full[st], c * 64, i * C::BM, plane0 + h);
            bars.do_items = ++nd;
          }
        }
        w.next(take);
      }
    }
  } else if (warp == C::MMA_WARP) {
    // ------------------------------------------------------------ MMA issue
    if (lane == 0) {
      constexpr Elt E = FP16 ? Elt::F16 : Elt::BF16;
      constexpr uint32_t idSP = idesc_f16(E, 128, 128, false, false);   // S^T and dP^T
      constexpr uint32_t idKV = idesc_f16(E, 128, D, false, true);      // dV and dK (A in TMEM)
      constexpr uint32_t idQ = idesc_f16(E, 128, D, true, true);        // dQ = dS K_j
      const uint32_t sK = smem_u32(smem + C::OFF_K);
      const uint32_t sV = smem_u32(smem + C::OFF_V);
      const uint64_t mK = opaque(sdesc_sw128(sK, C::CHUNK, 1024));
      const uint64_t mDS = opaque(sdesc_sw128(smem_u32(smem + C::OFF_DS), C::CHUNK, 1024));
      // S^T(i) = K_j Q_i^T, dP^T(i) = V_j dO_i^T
      auto issue = [&](uint32_t col, uint32_t a, uint32_t bb, uint64_t* full) {
        const uint64_t da = opaque(sdesc_sw128(a, 16, 1024));
        const uint64_t db = opaque(sdesc_sw128(bb, 16, 1024));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk / 4) * C::CHUNK + (kk % 4) * 32;
          mma_f16_ss(tmem + col, sdesc_add(da, off), sdesc_add(db, off), idSP, kk > 0 ? 1u : 0u);
        }
        mma_commit(full);
      };
      auto slot_q = [&](int x) { return smem_u32(smem + C::OFF_Q + (x % C::NQS) * C::TILE); };
      auto slot_do = [&](int x) { return smem_u32(smem + C::OFF_DO + (x % C::NDS) * C::TILE); };
      auto wait_q = [&](int x) {
        return mbar_wait(&bars.q_full[x % C::NQS], (x / C::NQS) & 1, ab, kDevTimeoutMma);
      };
      // Issue order of a step, as in bwd.cu: dP^T(n), dV(n), S^T(n + 1), dK(n), dQ(n);
      // a part's first S^T waits for its K and V.
      bool ok = true;
      int n = 0;
      for (int part = 0; ok && w.left > 0; ++part) {
        const int take = w.take();
        ok = mbar_wait(&bars.kv_full, part & 1, ab, kDevTimeoutMma) &&
             (!kp.kv_lens || mbar_wait(&bars.kv_clean, part & 1, ab, kDevTimeoutMma)) && wait_q(n);
        if (!ok) break;
        tc_fence_after_sync();
        issue(C::S_COL, sK, slot_q(n), &bars.s_full);
        for (int s = 0; s < take; ++s, ++n) {
          const uint32_t sQ = slot_q(n);
          const uint32_t sDO = slot_do(n);
          // dP^T(n); at d = 128 its columns must have been read out (dQ(n - 1)).  Its
          // completion also means dQ(n - 1) has finished reading the dS^T buffer.
          if (C::DQ_IN_DP && n > 0 && !(ok = mbar_wait(&bars.dq_free, (n - 1) & 1, ab, kDevTimeoutMma))) break;
          if (!(ok = mbar_wait(&bars.do_full[n % C::NDS], (n / C::NDS) & 1, ab, kDevTimeoutMma))) break;
          tc_fence_after_sync();
          issue(C::DP_COL, sV, sDO, &bars.dp_full);
          // dV += P^T dO_i.  A part's first product overwrites dV (and dK below): the
          // compute warps have read the part before's, which they do ahead of this P^T.
          if (!(ok = mbar_wait(&bars.p_ready, n & 1, ab, kDevTimeoutMma))) break;
          tc_fence_after_sync();
          const uint64_t mDO = opaque(sdesc_sw128(sDO, C::CHUNK, 1024));
#pragma unroll
          for (int kk = 0; kk < C::BM / 16; ++kk)
            mma_f16_ts(tmem + C::DV_COL, tmem + C::S_COL + C::half_col(kk), sdesc_add(mDO, kk * 16 * 128),
                       idKV, (s > 0 || kk > 0) ? 1u : 0u);
          if (n + C::NDS < total) mma_commit(&bars.do_empty[n % C::NDS]);
          // S^T of the part's next step (its columns now only hold P^T(n), read above)
          if (s + 1 < take) {
            if (!(ok = wait_q(n + 1))) break;
            tc_fence_after_sync();
            issue(C::S_COL, sK, slot_q(n + 1), &bars.s_full);
          }
          // dK += dS^T Q_i; the Q slot is free after it
          if (!(ok = mbar_wait(&bars.ds_ready, n & 1, ab, kDevTimeoutMma))) break;
          tc_fence_after_sync();
          const uint64_t mQ = opaque(sdesc_sw128(sQ, C::CHUNK, 1024));
#pragma unroll
          for (int kk = 0; kk < C::BM / 16; ++kk)
            mma_f16_ts(tmem + C::DK_COL, tmem + C::DP_COL + C::half_col(kk), sdesc_add(mQ, kk * 16 * 128),
                       idKV, (s > 0 || kk > 0) ? 1u : 0u);
          if (n + C::NQS < total) mma_commit(&bars.q_empty[n % C::NQS]);
          // dQ_i = dS K_j into its columns (at d = 64 once dQ(n - 1) was read out)
          if (!C::DQ_IN_DP && n > 0) {
            if (!(ok = mbar_wait(&bars.dq_free, (n - 1) & 1, ab, kDevTimeoutMma))) break;
            tc_fence_after_sync();
          }
#pragma unroll
          for (int kk = 0; kk < C::BN / 16; ++kk)
            mma_f16_ss(tmem + C::DQ_COL, sdesc_add(mDS, kk * 16 * 128), sdesc_add(mK, kk * 16 * 128),
                       idQ, kk > 0 ? 1u : 0u);
          mma_commit(&bars.dq_full);
        }
        if (ok) mma_commit(&bars.dkv_full);
        w.next(take);
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ compute WGs
    const int h = warp >> 2;                         // query half: columns [64 h, 64 h + 64)
    const int quarter = warp & 3;
    const int k = quarter * 32 + lane;               // key row of the tile = TMEM lane
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const float c2 = kp.scale_log2;
    const uint32_t sDSrow = smem_u32(smem + C::OFF_DS) + h * C::CHUNK + k * 128;
    bool ok = true;
    int n = 0;
    for (int part = 0; w.left > 0; ++part) {
      const int take = w.take();
      const int key_g = w.tile() * C::BN + k;
      const bool key_ok = key_g < w.keys;
      if (kp.kv_lens) {
        // without kv_lens, rows past the tensor were loaded as zeros
        if (!(ok = mbar_wait(&bars.kv_full, part & 1, ab, kDevTimeoutSoftmax))) break;
        const int row0 = w.keys - w.tile() * C::BN;
        if (row0 < C::BN) {
          zero_tile_rows<C::CH, C::CHUNK>(smem + C::OFF_K, row0, threadIdx.x, 256);
          zero_tile_rows<C::CH, C::CHUNK>(smem + C::OFF_V, row0, threadIdx.x, 256);
          fence_proxy_async_smem();
        }
        mbar_arrive(&bars.kv_clean);
      }
      for (int s = 0; s < take; ++s, ++n) {
        const int st = n % C::NQS;
        const float4* nlse4 = reinterpret_cast<const float4*>(smem + C::OFF_LD + st * 1024);  // -L log2 e
        const float4* ndvec4 = nlse4 + 32;                                                  // -D
        // phase A: P^T = exp2(S^T c - L log2 e), written back as 16-bit
        if (!(ok = mbar_wait(&bars.s_full, n & 1, ab, kDevTimeoutSoftmax))) break;
        tc_fence_after_sync();
        // this half's P^T for dS, the upper 24 bits of each float, four in three words
        uint32_t p24[48];
        const uint64_t cc = pack2(c2, c2);
        auto probabilities = [&](int c, const uint32_t* sv) {     // queries [64 h + 16 c, +16)
          const int qb = 64 * h + 16 * c;
          uint32_t pb[8];
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 l4 = nlse4[(qb + e) / 4];
            const uint64_t y0 = ffma2(pack2(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])), cc,
                                      pack2(l4.x, l4.y));
            const uint64_t y1 = ffma2(pack2(__uint_as_float(sv[e + 2]), __uint_as_float(sv[e + 3])), cc,
                                      pack2(l4.z, l4.w));
            float p[4] = {ex2_approx(lo2(y0)), ex2_approx(hi2(y0)), ex2_approx(lo2(y1)), ex2_approx(hi2(y1))};
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (!key_ok) p[u] = 0.f;
            pb[e / 2] = FP16 ? cvt_pack_f16(p[0], p[1]) : cvt_pack_bf16(p[0], p[1]);
            pb[e / 2 + 1] = FP16 ? cvt_pack_f16(p[2], p[3]) : cvt_pack_bf16(p[2], p[3]);
            uint32_t w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) w[u] = __float_as_uint(p[u]);
            uint32_t* const at = p24 + (16 * c + e) / 4 * 3;
            at[0] = __byte_perm(w[0], w[1], 0x5321);
            at[1] = __byte_perm(w[1], w[2], 0x6532);
            at[2] = __byte_perm(w[2], w[3], 0x7653);
          }
          // packed P^T of queries [qb, qb + 16) -> columns [64 h + 8 c, +8)
          tmem_st_x8(tmem + lane_addr + C::S_COL + 64 * h + 8 * c, pb);
        };
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t sv[16];
          tmem_ld16(tmem + lane_addr + C::S_COL + 64 * h + 16 * c, sv);
          tmem_ld_wait();
          probabilities(c, sv);
        }
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(&bars.p_ready);
        // phase B: dS^T = P^T (dP^T - D), into tensor memory (for dK) and the shared
        // dS^T buffer (for dQ)
        if (!(ok = mbar_wait(&bars.dp_full, n & 1, ab, kDevTimeoutSoftmax))) break;
        tc_fence_after_sync();
        auto differences = [&](int c, const uint32_t* dpv) {      // queries [64 h + 16 c, +16)
          const int qb = 64 * h + 16 * c;
          uint32_t dd[8];
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 d4 = ndvec4[(qb + e) / 4];
            // widened here, not earlier: keeps packed registers live instead of floats.  What
            // stands in the lowest byte is 2^-15 of the value at most.
            const uint32_t* const at = p24 + (16 * c + e) / 4 * 3;
            const uint32_t w0 = opaque32(at[0]), w1 = opaque32(at[1]), w2 = opaque32(at[2]);
            const uint64_t pa = pack2(__uint_as_float(__byte_perm(w0, w0, 0x2100)),
                                      __uint_as_float(__byte_perm(w0, w1, 0x5433)));
            const uint64_t pc = pack2(__uint_as_float(__byte_perm(w1, w2, 0x4322)), __uint_as_float(w2));
            const uint64_t dsa = fmul2(pa, fadd2(pack2(__uint_as_float(dpv[e]), __uint_as_float(dpv[e + 1])),
                                                 pack2(d4.x, d4.y)));
            const uint64_t dsc = fmul2(pc, fadd2(pack2(__uint_as_float(dpv[e + 2]), __uint_as_float(dpv[e + 3])),
                                                 pack2(d4.z, d4.w)));
            dd[e / 2] = FP16 ? cvt_pack_f16(lo2(dsa), hi2(dsa)) : cvt_pack_bf16(lo2(dsa), hi2(dsa));
            dd[e / 2 + 1] = FP16 ? cvt_pack_f16(lo2(dsc), hi2(dsc)) : cvt_pack_bf16(lo2(dsc), hi2(dsc));
          }
          tmem_st_x8(tmem + lane_addr + C::DP_COL + 64 * h + 8 * c, dd);
          // dS^T row k, queries [qb, qb + 16) = 16-byte pieces 2c and 2c + 1 of
          // chunk h, placed with the 128-byte swizzle
#pragma unroll
          for (int pc2 = 0; pc2 < 2; ++pc2) {
            const uint32_t piece = static_cast<uint32_t>(2 * c + pc2);
            st_shared_v4(sDSrow + ((piece ^ (k & 7)) * 16), dd[4 * pc2], dd[4 * pc2 + 1], dd[4 * pc2 + 2],
                         dd[4 * pc2 + 3]);
          }
        };
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t dpv[16];
          tmem_ld16(tmem + lane_addr + C::DP_COL + 64 * h + 16 * c, dpv);
          tmem_ld_wait();
          differences(c, dpv);
        }
        tmem_st_wait();
        fence_proxy_async_smem();
        tc_fence_before_sync();
        mbar_arrive(&bars.ds_ready);
      }
      // ---- the part's dV (half 0) or dK (half 1): final, or float32 for the join
      if (!ok || !(ok = mbar_wait(&bars.dkv_full, part & 1, ab, kDevTimeoutEpilogue))) break;
      tc_fence_after_sync();
      const uint32_t col = h ? C::DK_COL : C::DV_COL;
      if (take == nsteps) {
        const float mul = h ? kp.scale : 1.f;
        uint16_t* dst_row = static_cast<uint16_t*>(h ? kp.dk : kp.dv) +
                            (static_cast<size_t>(w.b * kp.H_kv + w.head()) * kp.Nk + key_g) * D;
#pragma unroll 1
        for (int c0 = 0; c0 < D / 32; ++c0) {
          uint32_t v[32];
          tmem_ld32(tmem + lane_addr + col + c0 * 32, v);
          tmem_ld_wait();
          if (key_ok) {                              // rows behind the keys: the join's
            uint4* dst = reinterpret_cast<uint4*>(dst_row + c0 * 32);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint32_t pk[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float a = __uint_as_float(v[8 * x + 2 * e]) * mul;
                const float bb = __uint_as_float(v[8 * x + 2 * e + 1]) * mul;
                pk[e] = FP16 ? cvt_pack_f16(a, bb) : cvt_pack_bf16(a, bb);
              }
              dst[x] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            }
          }
        }
      } else {
        float* dst_row = kp.part + ((static_cast<size_t>(2 * blockIdx.x + (part > 0 ? 1 : 0)) * 2 + h) * 128 + k) * D;
#pragma unroll 1
        for (int c0 = 0; c0 < D / 32; ++c0) {
          uint32_t v[32];
          tmem_ld32(tmem + lane_addr + col + c0 * 32, v);
          tmem_ld_wait();
          uint4* dst = reinterpret_cast<uint4*>(dst_row + c0 * 32);
#pragma unroll
          for (int x = 0; x < 8; ++x) dst[x] = make_uint4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
        }
      }
      w.next(take);
    }
  } else {
    // ------------------------------------------------------------ dQ reduce WGs
    // As in bwd.cu: TMEM lane = query row; each warp moves its 32 rows x D / 2 columns
    // through a 4 KB staging box per 32 columns and adds it with a TMA reduce-add.
    const int g = (warp - 8) >> 2;
    const int quarter = warp & 3;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    constexpr int HC = D / 2;                        // columns per reduce warpgroup
    uint8_t* const stg = smem + C::OFF_STG + (warp - 8) * C::STG_BOX;
    const uint32_t stg_row = smem_u32(stg) + lane * 128;
    bool pending = false;                            // a reduce from `stg` may be reading it
    bool ok = true;
    int n = 0;
    while (ok && w.left > 0) {
      const int take = w.take();
      int h = w.first() / nQ, i = w.first() % nQ;
      const int plane0 = w.b * kp.H + w.head() * kp.group;
      for (int s = 0; s < take; ++s, ++n, (++i == nQ) ? (i = 0, (++h == kp.group) ? (h = 0) : 0) : 0) {
        if (!(ok = mbar_wait(&bars.dq_full, n & 1, ab, kDevTimeoutReduce))) break;
        tc_fence_after_sync();
        uint32_t v[HC];
#pragma unroll
        for (int c0 = 0; c0 < HC / 32; ++c0)
          tmem_ld32(tmem + lane_addr + C::DQ_COL + g * HC + c0 * 32,
                    *reinterpret_cast<uint32_t(*)[32]>(&v[c0 * 32]));
        tmem_ld_wait();
        tc_fence_before_sync();
        mbar_arrive(&bars.dq_free);
        const int row0 = i * C::BM + quarter * 32;   // first query row of this warp's box
#pragma unroll
        for (int bx = 0; bx < HC / 32; ++bx) {
          if (pending) {
            if (lane == 0) bulk_wait_read_all();
            __syncwarp();
          }
#pragma unroll
          for (int c = 0; c < 8; ++c)
            st_shared_v4(stg_row + ((c ^ (lane & 7)) * 16), v[32 * bx + 4 * c], v[32 * bx + 4 * c + 1],
                         v[32 * bx + 4 * c + 2], v[32 * bx + 4 * c + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_reduce_add_3d(&tmDQ, stg, g * HC + 32 * bx, row0, plane0 + h);
            bulk_commit_group();
          }
          pending = true;
        }
      }
      w.next(take);
    }
    // every reduce this warp issued has finished before the CTA ends
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before_sync();
  __syncthreads();
  if (bars.abort_flag) {
    if (warp == C::LOAD_WARP && lane == 0) {
      if (bars.kv_items > 0) mbar_wait_drain(&bars.kv_full, (bars.kv_items - 1) & 1);
      const int nq = bars.q_items;
      for (int s = 0; s < C::NQS && s < nq; ++s)
        mbar_wait_drain(&bars.q_full[s], ((nq - 1 - s) / C::NQS) & 1);
      const int nd = bars.do_items;
      for (int s = 0; s < C::NDS && s < nd; ++s)
        mbar_wait_drain(&bars.do_full[s], ((nd - 1 - s) / C::NDS) & 1);
    }
    if (warp == C::MMA_WARP && lane == 0) {
      mma_commit(&bars.drain);
      mbar_wait_drain(&bars.drain, 0);
    }
    __syncthreads();
  }
  if (warp == C::MMA_WARP) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// The pre-pass of batch entries that see at most kFewKeys keys: as bwd_prep_kernel, but D =
// sum_j P_j dP_j from the keys themselves.  Of one or a few keys O is of V's size, and its
// rounding weighs in dO . O against the differences dP - D: relative error of dQ and dK in float16
// 0.00047 (2 keys), 0.00038 (4), 0.00033 (8), 0.00032 (16), so 0.0003; with more keys it tends to
// 0.0003 either way.  MIXED: entries of other lengths are in the batch too and take dO . O, with
// bwd_prep_kernel's sums; an entry's gradients do not depend on how far the others pad it.
// Bound: the products' issue slots, 0.7 us per key and 75 K rows (whole backward pass of
// those: 28 us with the other pre-pass; 30, 34 and 39 so at 2, 8 and 16 keys); DRAM for dO . O.
constexpr int kFewKeys = 16;

// Rows that a group of D / 8 lanes takes at a time, so that what is read of a key serves them
// all, and rows of a block.  MIXED: few enough for the occupancy that dO . O needs (two rows of a
// long training step's batch: 64 registers; four, in blocks of 128 rows, took 17 us more).
template <int D, bool MIXED>
struct FewKeysCfg {
  static constexpr int L = D / 8;
  static constexpr int ROWS = 256 / L;
  static constexpr int R = MIXED ? 2 : 4;
  static constexpr int BLOCK_ROWS = MIXED ? R * ROWS : 128;
};

template <int D, bool FP16, bool MIXED>
__global__ void __launch_bounds__(256, MIXED ? 4 : 1)
    cross_few_keys_prep_kernel(const XBwdKParams kp, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                               const uint16_t* o, const uint16_t* dout, const float* lse, float* lse2, float* delta,
                               float* dq_acc) {
  using C = FewKeysCfg<D, MIXED>;
  constexpr int L = C::L, ROWS = C::ROWS, R = C::R;
  __shared__ __align__(16) float ks[kFewKeys][D], vs[kFewKeys][D];
  wait_for_previous_kernel();
  release_dependents();
  // rows of one head
  const int tiles = kp.Npad / C::BLOCK_ROWS;
  const long long bh = blockIdx.x / tiles;
  const int n0 = static_cast<int>(blockIdx.x % tiles) * C::BLOCK_ROWS;
  const int b = static_cast<int>(bh / kp.H), h = static_cast<int>(bh % kp.H);
  const int sub = threadIdx.x / L, li = threadIdx.x % L;
  auto widen8 = [](const uint4& w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = FP16 ? __half22float2(*reinterpret_cast<const __half2*>(&u[e]))
                            : make_float2(__uint_as_float(u[e] << 16), __uint_as_float(u[e] & 0xffff0000u));
      x[2 * e] = f.x;
      x[2 * e + 1] = f.y;
    }
  };
  auto load8 = [&](const uint16_t* at, float (&x)[8]) { widen8(__ldcg(reinterpret_cast<const uint4*>(at)), x); };
  int keys = kp.Nk;
  if (kp.kv_lens) {
    keys = ld_l2_s32(kp.kv_lens + b);
    if (keys < 0 || keys > kp.Nk) keys = 0;
  }
  if constexpr (MIXED) {
    // D = dO . O: the loads are on their way before the keys' number is known
    uint4 x[R], y[R];
    float nl[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int n = n0 + sub + r * ROWS;
      const size_t at = (bh * kp.N + n) * D + 8 * li;
      x[r] = y[r] = make_uint4(0u, 0u, 0u, 0u);
      nl[r] = -INFINITY;
      if (n >= kp.N) continue;
      x[r] = __ldcg(reinterpret_cast<const uint4*>(o + at));
      y[r] = __ldcg(reinterpret_cast<const uint4*>(dout + at));
      nl[r] = -__ldcg(lse + bh * kp.N + n) * kLog2e;
    }
    if (keys > kFewKeys) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int n = n0 + sub + r * ROWS;
        float a[8], c[8], sum = 0.f;
        widen8(x[r], a);
        widen8(y[r], c);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(a[e], c[e], sum);
#pragma unroll
        for (int off = L / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (n < kp.N) {
          float4* z = reinterpret_cast<float4*>(dq_acc + (bh * kp.N + n) * D + 8 * li);
          z[0] = z[1] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (li == 0) {
          // stored negated, as the other pre-pass does
          const size_t prow = bh * kp.Npad + n;
          delta[prow] = n < kp.N ? -sum : 0.f;
          lse2[prow] = nl[r];
        }
      }
      return;
    }
  }
  const size_t kv0 = (static_cast<size_t>(b) * kp.H_kv + h / kp.group) * kp.Nk * D;
  for (int i = threadIdx.x; i < 2 * keys * L; i += 256) {
    const int j = i % (keys * L);
    float x[8];
    load8((i < keys * L ? k : v) + kv0 + 8 * j, x);
    float4* dst = reinterpret_cast<float4*>((i < keys * L ? &ks[0][0] : &vs[0][0]) + 8 * j);
    dst[0] = make_float4(x[0], x[1], x[2], x[3]);
    dst[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
  __syncthreads();
  for (int n1 = n0 + sub; n1 < n0 + C::BLOCK_ROWS; n1 += R * ROWS) {
    float qr[R][8] = {}, dr[R][8] = {};
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int n = n1 + r * ROWS;
      if (n >= kp.N) continue;
      const size_t at = (bh * kp.N + n) * D + 8 * li;
      load8(q + at, qr[r]);
      load8(dout + at, dr[r]);
      float4* z = reinterpret_cast<float4*>(dq_acc + at);
      z[0] = z[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // of the 2 R sums (S, dP of R rows) lane i keeps sum i mod 2 R, the even lanes the rows'
    const int n = n1 + (li % (2 * R) / 2) * ROWS;
    const float nl = n < kp.N ? -__ldcg(lse + bh * kp.N + n) * kLog2e : -INFINITY;
    float sum = 0.f;
    for (int j = 0; j < keys; ++j) {
      float x[8], y[8], w[2 * R];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        *reinterpret_cast<float4*>(x + 4 * e) = *reinterpret_cast<const float4*>(&ks[j][8 * li + 4 * e]);
        *reinterpret_cast<float4*>(y + 4 * e) = *reinterpret_cast<const float4*>(&vs[j][8 * li + 4 * e]);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        w[2 * r] = w[2 * r + 1] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          w[2 * r] = fmaf(qr[r][e], x[e], w[2 * r]);
          w[2 * r + 1] = fmaf(dr[r][e], y[e], w[2 * r + 1]);
        }
      }
#pragma unroll
      for (int off = R; off > 0; off >>= 1) {
#pragma unroll
        for (int i = 0; i < off; ++i) {
          const float send = (li & off) ? w[i] : w[i + off], keep = (li & off) ? w[i + off] : w[i];
          w[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
        }
      }
#pragma unroll
      for (int off = 2 * R; off < L; off <<= 1) w[0] += __shfl_xor_sync(0xffffffffu, w[0], off);
      const float dp = __shfl_xor_sync(0xffffffffu, w[0], 1);
      sum = fmaf(ex2_approx(fmaf(w[0], kp.scale_log2, nl)), dp, sum);
    }
    if (li < 2 * R && li % 2 == 0) {
      const size_t prow = bh * kp.Npad + n;
      delta[prow] = n < kp.N ? -sum : 0.f;
      lse2[prow] = nl;
    }
  }
}

// Blocks [0, join_blocks): kJoinRows keys of a key tile each -- the sum of their partial
// dK and dV in the order of the CTAs that left them, and zeros behind the keys.  The
// other blocks: dQ = scale * accumulator, rounded to the 16-bit type.
// Bound: DRAM, 4 bytes of the accumulator and 2 of dQ per element.
constexpr int kJoinRows = 16;

template <int D, bool FP16>
__global__ void __launch_bounds__(256)
    cross_bwd_join_kernel(const XBwdKParams kp, int ctas, int ktiles, unsigned join_blocks,
                          const float* acc, uint16_t* dq, long long n8) {
  auto pack8 = [](const float4& a, const float4& b, float m) {
    return FP16 ? make_uint4(cvt_pack_f16(a.x * m, a.y * m), cvt_pack_f16(a.z * m, a.w * m),
                             cvt_pack_f16(b.x * m, b.y * m), cvt_pack_f16(b.z * m, b.w * m))
                : make_uint4(cvt_pack_bf16(a.x * m, a.y * m), cvt_pack_bf16(a.z * m, a.w * m),
                             cvt_pack_bf16(b.x * m, b.y * m), cvt_pack_bf16(b.z * m, b.w * m));
  };
  if (blockIdx.x >= join_blocks) {
    wait_for_previous_kernel();
    const unsigned blocks = gridDim.x - join_blocks;
    for (long long i = static_cast<long long>(blockIdx.x - join_blocks) * 256 + threadIdx.x; i < n8;
         i += static_cast<long long>(blocks) * 256) {
      const float4 a = reinterpret_cast<const float4*>(acc)[2 * i];
      const float4 b = reinterpret_cast<const float4*>(acc)[2 * i + 1];
      reinterpret_cast<uint4*>(dq)[i] = pack8(a, b, kp.scale);
    }
    return;
  }
  __shared__ int sums[2][8];
  const int tile = blockIdx.x / (128 / kJoinRows);
  const int r0 = blockIdx.x % (128 / kJoinRows) * kJoinRows;   // first row of the tile
  const int j = tile % ktiles;
  const int bhk = tile / ktiles;
  const int b = bhk / kp.H_kv, hk = bhk - b * kp.H_kv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int before = 0, all = 0;                           // key tiles of the entries before b, and of all
  for (int i = threadIdx.x; i < kp.B; i += 256) {
    const int n = (seen_keys(kp.kv_lens, i, kp.Nk) + 127) / 128;
    all += n;
    if (i < b) before += n;
  }
  before = __reduce_add_sync(0xffffffffu, before);
  all = __reduce_add_sync(0xffffffffu, all);
  if (lane == 0) {
    sums[0][warp] = before;
    sums[1][warp] = all;
  }
  __syncthreads();
  before = all = 0;
  for (int x = 0; x < 8; ++x) {
    before += sums[0][x];
    all += sums[1][x];
  }
  const int keys = seen_keys(kp.kv_lens, b, kp.Nk);
  const int kt = (keys + 127) / 128;
  const int nsteps = kp.group * ((kp.N + 127) / 128);
  int c0 = 0, c1 = -1, slot0 = 0;                    // CTAs that left partial sums
  if (j < kt) {
    const int T = all * kp.H_kv * nsteps;
    const long long g0 = static_cast<long long>(before * kp.H_kv + hk * kt + j) * nsteps, g1 = g0 + nsteps - 1;
    const int C = min(share_count(all * kp.H_kv, nsteps, ctas), T);
    // CTA whose share holds step g: the last c with c T / C <= g
    c0 = static_cast<int>(((g0 + 1) * C - 1) / T);
    c1 = static_cast<int>(((g1 + 1) * C - 1) / T);
    // a share's first part is its slot 0, a later one its slot 1; the segment is a later
    // part only where it starts inside a share
    slot0 = 2 * c0 + (step_share(c0, C, T) == g0 ? 0 : 1);
  }
  wait_for_previous_kernel();
  const int rows = min(kJoinRows, kp.Nk - j * 128 - r0);
  const size_t first = (static_cast<size_t>(bhk) * kp.Nk + j * 128 + r0) * D;
  for (int i = threadIdx.x; i < 2 * rows * (D / 8); i += 256) {
    const int h = i / (rows * (D / 8));              // 0: dV, 1: dK
    const int x = i - h * rows * (D / 8);
    const int r = r0 + x / (D / 8), c8 = x % (D / 8);
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(h ? kp.dk : kp.dv) + first) + x;
    if (j * 128 + r >= keys) {
      *dst = make_uint4(0u, 0u, 0u, 0u);
    } else if (c0 != c1) {
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f), bb = a;
      for (int c = c0; c <= c1; c += 4) {            // four loads in flight
        float4 s[4], t[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          s[y] = t[y] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (c + y <= c1) {
            const float4* src = reinterpret_cast<const float4*>(
                kp.part + ((static_cast<size_t>(c + y == c0 ? slot0 : 2 * (c + y)) * 2 + h) * 128 + r) * D) + 2 * c8;
            s[y] = src[0];
            t[y] = src[1];
          }
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          a = make_float4(a.x + s[y].x, a.y + s[y].y, a.z + s[y].z, a.w + s[y].w);
          bb = make_float4(bb.x + t[y].x, bb.y + t[y].y, bb.z + t[y].z, bb.w + t[y].w);
        }
      }
      *dst = pack8(a, bb, h ? kp.scale : 1.f);
    }
  }
}

template <int D, bool FP16>
attn_status_t launch_cross_bwd_t(const BwdParams& p, float* part, int ctas, cudaStream_t stream) {
  using C = BwdCfg<D>;
  const int Npad = (p.N + 127) / 128 * 128;
  const long long rows_pad = static_cast<long long>(p.B) * p.H * Npad;
  int* status = device_status_word();
  if (!status) return fail(ATTN_ERR_CUDA, "status word unavailable");
  XBwdKParams kp{p.dk, p.dv, part, p.lse2, p.delta, p.kv_lens, status, p.B, p.N, Npad, p.N_k,
                 p.H, p.H_kv, p.H / p.H_kv, p.scale, p.scale * kLog2e};
  cudaError_t e;
  // 1. pre-pass: row vectors, dQ accumulator zeroed
  {
    auto rows = [](const void* x) { return static_cast<const uint16_t*>(x); };
    if (p.N_k <= kFewKeys || p.kv_lens) {
      const auto kern = p.N_k <= kFewKeys ? cross_few_keys_prep_kernel<D, FP16, false>
                                          : cross_few_keys_prep_kernel<D, FP16, true>;
      const int block_rows = p.N_k <= kFewKeys ? FewKeysCfg<D, false>::BLOCK_ROWS : FewKeysCfg<D, true>::BLOCK_ROWS;
      e = launch_dependent(kern, dim3(static_cast<unsigned>(rows_pad / block_rows)), 256, 0, stream, 0, kp, rows(p.q),
                           rows(p.k), rows(p.v), rows(p.o), rows(p.dout), p.lse, p.lse2, p.delta, p.dq_acc);
    } else {
      constexpr int rows_per_block = 8 * (32 / (D / 8));
      e = launch_dependent(bwd_prep_kernel<D, FP16, false, true>,
                           dim3(static_cast<unsigned>((rows_pad + rows_per_block - 1) / rows_per_block)), 256, 0, stream,
                           0, rows(p.o), rows(p.dout), p.lse, p.lse2, p.delta, p.dq_acc, p.N, Npad, rows_pad, p.H,
                           nullptr, 0);
    }
    if (e != cudaSuccess) return fail_cuda(e, "cross-attention backward prep launch");
  }
  // 2. main
  {
    auto kern = cross_bwd_kernel<D, FP16>;
    attn_status_t s = set_smem(reinterpret_cast<const void*>(kern), C::SMEM_BYTES);
    if (s != ATTN_OK) return s;
    CUtensorMap tq, tk, tv, tdo, tdq;
    const uint64_t pq = static_cast<uint64_t>(p.B) * p.H, pkv = static_cast<uint64_t>(p.B) * p.H_kv;
    if ((s = make_tmap_3d(&tq, p.q, 2, D, p.N, pq, 64, 128)) != ATTN_OK) return s;
    if ((s = make_tmap_3d(&tdo, p.dout, 2, D, p.N, pq, 64, 128)) != ATTN_OK) return s;
    if ((s = make_tmap_3d(&tk, p.k, 2, D, p.N_k, pkv, 64, 128)) != ATTN_OK) return s;
    if ((s = make_tmap_3d(&tv, p.v, 2, D, p.N_k, pkv, 64, 128)) != ATTN_OK) return s;
    if ((s = make_tmap_3d(&tdq, p.dq_acc, 4, D, p.N, pq, 32, 32)) != ATTN_OK) return s;
    e = launch_dependent(kern, dim3(ctas), C::THREADS, C::SMEM_BYTES, stream, 0, tq, tk, tv, tdo, tdq, kp);
    if (e != cudaSuccess) return fail_cuda(e, "cross-attention backward main launch");
  }
  // 3. join dK and dV, convert dQ
  const int ktiles = (p.N_k + 127) / 128;
  const long long join = static_cast<long long>(ktiles) * p.H_kv * p.B * (128 / kJoinRows);
  const long long n8 = static_cast<long long>(p.B) * p.H * p.N * D / 8;
  const long long want = (n8 + 255) / 256;
  const long long convert = want < 152 * 16 ? want : 152 * 16;
  e = launch_dependent(cross_bwd_join_kernel<D, FP16>, dim3(static_cast<unsigned>(join + convert)), 256, 0, stream, 0,
                       kp, ctas, ktiles, static_cast<unsigned>(join), p.dq_acc, static_cast<uint16_t*>(p.dq), n8);
  if (e != cudaSuccess) return fail_cuda(e, "cross-attention backward join launch");
  return ATTN_OK;
}

}  // namespace

attn_status_t launch_cross_bwd(const BwdParams& p, float* part, int ctas, cudaStream_t stream) {
  switch (p.d) {
    case 64:
      return p.fp16 ? launch_cross_bwd_t<64, true>(p, part, ctas, stream)
                    : launch_cross_bwd_t<64, false>(p, part, ctas, stream);
    case 128:
      return p.fp16 ? launch_cross_bwd_t<128, true>(p, part, ctas, stream)
                    : launch_cross_bwd_t<128, false>(p, part, ctas, stream);
  }
  return fail(ATTN_ERR_UNSUPPORTED, "the backward pass supports d = 64 and 128");
}

}  // namespace attn
