// Cross attention of few query rows: the tiles of all keys dealt out evenly.
//
// A decode step, or a short decoder sequence, against encoder states is bound by
// reading K and V once.  The G * N_q query rows of a key/value head (G = H / H_kv),
// contiguous in [B, H, N_q, d], form tiles of up to 128 rows; a segment is one such
// tile with the keys of its batch entry, kv_lens[b] of them in tiles of 128.
//
//  * All tiles of all segments stand in one line, and CTA c of C (one per SM)
//    takes an even share, [c T / C, (c + 1) T / C): lengths differ between batch
//    entries, and one CTA per segment left SMs idle in the last wave (B = 32,
//    H_kv = 8, N_k = 2048, half of it to all of it seen: 42 us).
//  * A CTA walks through the parts of segments in its share without draining its
//    ring of K and V tiles between them; scores and outputs are double-buffered
//    in tensor memory, so a part's output is written while the next part's first
//    products run.
//  * A segment inside one share is finished there.  One that crosses shares
//    leaves float32 partial outputs and log-sum-exps, at most two per CTA, which a
//    second kernel merges; its launch overlaps the first kernel.
//  * With few segments, a cluster of up to eight CTAs takes one instead and merges its
//    partial outputs through distributed shared memory: one launch, no scratch, no
//    prefix sums.  (1 x 16 heads, N_q = 1, N_k = 1500, d = 64: 9.4 us shared, 8.0 so;
//    2 x 16 heads, N_k = 4096: 13.7 and 12.3.)
//
// Roles: key and value producer warps, an MMA warp for the score products and one for
// the P V products (issuing a product or a commit costs a thread some hundred cycles:
// one thread for both took 1.04 us a tile at d = 64, where HBM delivers one in 0.75),
// four softmax warps.
#include <cmath>

#include "common.h"
#include "sm103_prims.cuh"

namespace attn {
namespace {

constexpr int kSmemLimit = 232448;
constexpr int BM = 128;   // query rows of a tile
constexpr int BN = 128;   // keys of a tile

// FEW: at most 16 query rows.  They are laid into the query tile four times, at rows
// 0, 32, 64 and 96, so every softmax warp finds them in its own quarter of tensor
// memory; warp w takes keys [32 w, 32 w + 32) of each tile, with statistics of its
// own, its products are written to its quarter only (zeros as its probabilities of the
// other keys would meet their values: 0 * inf = NaN), and the four partial outputs are
// added when a part ends.  (One warp with all 128 keys of a tile needs some
// 1400 cycles a tile, most of them exponentials: at d = 64 that is more than the
// tile's share of HBM time, 5.0 TB/s.)  The gaps behind the four copies hold the
// other Q buffer's four.
// Otherwise: 128 query rows, a thread per row.
template <int D, bool FEW>
struct CrossCfg {
  static constexpr int CH = D / 64;
  static constexpr int CHUNK = 128 * 128;
  static constexpr int TILE = 128 * D * 2;
  static constexpr int QROWS = FEW ? 16 : 128;           // rows of a copy's box
  static constexpr int COPIES = FEW ? 4 : 1;
  static constexpr int QBYTES = COPIES * QROWS * D * 2;  // copied per part
  static constexpr int QSTEP = FEW ? QROWS * 128 : TILE; // from one Q buffer to the other
  static constexpr int QSMEM = FEW ? TILE : 2 * TILE;
  static constexpr int XCH = FEW ? 4 * 16 * 65 * 4 + 4 * 16 * 8 : 0;   // the sum of the four outputs
  static constexpr int LENS = 8 * (kCrossMaxB + 1);      // lengths and tile prefix sums
  static constexpr int NSLOT_FIT = (kSmemLimit - 2048 - LENS - XCH - QSMEM) / TILE;
  static constexpr int NSLOT = NSLOT_FIT > 10 ? 10 : NSLOT_FIT;
  // a product reads 128 rows from its Q buffer: the second one's end in the ring
  static constexpr int SMEM = 1024 + QSMEM + NSLOT * TILE;
  static constexpr int THREADS = 8 * 32;
  static constexpr int LOAD_WARP = 4;
  static constexpr int MMA_S_WARP = 5;
  static constexpr int LOAD_V_WARP = 6;
  static constexpr int MMA_PV_WARP = 7;
  __host__ __device__ static constexpr uint32_t S_COL(int buf) { return 128u * buf; }
  __host__ __device__ static constexpr uint32_t O_COL(int buf) { return 256u + static_cast<uint32_t>(D) * buf; }
  static_assert(NSLOT >= 4 && O_COL(1) + D <= 512, "ring or tensor memory");
};

struct CrossKParams {
  const int* kv_lens;      // [B], or nullptr: Nk
  void* o;
  float* lse;
  float* o_part;           // [2 C][rows of a segment][D]
  float* lse_part;         // [2 C][rows of a segment]
  int* status;
  int B, H_kv, Nk;
  int rows;                // G * N_q: query rows of a key/value head
  int segs;                // segments per batch entry: H_kv * query tiles
  int qtiles;
  int seg_rows;            // rows of a partial result: min(rows, 128)
  float scale_log2;
};

__device__ __forceinline__ float lg2f_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Keys that batch entry b sees; an entry out of range counts as none.
__device__ __forceinline__ int keys_of(const int* kv_lens, int b, int Nk) {
  if (!kv_lens) return Nk;
  const int n = __ldg(kv_lens + b);
  return n < 0 || n > Nk ? 0 : n;
}

// First tile of CTA c's share of T tiles.  At most T CTAs get one, so none of
// theirs is empty; the others' start at T.
__device__ __forceinline__ int share_start(int c, int C, int T) {
  C = min(C, T);
  return c >= C ? T : static_cast<int>(static_cast<long long>(c) * T / C);
}

// A walk over the parts of segments in a share.  pre[b]: tiles of one segment of
// the batch entries before b.
struct Cursor {
  const int* pre;
  int segs, B;
  int b, y, j;      // batch entry, segment of it, tile of the segment
  int left;         // tiles of the share from here on
  __device__ __forceinline__ int tiles() const { return pre[b + 1] - pre[b]; }
  // at the part's first tile: the part's tiles
  __device__ __forceinline__ int part() const { return min(tiles() - j, left); }
  __device__ __forceinline__ void next_part(int n) {
    left -= n;
    if (left <= 0) return;
    j = 0;
    if (++y == segs) {
      y = 0;
      do {
        ++b;
      } while (b < B && pre[b + 1] == pre[b]);
    }
  }
};

__device__ __forceinline__ Cursor cursor_at(const int* pre, int segs, int B, int g, int left) {
  int lo = 0, hi = B;      // last entry whose tiles start at or before g
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (static_cast<long long>(pre[mid]) * segs <= g) lo = mid;
    else hi = mid;
  }
  Cursor c{pre, segs, B, lo, 0, 0, left};
  const int rem = g - pre[lo] * segs;
  const int n = c.tiles();
  if (n > 0) {
    c.y = rem / n;
    c.j = rem - c.y * n;
  }
  return c;
}

// CLUSTER: the cluster's CTAs share one segment, batch entry and segment of it from
// the cluster's index.
template <int D, bool FP16, bool FEW, bool CLUSTER>
__global__ void __launch_bounds__(CrossCfg<D, FEW>::THREADS, 1)
    cross_rows_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const CrossKParams kp) {
  using C = CrossCfg<D, FEW>;
  constexpr int NSLOT = C::NSLOT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + C::QSMEM;

  __shared__ __align__(8) uint64_t q_full[2];
  __shared__ __align__(8) uint64_t q_empty[2];
  __shared__ __align__(8) uint64_t kv_full[NSLOT];
  __shared__ __align__(8) uint64_t kv_empty[NSLOT];
  __shared__ __align__(8) uint64_t s_full[2];
  __shared__ __align__(8) uint64_t p_full[2];
  __shared__ __align__(8) uint64_t o_full[2];
  __shared__ __align__(8) uint64_t o_empty[2];
  __shared__ __align__(8) uint64_t drain_bar[2];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  __shared__ int issued_sh[2];      // items that a producer issued: keys, values
  __shared__ int parts_sh;          // Q tiles issued
  __shared__ int warp_sum[C::THREADS / 32];
  __shared__ int pre_sh[(CLUSTER ? 1 : kCrossMaxB) + 1];
  __shared__ int lens_sh[CLUSTER ? 1 : kCrossMaxB];
  __shared__ float lse_sh[CLUSTER ? BM : 1];       // of the partial output in the ring's place
  __shared__ float xch[FEW ? 4 : 1][16][65];       // 64 columns of the four outputs
  __shared__ float2 stat[FEW ? 4 : 1][16];         // their maxima and sums
  __shared__ __align__(8) uint64_t xch_bar;        // the softmax threads meet around them

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;

  // ---- prologue: tiles of a segment of the batch entries before each, while the
  // barriers are set up, tensor memory is allocated and the tensor maps arrive
  const int ranks = CLUSTER ? static_cast<int>(cluster_size()) : 1;
  const int rank = CLUSTER ? static_cast<int>(cluster_rank()) : 0;
  const int seg = static_cast<int>(blockIdx.x) / ranks;            // CLUSTER: of all
  const int my_b = CLUSTER ? seg / kp.segs : 0;
  const int per = CLUSTER ? 0 : (kp.B + C::THREADS - 1) / C::THREADS;
  const int b0 = min(static_cast<int>(threadIdx.x) * per, kp.B), b1 = min(b0 + per, kp.B);
  if (warp == C::MMA_S_WARP) {
    tmem_alloc(&tmem_base_sh, 512);
    tmem_relinquish();
  } else if (threadIdx.x == C::LOAD_WARP * 32) {
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
    prefetch_tmap(&tmQ);
  } else if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&o_full[i], 1);
      mbar_init(&o_empty[i], 128);
    }
    if constexpr (FEW) mbar_init(&xch_bar, 128);
    for (int s = 0; s < NSLOT; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    mbar_init(&drain_bar[0], 1);
    mbar_init(&drain_bar[1], 1);
    abort_sh = 0;
    issued_sh[0] = issued_sh[1] = parts_sh = 0;
    fence_mbar_init();
  }
  // This launch may have overtaken the end of the stream's previous kernel: from here on
  // that is over, and the next one may come up behind this one in the same way.  The
  // merging kernel reads kv_lens at once, so it is released no earlier.
  wait_for_previous_kernel();
  release_dependents();
  if constexpr (CLUSTER) {
    if (threadIdx.x == 32) {
      int n = kp.kv_lens ? ld_l2_s32(kp.kv_lens + my_b) : kp.Nk;
      if (n < 0 || n > kp.Nk) {
        if (seg % kp.segs == 0 && rank == 0) atomicCAS(kp.status, 0, kDevBadSeqlens);
        n = 0;
      }
      lens_sh[0] = n;
      pre_sh[0] = 0;
      pre_sh[1] = (n + BN - 1) / BN;
    }
  } else {
    int sum = 0;
    for (int b = b0; b < b1; ++b) {
      int n = kp.kv_lens ? ld_l2_s32(kp.kv_lens + b) : kp.Nk;
      if (n < 0 || n > kp.Nk) {
        if (blockIdx.x == 0) atomicCAS(kp.status, 0, kDevBadSeqlens);
        n = 0;
      }
      lens_sh[b] = n;
      sum += (n + BN - 1) / BN;
    }
    int scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += t;
    }
    if (lane == 31) warp_sum[warp] = scan;
    __syncthreads();
    int base = scan - sum;
    for (int w = 0; w < warp; ++w) base += warp_sum[w];
    for (int b = b0; b < b1; ++b) {
      pre_sh[b] = base;
      base += (lens_sh[b] + BN - 1) / BN;
    }
    if (b1 == kp.B && b0 < b1) pre_sh[kp.B] = base;
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = tmem_base_sh;
  const Abort ab{&abort_sh, kp.status};
  // indexed by batch entry; a cluster's has one
  const int* const pre = pre_sh - my_b;
  const int* const lens = lens_sh - my_b;
  int g0, total;                                   // first tile and tiles of this CTA
  Cursor cur;
  if constexpr (CLUSTER) {
    const int nt = pre_sh[1];
    g0 = rank * nt / ranks;
    total = (rank + 1) * nt / ranks - g0;
    cur = Cursor{pre, kp.segs, kp.B, my_b, seg % kp.segs, g0, total};
  } else {
    const int T = pre[kp.B] * kp.segs;
    g0 = share_start(blockIdx.x, gridDim.x, T);
    total = share_start(blockIdx.x + 1, gridDim.x, T) - g0;
    cur = cursor_at(pre, kp.segs, kp.B, g0, total);
  }

  if (warp == C::LOAD_WARP || warp == C::LOAD_V_WARP) {
    // ------------------------------------------------------------ producers
    // Two threads stream into the ring, one copy per tile (its 64-column chunks are a
    // dimension of the map's box).  Item 2 n is the n-th K tile of the share, item
    // 2 n + 1 its V tile.  The part's Q follows its first K tile's copy: HBM first.
    if (lane == 0) {
      const int kv = warp == C::LOAD_WARP ? 0 : 1;
      int n = 0, part = 0;
      bool ok = true;
      while (ok && cur.left > 0) {
        const int take = cur.part();
        const int hk = cur.y / kp.qtiles;
        for (int i = 0; i < take; ++i) {
          const int item = 2 * n + kv;
          const int slot = item % NSLOT, use = item / NSLOT;
          if (use >= 1 && !mbar_wait(&kv_empty[slot], (use - 1) & 1, ab, kDevTimeoutLoad)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&kv_full[slot], C::TILE);
          tma_load_4d(sKV + slot * C::TILE, kv ? &tmV : &tmK, &kv_full[slot], 0, (cur.j + i) * BN, 0,
                      cur.b * kp.H_kv + hk);
          ++n;
          if (kv == 0 && i == 0) {
            if (part >= 2 && !mbar_wait(&q_empty[part & 1], ((part >> 1) - 1) & 1, ab, kDevTimeoutLoad)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&q_full[part & 1], C::QBYTES);
            uint8_t* dst = sQ + (part & 1) * C::QSTEP;
            const int row = hk * kp.rows + (cur.y - hk * kp.qtiles) * BM;
            if constexpr (FEW) {
              // a box is 16 rows of one 64-column chunk
              for (int c = 0; c < C::CH; ++c)
                for (int x = 0; x < 4; ++x)
                  tma_load_4d(dst + c * C::CHUNK + x * 32 * 128, &tmQ, &q_full[part & 1], 0, row, c, cur.b);
            } else {
              tma_load_4d(dst, &tmQ, &q_full[part & 1], 0, row, 0, cur.b);
            }
            ++part;
          }
        }
        cur.next_part(take);
      }
      issued_sh[kv] = n;
      if (kv == 0) parts_sh = part;
    }
  } else if (warp == C::MMA_S_WARP) {
    // ------------------------------------------------------------ S = Q K^T
    // S(n) into buffer n % 2, once the P V product of tile n - 2 has read its
    // probabilities there (the phase of that value slot's empty barrier).  The
    // softmax hands the key slot back when it sees S(n).
    if (lane == 0) {
      constexpr uint32_t idS = idesc_f16(FP16 ? Elt::F16 : Elt::BF16, 128, BN, false, false);
      const uint64_t qdesc0 = sdesc_sw128(smem_u32(sQ), 16, 1024);             // K-major Q
      const uint64_t kdesc0 = sdesc_sw128(smem_u32(sKV), 16, 1024);            // K-major K
      bool ok = true;
      for (int n = 0, part = 0; n < total && ok; ++part) {
        const int take = cur.part();
        if (!(ok = mbar_wait(&q_full[part & 1], (part >> 1) & 1, ab, kDevTimeoutMma))) break;
        const uint64_t qdesc = opaque(sdesc_add(qdesc0, (part & 1) * C::QSTEP));
        for (int i = 0; i < take; ++i, ++n) {
          const int item = 2 * n, slot = item % NSLOT;
          if (!(ok = mbar_wait(&kv_full[slot], (item / NSLOT) & 1, ab, kDevTimeoutMma))) break;
          const int old = 2 * n - 3;             // item of V of tile n - 2
          if (n >= 2 && !(ok = mbar_wait(&kv_empty[old % NSLOT], (old / NSLOT) & 1, ab, kDevTimeoutMma))) break;
          tc_fence_after_sync();
          const uint64_t kdesc = opaque(sdesc_add(kdesc0, slot * C::TILE));
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk / 4) * C::CHUNK + (kk % 4) * 32;
            mma_f16_ss(tmem + C::S_COL(n & 1), sdesc_add(qdesc, off), sdesc_add(kdesc, off), idS, kk > 0 ? 1u : 0u);
          }
          mma_commit(&s_full[n & 1]);
        }
        if (ok) mma_commit(&q_empty[part & 1]);  // the part's Q has been read
        cur.next_part(take);
      }
    }
  } else if (warp == C::MMA_PV_WARP) {
    // ------------------------------------------------------------ O += P V
    // P(n) packed 16-bit in columns [0, 64) of buffer n % 2, O of a part in buffer
    // part % 2.  Every use of a value slot gets its phase on the empty barrier: the
    // producer, the score products and the rescale wait for it.
    if (lane == 0) {
      constexpr uint32_t idPV = idesc_f16(FP16 ? Elt::F16 : Elt::BF16, 128, D, false, true);
      const uint64_t vdesc0 = sdesc_sw128(smem_u32(sKV), C::CHUNK, 1024);      // MN-major V
      bool ok = true;
      for (int n = 0, part = 0; n < total && ok; ++part) {
        const int take = cur.part();
        const uint32_t o_col = C::O_COL(part & 1);
        for (int i = 0; i < take; ++i, ++n) {
          const int item = 2 * n + 1, slot = item % NSLOT;
          if (!(ok = mbar_wait(&kv_full[slot], (item / NSLOT) & 1, ab, kDevTimeoutMma))) break;
          const uint64_t vdesc = opaque(sdesc_add(vdesc0, slot * C::TILE));
          if (!(ok = mbar_wait(&p_full[n & 1], (n >> 1) & 1, ab, kDevTimeoutMma))) break;
          // the buffer's output of two parts ago has been read
          if (i == 0 && part >= 2 &&
              !(ok = mbar_wait(&o_empty[part & 1], ((part >> 1) - 1) & 1, ab, kDevTimeoutMma)))
            break;
          tc_fence_after_sync();
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk) {
            const uint32_t p_col = tmem + C::S_COL(n & 1) + 8 * kk;
            const uint64_t v_at = sdesc_add(vdesc, kk * 16 * 128);
            if constexpr (FEW)   // 16 keys of warp kk / 2, for its rows only
              mma_f16_ts_quarter(tmem + o_col, p_col, v_at, idPV, (i > 0 || kk % 2 > 0) ? 1u : 0u, kk / 2);
            else
              mma_f16_ts(tmem + o_col, p_col, v_at, idPV, (i > 0 || kk > 0) ? 1u : 0u);
          }
          mma_commit(&kv_empty[slot]);
          if (i == take - 1) mma_commit(&o_full[part & 1]);
        }
        cur.next_part(take);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    // Thread r: query row r, all keys of a tile; or (FEW) query row lane, keys [32
    // warp, 32 warp + 32).
    const int r = warp * 32 + lane;
    constexpr int W = FEW ? 32 : BN;                 // keys of a thread in a tile
    const int k0 = FEW ? 32 * warp : 0;
    const uint32_t lane_addr = static_cast<uint32_t>(warp * 32) << 16;
    const float c2 = kp.scale_log2;
    bool ok = true;
    // output of a finished part: where it goes, and its row's statistics
    struct Done {
      int part, b, y;
      bool whole, last;
      float m, l;
    } done{-1, 0, 0, false, false, 0.f, 0.f};
    // partial outputs: the workspace's, or this CTA's for its cluster (the ring is free by
    // then: every copy has been consumed)
    float* const o_part = CLUSTER ? reinterpret_cast<float*>(sKV) : kp.o_part;
    float* const lse_part = CLUSTER ? lse_sh : kp.lse_part;
    auto store_lse = [&](size_t at, size_t part_at, float m, float l) {
      *(done.whole ? kp.lse + at : lse_part + part_at) =
          (m * c2 + lg2f_approx(l)) * 0.69314718055994530942f;
    };
    // all softmax threads meet (an mbarrier, whose wait ends when another warp gave up)
    uint32_t met = 0;
    auto meet = [&]() -> bool {
      mbar_arrive(&xch_bar);
      const bool came = !__any_sync(0xffffffffu, !mbar_wait(&xch_bar, met & 1, ab, kDevTimeoutEpilogue));
      ++met;
      return came;
    };
    auto write_out = [&]() -> bool {
      const int buf = done.part & 1;
      if (__any_sync(0xffffffffu, !mbar_wait(&o_full[buf], (done.part >> 1) & 1, ab, kDevTimeoutEpilogue)))
        return false;
      tc_fence_after_sync();
      const int hk = done.y / kp.qtiles;
      const int row0 = (done.y - hk * kp.qtiles) * BM;        // of the head's G * N_q rows
      // rows of a key/value head are contiguous in [B, H, N_q]
      const size_t at0 = (static_cast<size_t>(done.b) * kp.H_kv + hk) * kp.rows + row0;
      const size_t part0 = CLUSTER ? 0 : static_cast<size_t>(2 * blockIdx.x + (done.last ? 1 : 0)) * kp.seg_rows;
      if constexpr (FEW) {
        // weights of the four outputs of row `lane`: exp(m_w - m) / sum_w exp(m_w - m) l_w
        if (lane < 16) stat[warp][lane] = make_float2(done.m, done.l);
        if (!meet()) return false;
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) m = fmaxf(m, stat[w][lane & 15].x);
#pragma unroll
        for (int w = 0; w < 4; ++w) l += ex2_approx((stat[w][lane & 15].x - m) * c2) * stat[w][lane & 15].y;
        const float weight = ex2_approx((done.m - m) * c2) / l;
        if (warp == 0 && lane < kp.rows) store_lse(at0 + lane, part0 + lane, m, l);
#pragma unroll 1
        for (int c0 = 0; c0 < D / 64; ++c0) {
          if (c0 > 0 && !meet()) return false;       // the round before has been read
          uint32_t o[64];
#pragma unroll
          for (int x = 0; x < 2; ++x)
            tmem_ld32(tmem + lane_addr + C::O_COL(buf) + c0 * 64 + x * 32,
                      *reinterpret_cast<uint32_t(*)[32]>(&o[32 * x]));
          tmem_ld_wait();
          if (lane < 16) {
#pragma unroll
            for (int i = 0; i < 64; ++i) xch[warp][lane][i] = __uint_as_float(o[i]) * weight;
          }
          if (!meet()) return false;
          // rows warp, warp + 4, ...: lane = columns lane and lane + 32
          for (int x = warp; x < kp.rows; x += 4) {
#pragma unroll
            for (int i = lane; i < 64; i += 32) {
              const float sum = (xch[0][x][i] + xch[1][x][i]) + (xch[2][x][i] + xch[3][x][i]);
              if (done.whole) {
                const uint32_t pk = FP16 ? cvt_pack_f16(sum, 0.f) : cvt_pack_bf16(sum, 0.f);
                static_cast<uint16_t*>(kp.o)[(at0 + x) * D + c0 * 64 + i] = static_cast<uint16_t>(pk);
              } else {
                o_part[(part0 + x) * D + c0 * 64 + i] = sum;
              }
            }
          }
        }
      } else {
        const bool row_ok = row0 + r < kp.rows;
        const float inv_l = 1.f / done.l;
#pragma unroll 1
        for (int c0 = 0; c0 < D / 32; ++c0) {
          uint32_t o[32];
          tmem_ld32(tmem + lane_addr + C::O_COL(buf) + c0 * 32, o);
          tmem_ld_wait();
          if (row_ok && done.whole) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(kp.o) + (at0 + r) * D + c0 * 32);
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float x = __uint_as_float(o[2 * i]) * inv_l, z = __uint_as_float(o[2 * i + 1]) * inv_l;
              pk[i] = FP16 ? cvt_pack_f16(x, z) : cvt_pack_bf16(x, z);
            }
#pragma unroll
            for (int v = 0; v < 4; ++v)
              dst[v] = make_uint4(pk[4 * v], pk[4 * v + 1], pk[4 * v + 2], pk[4 * v + 3]);
          } else if (row_ok) {
            float4* dst = reinterpret_cast<float4*>(o_part + (part0 + r) * D + c0 * 32);
#pragma unroll
            for (int v = 0; v < 8; ++v)
              dst[v] = make_float4(__uint_as_float(o[4 * v]) * inv_l, __uint_as_float(o[4 * v + 1]) * inv_l,
                                   __uint_as_float(o[4 * v + 2]) * inv_l, __uint_as_float(o[4 * v + 3]) * inv_l);
          }
        }
        if (row_ok) store_lse(at0 + r, part0 + r, done.m, done.l);
      }
      tc_fence_before_sync();
      mbar_arrive(&o_empty[buf]);
      return true;
    };
    int n = 0, part = 0;
    while (ok && cur.left > 0) {
      const int take = cur.part();
      const int len = lens[cur.b];
      float m_ref = -INFINITY, l = 0.f;
      // a warp without query rows only keeps the others' pace
      const bool live = FEW || (cur.y % kp.qtiles) * BM + warp * 32 < kp.rows;
      for (int i = 0; i < take; ++i, ++n) {
        // a warp that gives up stops arriving at p_full (and where the warps meet), so
        // the others' next wait ends too
        if (__any_sync(0xffffffffu, !mbar_wait(&s_full[n & 1], (n >> 1) & 1, ab, kDevTimeoutSoftmax))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        if (r == 0) mbar_arrive(&kv_empty[(2 * n) % NSLOT]);   // K of tile n has been read
        const int lim = len - (cur.j + i) * BN;        // keys of this tile that are seen
        if (live) {
          const uint32_t tS = tmem + lane_addr + C::S_COL(n & 1);
          uint32_t sr[W];
#pragma unroll
          for (int c0 = 0; c0 < W / 32; ++c0)
            tmem_ld32(tS + k0 + c0 * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[c0 * 32]));
          tmem_ld_wait();
          if (lim < k0 + W) {
#pragma unroll
            for (int c = 0; c < W; ++c)
              if (k0 + c >= lim) sr[c] = __float_as_uint(-INFINITY);
          }
          float m_new = m_ref;
#pragma unroll
          for (int u = 0; u < W / 8; ++u)
            m_new = fmaxf(m_new, fmax3(fmax3(__uint_as_float(sr[8 * u]), __uint_as_float(sr[8 * u + 1]),
                                             __uint_as_float(sr[8 * u + 2])),
                                       fmax3(__uint_as_float(sr[8 * u + 3]), __uint_as_float(sr[8 * u + 4]),
                                             __uint_as_float(sr[8 * u + 5])),
                                       fmaxf(__uint_as_float(sr[8 * u + 6]), __uint_as_float(sr[8 * u + 7]))));
          // lazy rescale: the exponent reference moves when the maximum grew by over 2^8
          const bool need = (m_new - m_ref) * c2 > 8.f;
          float alpha = 1.f;
          if (need) {
            alpha = ex2_approx((m_ref - m_new) * c2);
            l *= alpha;
            m_ref = m_new;
          }
          const float neg = (m_ref == -INFINITY) ? 0.f : -m_ref * c2;
          const uint64_t cc = pack2(c2, c2);
          const uint64_t nn = pack2(neg, neg);
          uint64_t acc0 = 0, acc1 = 0;
#pragma unroll
          for (int c0 = 0; c0 < W / 32; ++c0) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int c = c0 * 32 + 2 * e;
              const uint64_t y = ffma2(pack2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), cc, nn);
              const float p0 = ex2_approx(lo2(y));
              const float p1 = ex2_approx(hi2(y));
              if (e & 1) acc1 = fadd2(acc1, pack2(p0, p1));
              else acc0 = fadd2(acc0, pack2(p0, p1));
              pk[e] = FP16 ? cvt_pack_f16(p0, p1) : cvt_pack_bf16(p0, p1);
            }
            // packed P of keys [k, +32) -> columns [k / 2, +16)
            tmem_st16(tS + k0 / 2 + c0 * 16, pk);
          }
          const uint64_t acc = fadd2(acc0, acc1);
          l += lo2(acc) + hi2(acc);
          if (i > 0 && __any_sync(0xffffffffu, need)) {
            // rescale O once P(n - 1) V has landed; this tile's product is issued
            // only after the arrive below
            const int old = 2 * n - 1;           // item of V of tile n - 1
            if (__any_sync(0xffffffffu, !mbar_wait(&kv_empty[old % NSLOT], (old / NSLOT) & 1, ab,
                                                   kDevTimeoutSoftmax))) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            const uint32_t tO = tmem + lane_addr + C::O_COL(part & 1);
#pragma unroll 1
            for (int c0 = 0; c0 < D / 32; ++c0) {
              uint32_t o[32];
              tmem_ld32(tO + c0 * 32, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(tO + c0 * 32, o);
            }
          }
        }
        if (lim < BN && len < kp.Nk) {
          // rows of V behind the keys may hold anything: they meet P = 0 in the
          // product, so they are zeroed first (0 * NaN = NaN)
          const int item = 2 * n + 1;
          if (__any_sync(0xffffffffu, !mbar_wait(&kv_full[item % NSLOT], (item / NSLOT) & 1, ab,
                                                 kDevTimeoutSoftmax))) {
            ok = false;
            break;
          }
          zero_tile_rows<C::CH, C::CHUNK>(sKV + (item % NSLOT) * C::TILE, lim, r, 128);
          fence_proxy_async_smem();
        }
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(&p_full[n & 1]);
        // the part before this one, while this tile's products run
        if (i == 0 && part > 0 && !write_out()) {
          ok = false;
          break;
        }
      }
      if (!ok) break;
      done = Done{part, cur.b, cur.y, !CLUSTER && take == cur.tiles(), part > 0, m_ref, l};
      cur.next_part(take);
      ++part;
    }
    if (ok && part > 0) write_out();
    if constexpr (CLUSTER) {
      if (total == 0) lse_sh[r] = -INFINITY;
    }
    // batch entries without keys: O = 0 and LSE = -inf (a cluster's merge finds them)
    const size_t rows_b = static_cast<size_t>(kp.H_kv) * kp.rows;
    for (int b = blockIdx.x; !CLUSTER && b < kp.B; b += gridDim.x) {
      if (pre[b + 1] != pre[b]) continue;
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(kp.o) + b * rows_b * D);
      for (size_t i = r; i < rows_b * (D / 8); i += 128) dst[i] = make_uint4(0u, 0u, 0u, 0u);
      for (size_t i = r; i < rows_b; i += 128) kp.lse[b * rows_b + i] = -INFINITY;
    }
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before_sync();
  __syncthreads();
  if (abort_sh) {
    // let every copy and MMA this CTA issued land before the memory goes away
    if ((warp == C::LOAD_WARP || warp == C::LOAD_V_WARP) && lane == 0) {
      const int kv = warp == C::LOAD_WARP ? 0 : 1;
      for (int i = issued_sh[kv] - 1; i >= 0 && 2 * i + kv >= 2 * issued_sh[kv] - 2 * NSLOT; --i) {
        const int item = 2 * i + kv;
        mbar_wait_drain(&kv_full[item % NSLOT], (item / NSLOT) & 1);
      }
      if (kv == 0)
        for (int i = parts_sh - 1; i >= 0 && i >= parts_sh - 2; --i) mbar_wait_drain(&q_full[i & 1], (i >> 1) & 1);
    }
    if ((warp == C::MMA_S_WARP || warp == C::MMA_PV_WARP) && lane == 0) {
      uint64_t* bar = &drain_bar[warp == C::MMA_S_WARP ? 0 : 1];
      mma_commit(bar);
      mbar_wait_drain(bar, 0);
    }
    __syncthreads();
  }
  if (warp == C::MMA_S_WARP) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
  if constexpr (CLUSTER) {
    // every thread of every CTA comes here, after an abort too.  The cluster's threads
    // share the segment's rows, four columns each.
    cluster_sync();
    const int y = seg % kp.segs, hk = y / kp.qtiles, row0 = (y - hk * kp.qtiles) * BM;
    const size_t at0 = (static_cast<size_t>(my_b) * kp.H_kv + hk) * kp.rows + row0;
    const int items = min(BM, kp.rows - row0) * (D / 4);
    for (int x = rank * C::THREADS + threadIdx.x; x < items; x += ranks * C::THREADS) {
      const int r = x / (D / 4), c4 = x % (D / 4);
      float lse[8], m = -INFINITY;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        lse[i] = i < ranks ? ld_cluster_f32(smem_u32(lse_sh + r), i) : -INFINITY;
        m = fmaxf(m, lse[i]);
      }
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (lse[i] == -INFINITY) continue;           // no keys: nothing was written there
        const float w = expf(lse[i] - m);
        const float4 o = ld_cluster_v4(smem_u32(reinterpret_cast<float*>(sKV) + r * D + 4 * c4), i);
        sum += w;
        acc = make_float4(fmaf(w, o.x, acc.x), fmaf(w, o.y, acc.y), fmaf(w, o.z, acc.z), fmaf(w, o.w, acc.w));
      }
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
      const uint2 pk = FP16 ? make_uint2(cvt_pack_f16(acc.x * inv, acc.y * inv), cvt_pack_f16(acc.z * inv, acc.w * inv))
                            : make_uint2(cvt_pack_bf16(acc.x * inv, acc.y * inv), cvt_pack_bf16(acc.z * inv, acc.w * inv));
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(kp.o) + (at0 + r) * D + 4 * c4) = pk;
      if (c4 == 0) kp.lse[at0 + r] = m + logf(sum);   // -inf without keys
    }
    cluster_sync();                                  // the others may still be reading here
  }
}

// Segments that cross shares: LSE = log sum_c exp(lse_c) and O = sum_c exp(lse_c -
// LSE) O_c over the CTAs whose shares they touch, with a running maximum.  One block
// per segment and kMergeRows of its rows, D / 4 threads per row; four partial
// results are loaded at a time.
constexpr int kMergeThreads = 128;
template <int D>
constexpr int kMergeRows = kMergeThreads / (D / 4);

template <int D, bool FP16>
__global__ void __launch_bounds__(kMergeThreads)
    cross_merge_kernel(const CrossKParams kp, int C) {
  __shared__ int sums[2][4];
  release_dependents();
  const int b = blockIdx.z, y = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // tiles of a segment of the entries before b, and of all
  int before = 0, all = 0;
  for (int i = threadIdx.x; i < kp.B; i += kMergeThreads) {
    const int n = (keys_of(kp.kv_lens, i, kp.Nk) + BN - 1) / BN;
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
  before = sums[0][0] + sums[0][1] + sums[0][2] + sums[0][3];
  const int T = (sums[1][0] + sums[1][1] + sums[1][2] + sums[1][3]) * kp.segs;
  const int nt = (keys_of(kp.kv_lens, b, kp.Nk) + BN - 1) / BN;
  const int g0 = before * kp.segs + y * nt, g1 = g0 + nt - 1;
  // CTA whose share holds tile g: the last c with c T / C <= g
  C = min(C, T);
  const int c0 = nt ? static_cast<int>(((g0 + 1ll) * C - 1) / T) : 0;
  const int c1 = nt ? static_cast<int>(((g1 + 1ll) * C - 1) / T) : 0;
  // a share's first part is its slot 0, a later one its slot 1; the segment is a
  // later part only where it starts inside a share
  const int slot0 = 2 * c0 + (nt == 0 || share_start(c0, C, T) == g0 ? 0 : 1);
  const int hk = y / kp.qtiles;
  const int row0 = (y - hk * kp.qtiles) * BM;
  const int r = blockIdx.y * kMergeRows<D> + threadIdx.x / (D / 4);
  const int col = (threadIdx.x % (D / 4)) * 4;
  wait_for_previous_kernel();
  if (c0 == c1 || r >= min(BM, kp.rows - row0)) return;
  float m = -INFINITY, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = c0; c <= c1; c += 4) {
    float lse[4];
    float4 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lse[i] = -INFINITY;
      o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c + i <= c1) {
        const size_t at = static_cast<size_t>(c + i == c0 ? slot0 : 2 * (c + i)) * kp.seg_rows + r;
        lse[i] = kp.lse_part[at];
        o[i] = *reinterpret_cast<const float4*>(kp.o_part + at * D + col);
      }
    }
    const float m_new = fmaxf(m, fmaxf(fmaxf(lse[0], lse[1]), fmaxf(lse[2], lse[3])));
    const float keep = m == -INFINITY ? 0.f : expf(m - m_new);
    sum *= keep;
    acc = make_float4(acc.x * keep, acc.y * keep, acc.z * keep, acc.w * keep);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float w = lse[i] == -INFINITY ? 0.f : expf(lse[i] - m_new);
      sum += w;
      acc.x = fmaf(w, o[i].x, acc.x);
      acc.y = fmaf(w, o[i].y, acc.y);
      acc.z = fmaf(w, o[i].z, acc.z);
      acc.w = fmaf(w, o[i].w, acc.w);
    }
    m = m_new;
  }
  const float inv = 1.f / sum;
  const size_t at = (static_cast<size_t>(b) * kp.H_kv + hk) * kp.rows + row0 + r;
  const uint2 pk = FP16 ? make_uint2(cvt_pack_f16(acc.x * inv, acc.y * inv), cvt_pack_f16(acc.z * inv, acc.w * inv))
                        : make_uint2(cvt_pack_bf16(acc.x * inv, acc.y * inv), cvt_pack_bf16(acc.z * inv, acc.w * inv));
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(kp.o) + at * D + col) = pk;
  if (col == 0) kp.lse[at] = m + logf(sum);
}

template <int D, bool FP16, bool FEW>
attn_status_t launch_cross_rows_t(const FwdParams& p, const CrossPlan& plan, void* workspace,
                                  cudaStream_t stream) {
  using C = CrossCfg<D, FEW>;
  auto kern = plan.cluster ? cross_rows_kernel<D, FP16, FEW, true> : cross_rows_kernel<D, FP16, FEW, false>;
  attn_status_t s = set_smem(reinterpret_cast<const void*>(kern), C::SMEM);
  if (s != ATTN_OK) return s;
  CUtensorMap tq, tk, tv;
  // {64 columns, rows, 64-column chunks, planes}: one box holds every chunk
  const uint64_t row_b = 2ull * D, q_rows = static_cast<uint64_t>(p.H) * p.N;
  const uint64_t planes = static_cast<uint64_t>(p.B) * p.H_kv;
  if ((s = make_tmap_4d(&tq, p.q, 2, 64, q_rows, C::CH, p.B, row_b, 128, row_b * q_rows, 64, C::QROWS,
                        FEW ? 1 : C::CH)) != ATTN_OK)
    return s;
  if ((s = make_tmap_4d(&tk, p.k, 2, 64, p.N_k, C::CH, planes, row_b, 128, row_b * p.N_k, 64, BN, C::CH)) != ATTN_OK)
    return s;
  if ((s = make_tmap_4d(&tv, p.v, 2, 64, p.N_k, C::CH, planes, row_b, 128, row_b * p.N_k, 64, BN, C::CH)) != ATTN_OK)
    return s;
  int* status = device_status_word();
  if (!status) return fail(ATTN_ERR_CUDA, "status word unavailable");
  const int rows = p.H / p.H_kv * p.N;
  const int seg_rows = rows < BM ? rows : BM;
  const size_t part_rows = 2ull * plan.ctas * seg_rows;
  char* ws = static_cast<char*>(workspace);
  CrossKParams kp{p.kv_lens, p.o, p.lse, reinterpret_cast<float*>(ws),
                  reinterpret_cast<float*>(ws + align_up(part_rows * D * sizeof(float), 256)), status,
                  p.B, p.H_kv, p.N_k, rows, p.H_kv * plan.qtiles, plan.qtiles, seg_rows,
                  p.scale * 1.4426950408889634f};
  cudaError_t e;
  if (plan.cluster) {
    e = launch_dependent(kern, dim3(plan.ctas), C::THREADS, C::SMEM, stream, plan.cluster, tq, tk, tv, kp);
    return e == cudaSuccess ? ATTN_OK : fail_cuda(e, "cross attention rows kernel launch");
  }
  e = launch_dependent(kern, dim3(plan.ctas), C::THREADS, C::SMEM, stream, 0, tq, tk, tv, kp);
  if (e != cudaSuccess) return fail_cuda(e, "cross attention rows kernel launch");
  e = launch_dependent(cross_merge_kernel<D, FP16>, dim3(kp.segs, (seg_rows + kMergeRows<D> - 1) / kMergeRows<D>, p.B),
                       kMergeThreads, 0, stream, 0, kp, plan.ctas);
  if (e != cudaSuccess) return fail_cuda(e, "cross attention merge kernel launch");
  return ATTN_OK;
}

}  // namespace

attn_status_t launch_cross_rows(const FwdParams& p, const CrossPlan& plan, void* workspace,
                                cudaStream_t stream) {
  const bool few = p.H / p.H_kv * p.N <= 16;
#define ATTN_CROSS_ROWS(D, F)                                                   \
  return few ? launch_cross_rows_t<D, F, true>(p, plan, workspace, stream)      \
             : launch_cross_rows_t<D, F, false>(p, plan, workspace, stream)
  if (p.d == 64) {
    if (p.fp16) ATTN_CROSS_ROWS(64, true);
    ATTN_CROSS_ROWS(64, false);
  }
  if (p.fp16) ATTN_CROSS_ROWS(128, true);
  ATTN_CROSS_ROWS(128, false);
#undef ATTN_CROSS_ROWS
}

}  // namespace attn
