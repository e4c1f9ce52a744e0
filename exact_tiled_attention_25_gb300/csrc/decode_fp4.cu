// Decode attention over a paged 4-bit cache (fp4.cuh): n_q new query tokens per sequence,
// grouped-query heads, keys optionally stored transformed.
//
//   S_ij = scale q_i . (k^_j s^k_j),   O_i = sum_j softmax(S)_ij (v^_j s^v_j),
// with k^, v^ the e2m1 values of a row and s^k, s^v its descales.  A step reads d + 4 bytes
// per token and head; at HBM's rate an SM has some 730 clocks for 128 tokens of a head, their
// keys and values.
//
//  * The codes are operands of the tensor cores as they are: TMA unpacks a row's 64 bytes to 128
//    of shared memory (eight bytes of codes and a gap of eight), which kind::f8f6f4 reads as
//    e2m1, the key tile K-major and the value tile MN-major.  Nothing is dequantised.  (The first
//    version of this kernel converted the codes to float16 operands of mma.sync in registers, 850
//    instructions for 32 keys: 57 us for 16 x 8192 tokens of 8 heads, where this takes 30.)
//  * The products run with the keys on the M side, S^T = K^ Q^T and O^T += V^^T P^T, and both
//    the queries and the probabilities are the other operand, e4m3.  They are held as sums of
//    several e4m3 terms, each 2^5 finer than the one before, in columns of their own (a product
//    this narrow costs what its 128 rows of codes cost, so the columns are free).  A term keeps
//    four bits and the sign of what is left gives a fifth, so n terms are off by 2^(1 - 5 n):
//    queries take two in bfloat16 and three in float16, which is exact, and four when they are
//    transformed (2^-19); probabilities two for a bfloat16 result (2^-9, what bfloat16 itself
//    would round) and three for a float16 one.
//  * A thread holds the scores of one key (d = 64: two) for four or eight query rows, so no lane idles.
//  * p = 2^(s - M), M a running reference of the scores; the row sums add p in float32, and what meets the
//    codes is P' = p s^v c with c = 2^(M - T + 5), T a running reference of s + log2 s^v: it is
//    the tokens that count for the result whose probabilities have all their bits, however the
//    descales differ.  What is 2^-11 of the largest or less loses bits (an error of 2^-20 of that
//    one; three terms: 2^-14 and 2^-25; float16, from which the terms are taken, adds up to 2^-30).
//    The references move only when a score exceeds M by 64 or P' would exceed 2^8, by a vote of the
//    softmax warps once a tile.
//  * d = 64: rows of two neighbouring tokens are one row of the tile.  Their scores are two
//    products over half the columns each; in O^T the first 64 lanes take the even tokens' columns
//    and the others the odd ones', and the two halves are added at the end.
//  * A segment is up to 16 query rows of a key/value head with all keys of a sequence.  The
//    tiles of all segments stand in one line, dealt out evenly to the CTAs (two to an SM); segments
//    that cross shares are joined by a second, dependent kernel from float32 partial results
//    (at most two per CTA).  With few segments a cluster of up to eight CTAs takes each instead and
//    joins its partial results through distributed shared memory: one launch, no scratch, no prefix
//    sums (one request of 1500 tokens, 8 heads: 10.4 us by shares when this took 8.0; 7.2 now).
//  * Measured: 16 x 8192 tokens, 8 heads of d = 128, 4 query rows each 29.7 us (4.7 TB/s; some 9 us
//    are the dealing out, the first tile, the last one and the joining), 8 rows 33.5, 16 rows 51.0 (bound by
//    the chain of a tile's softmax); 64 sequences of up to 16384 tokens, d = 64: 58.9 us (4.9 TB/s).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.h"
#include "fp4.cuh"
#include "rope.cuh"

namespace attn {
namespace {

constexpr int kSmemLimit = 232448;      // of one CTA; with two to an SM each has half of 1024 more, less 1024
constexpr float kFar = 3e38f;           // -M before the first token
constexpr float kPTop = 256.f;          // P' at most (e4m3: 448); 2^5 at its reference
constexpr float kPShift = 5.f;
constexpr float kMostC = 120.f;         // log2 of c at most: values of 2^-115 of the largest scores' and less count as that
constexpr int kPStep = 5;               // a term's steps are 2^-5 of those of the one before

constexpr int pad16(int n) { return (n + 15) / 16 * 16; }
constexpr int pow2(int n) {
  int p = 32;
  while (p < n) p *= 2;
  return p;
}

// NR: query rows of a segment.  TQ, TP: e4m3 terms of queries and of probabilities.
template <int D, int NR, int TQ, int TP>
struct Cfg {
  static constexpr int KP = 128 / D;                     // tokens of a tile's row
  static constexpr int TILE = 128 * KP;                  // tokens of a tile
  static constexpr int SLOT = 128 * 128;                 // its keys' or values' codes, unpacked
  static constexpr int NS = pad16(NR * TQ), NPV = pad16(NR * TP * KP);
  static constexpr int CW = NR == 16 ? 2 : 1;            // softmax warps per quarter of the keys
  static constexpr int SW = 4 * CW;
  static constexpr int NRW = NR / CW;                    // query rows of a softmax thread
  static constexpr int PART = NR == 4 ? 1 : 2;       // tiles that take the time of a part's start and end
  static constexpr int QW = NR == 16 ? NR * D / 512 : 1; // query warps: of 16 rows one for each 512 values
  // Copying warps: with two one has the keys, one the values (16 x 8192 tokens in pages of 16: 38.2 us with one,
  // 31.9 with two).  Of 8 rows one: with 18 warps on an SM there are 96 registers a thread (33.4 us; two: 34.6).
  static constexpr int LW = NR == 8 ? 1 : 2;
  static constexpr int LOAD = SW, MMA_S = SW + LW, MMA_PV = MMA_S + 1, QUERY = MMA_PV + 1;
  static constexpr int THREADS = (QUERY + QW) * 32;
  static constexpr int CTAS = NR == 16 ? 1 : 2;          // of an SM (16 rows: registers)
  // The two query tiles (NS rows of D bytes); of d = 64 they are the halves of one of 128 bytes a row.
  static constexpr int Q_BYTES = 2 * NS * D, P_TILE = NPV * 128;
  static constexpr int Q_STEP = KP == 2 ? 64 : NS * 128;
  static constexpr int PB = NR == 4 && KP == 1 ? 3 : 2;  // buffers of P'
  static constexpr int FIXED = 1024 + Q_BYTES + PB * P_TILE;
  static constexpr int STATIC = 1024 + NR * 140 + (KP == 2 ? NR * 256 : 0);   // at most
  static constexpr int PER_CTA = (CTAS == 1 ? kSmemLimit : (kSmemLimit + 1024) / 2 - 1024) - STATIC;
  static constexpr int FIT = (PER_CTA - FIXED) / (SLOT + 2 * TILE) / 2 * 2;
  static constexpr int NSLOT = FIT > 12 ? 12 : FIT;      // even: keys in even slots, values in odd ones
  static constexpr uint32_t S_COLS = KP * NS;            // of one score buffer
  static constexpr int SB_FIT = (512 / CTAS - 2 * NPV) / S_COLS;
  static constexpr int SB = SB_FIT < NSLOT / 2 ? SB_FIT : NSLOT / 2;   // score buffers
  __host__ __device__ static constexpr uint32_t S_COL(int buf) { return S_COLS * buf; }
  __host__ __device__ static constexpr uint32_t O_COL(int buf) { return SB * S_COLS + NPV * buf; }
  static constexpr int TMEM = pow2(SB * S_COLS + 2 * NPV);
  static constexpr int DESC_OFF = Q_BYTES + PB * P_TILE + NSLOT * SLOT;
  static constexpr int SMEM = 1024 + DESC_OFF + NSLOT / 2 * 4 * TILE;
  static_assert(NSLOT >= 2 * PB && SB >= 2 && TMEM * CTAS <= 512, "ring or tensor memory");
};

struct KParams {
  const uint16_t* q;
  const uint16_t* descale[2];
  const float* signs;
  const int* block_table;
  const int* seq_lens;
  uint16_t* o;
  float* lse;
  float* o_part;          // [2 C][seg_rows][D]
  float* lse_part;        // [2 C][seg_rows]
  int4* crossing;         // [C]: the segment whose first part CTA c left unfinished
  int* status;
  int B, H, H_kv, n_q, rows, qtiles, segs, seg_rows;
  int num_pages, page_size, page_shift, max_pages, causal;
  int cluster;            // CTAs of a segment's cluster, or 0: shares of the line
  int solo;               // shares of whole segments only
  int most_tokens;        // of a sequence
  float scale_log2;
};

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two float32 as e4m3 codes (lo: low byte), and two codes as exact float16.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_pair_h(uint32_t h2) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h2));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_halves(uint32_t pair) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(pair)));
  return h2;
}
__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
__device__ __forceinline__ uint32_t half2_bits(__half2 x) { return *reinterpret_cast<const uint32_t*>(&x); }
__device__ __forceinline__ void st_shared_v2(uint32_t saddr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(saddr), "r"(a), "r"(b) : "memory");
}

// Whether any of the n threads of named barrier `id` says so.
__device__ __forceinline__ bool any_of(uint32_t id, uint32_t n, bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 q, %3, 0;\n barrier.cta.red.or.pred p, %1, %2, q;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(r)
      : "r"(id), "r"(n), "r"(v ? 1u : 0u)
      : "memory");
  return r != 0;
}

template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[N]) {
  static_assert(N == 4 || N == 8 || N == 16 || N == 32, "columns");
  if constexpr (N == 32) tmem_ld32(taddr, r);
  else if constexpr (N == 16) tmem_ld16(taddr, r);
  else if constexpr (N == 8) tmem_ld8(taddr, r);
  else tmem_ld4(taddr, r);
}
template <int N>
__device__ __forceinline__ void tmem_st_cols(uint32_t taddr, const uint32_t (&r)[N]) {
  if constexpr (N == 8) tmem_st_x8(taddr, r);
  else tmem_st4(taddr, r);
}

// Sums of N values over the warp's lanes: in each round a lane sends half of the values it still
// holds to the lane `step` away and adds what it gets to the others.  Lane l ends with the sum of
// value `which`, the first bits of l from above.
template <int N>
__device__ __forceinline__ float warp_sums(float (&v)[N], int lane, int* which) {
  int held = N, first = 0;
#pragma unroll
  for (int step = 16; step > 0; step >>= 1) {
    if (held > 1) {
      held /= 2;
      const bool up = (lane & step) != 0;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        if (i >= held) break;
        const float send = up ? v[i] : v[i + held], keep = up ? v[i + held] : v[i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, step);
      }
      if (up) first += held;
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], step);
    }
  }
  *which = first;
  return v[0];
}

// Rows that see a key (it stands before their ends) get this mark.  Not inlined: unrolled within the
// softmax it cost 16 query rows 4 % (16 x 8192 tokens 50.5 -> 52.5 us; so 51.0).
__device__ __noinline__ void mark_nan(int* marks, const unsigned* ends, unsigned key, int rows, int mark) {
  for (int e = 0; e < rows; ++e)
    if (key < ends[e]) marks[e] = mark;
}

// Tokens of a sequence; a count out of range is none.
__device__ __forceinline__ int tokens_of(const KParams& p, int b) {
  const int n = __ldcg(p.seq_lens + b);
  return n < 0 || n > p.most_tokens ? 0 : n;
}
template <int TILE>
__device__ __forceinline__ int tiles_of(int len) { return static_cast<int>((static_cast<unsigned>(len) + TILE - 1) / TILE); }

// T units dealt out to the first n of C CTAs (n = min(T, C)), one more to the first `rest` of them.
// The host keeps T below 2^31: the dealing out stands before all else that a CTA does, and in 64 bits
// it took half a microsecond more.
struct Shares {
  int per, rest, T;
  __device__ __forceinline__ Shares(int T_, int C) : T(T_) {
    const unsigned n = max(1, min(T, C));
    per = static_cast<int>(T / n);
    rest = static_cast<int>(T - per * n);
  }
  // first unit of CTA c's (T behind the last that gets one)
  __device__ __forceinline__ int start(int c) const { return min(T, c * per + min(c, rest)); }
  // the CTA that has unit u
  __device__ __forceinline__ int owner(int u) const {
    const int more = rest * (per + 1);
    return u < more ? static_cast<unsigned>(u) / (per + 1) : rest + static_cast<unsigned>(u - more) / per;
  }
};

// A walk over the parts of segments in a share.  A segment is `extra` units for its start and its
// end, then one for each tile but that the first comes with the start: a share that begins in
// the extra ones begins at tile 1.
template <int TILE>
struct Cursor {
  int b, hk, qt;         // sequence, key/value head, 16 query rows of it
  int len;
  int at;                // first unit in the segment
  int extra;
  int solo;              // a segment is all of the share's in which it begins
  int left;              // units of the share from here on
  __device__ __forceinline__ int tiles() const { return tiles_of<TILE>(len); }
  __device__ __forceinline__ int units() const {
    const int rest = tiles() + extra - at;
    return left < rest ? left : rest;
  }
  __device__ __forceinline__ int tile_at(int u) const { return u == 0 ? 0 : solo ? tiles() : max(1, u - extra); }
  __device__ __forceinline__ int first() const { return tile_at(at); }           // tile
  __device__ __forceinline__ int part() const { return tile_at(at + units()) - first(); }   // tiles
  __device__ __forceinline__ void next_part(const KParams& p) {
    left -= units();
    if (left <= 0) return;
    at = 0;
    if (++qt == p.qtiles) {
      qt = 0;
      if (++hk == p.H_kv) {
        hk = 0;
        do {
          len = tokens_of(p, ++b);
        } while (len == 0);
      }
    }
  }
};

// A place in a ring of N buffers, used every STEP-th (a tile's keys stand in even slots, its values
// in odd ones), and the phase of its barriers' use.
template <int N, int STEP = 1>
struct Ring {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    at += STEP;
    if (at >= N) {
      at -= N;
      phase ^= 1u;
    }
  }
};

template <int D, int NR, int TQ, int TP, bool FP16, bool SIGNS>
__global__ void __launch_bounds__(Cfg<D, NR, TQ, TP>::THREADS, Cfg<D, NR, TQ, TP>::CTAS)
    decode_fp4_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const KParams p) {
  using C = Cfg<D, NR, TQ, TP>;
  constexpr int NSLOT = C::NSLOT, KP = C::KP, TILE = C::TILE, NRW = C::NRW;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* const sQ = smem;                              // two query tiles
  // PB tiles of P': a key's 16 columns side by side, the tile's 128 keys, the next 16 columns
  uint8_t* const sP = smem + C::Q_BYTES;
  uint8_t* const sKV = sP + C::PB * C::P_TILE;
  uint8_t* const sDesc = smem + C::DESC_OFF;             // per key slot: TILE key descales, TILE value descales

  __shared__ __align__(8) uint64_t q_full[2], q_empty[2], kv_full[NSLOT], kv_empty[NSLOT], s_full[C::SB], p_full[C::PB],
      o_full[2], o_empty[2], drain_bar[2];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh, issued_sh[2];                 // key and value tiles whose copies have been issued
  __shared__ int warp_sum[2][C::THREADS / 32];
  __shared__ int start_sh[4];                            // where the share begins
  __shared__ unsigned there_sh[NSLOT / 2];               // boxes of a key tile that were copied
  __shared__ __align__(16) float cq_sh[2][NR];           // of a part's query rows: score coefficients,
  __shared__ unsigned vend_sh[2][NR];                    // ends of the visible tokens,
  __shared__ float2 ref_sh[2][NR];                       // c and -M at its end,
  __shared__ __align__(16) float l_sh[2][NR][4];         // sums by key quarter
  __shared__ __align__(16) float red_sh[2][2][NR][4];    // maxima of a tile (by parity) by key quarter
  // part + 1 where a row sees a NaN among the values that not all rows see.  (Of four parts: a warp may be in the
  // part after the next while another still writes one out.)
  __shared__ int nan_sh[4][NR];
  __shared__ float part_lse[NR];                         // of the partial results of a cluster's CTA
  __shared__ float xch_sh[KP == 2 ? NR : 1][KP == 2 ? 64 : 1];

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], C::QW);
      mbar_init(&q_empty[i], 1 + C::SW);
      mbar_init(&o_full[i], 1);
      mbar_init(&o_empty[i], C::SW);
      mbar_init(&drain_bar[i], 1);
    }
    for (int i = 0; i < C::SB; ++i) mbar_init(&s_full[i], 1);
    for (int i = 0; i < C::PB; ++i) mbar_init(&p_full[i], C::SW);
    for (int s = 0; s < NSLOT; ++s) {
      mbar_init(&kv_full[s], s & 1 ? 1 : 33);            // keys: the tile's bytes, and each lane's descales
      mbar_init(&kv_empty[s], s & 1 ? 1 : C::SW);
    }
    abort_sh = 0;
    issued_sh[0] = issued_sh[1] = 0;
    fence_mbar_init();
  }
  if (warp == C::MMA_S) {
    tmem_alloc(&tmem_base_sh, C::TMEM);
    tmem_relinquish();
  }
  if (threadIdx.x == C::LOAD * 32) {
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  // columns that no row of queries or of P' fills stay zero
  for (int i = threadIdx.x; i < (C::Q_BYTES + C::PB * C::P_TILE) / 16; i += C::THREADS)
    reinterpret_cast<uint4*>(sQ)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (threadIdx.x < 4 * NR) nan_sh[0][threadIdx.x] = 0;
  fence_proxy_async_smem();
  wait_for_previous_kernel();

  int T = 0, g0 = 0, total = 0;       // units of all, first of this CTA and its number
  int extra = 0;
  const int ranks = p.cluster > 0 ? p.cluster : 1, seg = static_cast<int>(blockIdx.x) / ranks;
  const int rank = static_cast<int>(blockIdx.x) - seg * ranks;
  if (p.cluster > 0) {
    if (threadIdx.x == 0) {
      const int b = seg / p.segs, len = tokens_of(p, b);
      if (len == 0 && seg % p.segs == 0 && rank == 0 && __ldcg(p.seq_lens + b) != 0) atomicCAS(p.status, 0, kDevBadSeqlens);
      start_sh[2] = len;
    }
  } else {
    // ---- units of one segment of the entries before each; this CTA's share
    const int per = (p.B + C::THREADS - 1) / C::THREADS, warps = (p.B + 32 * per - 1) / (32 * per);
    const int b0 = min(static_cast<int>(threadIdx.x) * per, p.B), b1 = min(b0 + per, p.B);
    int sum = 0, len = 0, some = 0;           // some: entries with tokens
    int base = 0, base_some = 0, all = 0, all_some = 0;
    if (warp < warps) {
      for (int b = b0; b < b1; ++b) {
        len = tokens_of(p, b);
        if (len == 0 && blockIdx.x == 0 && __ldcg(p.seq_lens + b) != 0) atomicCAS(p.status, 0, kDevBadSeqlens);
        sum += tiles_of<TILE>(len);
        some += len > 0;
      }
      base = sum;
      base_some = some;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, base, o), z = __shfl_up_sync(0xffffffffu, base_some, o);
        if (lane >= o) {
          base += x;
          base_some += z;
        }
      }
      if (lane == 31) {
        warp_sum[0][warp] = base;
        warp_sum[1][warp] = base_some;
      }
      base -= sum;
      base_some -= some;
    }
    __syncthreads();
    for (int w = 0; w < warps; ++w) {
      if (w < warp) {
        base += warp_sum[0][w];
        base_some += warp_sum[1][w];
      }
      all += warp_sum[0][w];
      all_some += warp_sum[1][w];
    }
    // A part's start and end are counted as tiles, as far as a share has four times as many (64
    // sequences of up to 16384 tokens, d = 64: 75 us without them, 66.6 so; two tiles instead of one 67.0).
    extra = static_cast<int>(fminf(C::PART, __fdividef(static_cast<float>(all) * p.segs, 4.f * gridDim.x)));
    base += extra * base_some;
    sum += extra * some;
    T = (all + extra * all_some) * p.segs;
    const Shares shares(T, gridDim.x);
    g0 = shares.start(blockIdx.x);
    total = shares.start(blockIdx.x + 1) - g0;
    if (total > 0 && base * p.segs <= g0 && g0 < (base + sum) * p.segs) {
      int b = b0;
      for (; b1 - b0 > 1; ++b) {
        len = tokens_of(p, b);
        const int n = len > 0 ? tiles_of<TILE>(len) + extra : 0;
        if (g0 < (base + n) * p.segs) break;
        base += n;
      }
      const int n = tiles_of<TILE>(len) + extra;
      const int in = g0 - base * p.segs, y = in / n;
      start_sh[0] = b;
      start_sh[1] = y;
      start_sh[2] = len;
      start_sh[3] = in - y * n;
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  release_dependents();       // not before this CTA has its tensor memory: the next kernel may want some
  const uint32_t tmem = tmem_base_sh;
  const Abort ab{&abort_sh, p.status};

  Cursor<TILE> cur{0, 0, 0, 0, 0, extra, p.solo, 0};
  if (p.cluster > 0) {
    cur.b = seg / p.segs;
    cur.hk = (seg - cur.b * p.segs) / p.qtiles;
    cur.qt = seg - cur.b * p.segs - cur.hk * p.qtiles;
    cur.len = start_sh[2];
    const unsigned n = cur.tiles();
    cur.at = rank * n / ranks;
    cur.left = (rank + 1) * n / ranks - cur.at;
  } else if (total > 0) {
    cur.left = total;
    cur.b = start_sh[0];
    cur.hk = start_sh[1] / p.qtiles;
    cur.qt = start_sh[1] - cur.hk * p.qtiles;
    cur.len = start_sh[2];
    cur.at = start_sh[3];
    if (cur.part() == 0) cur.next_part(p);            // its tiles are the CTA's before
  }
  const Cursor<TILE> begin = cur;

  if (warp >= C::LOAD && warp < C::LOAD + C::LW) {
    // ------------------------------------------------------------ producer
    // A tile is fetched page by page: a box is min(page_size, TILE) tokens of one page, at most
    // 16 of them.  Lane x issues box x (a copy costs its warp some hundred clocks).  The descales of
    // the tile's keys and values come with its keys, by 16-byte copies of all lanes (8 tokens each; a
    // bulk copy for each page took as long as the codes' own).  The pages of 32 boxes are read from
    // the block table at a time, the next 32 while those are in use.  Boxes behind the sequence are
    // left out, as are those on pages outside the cache (reported): what the slot held before is
    // finite codes, and their tokens are masked.
    const int box_shift = min(p.page_shift, KP == 2 ? 8 : 7), box = 1 << box_shift, nbox = TILE >> box_shift;
    int n = 0;
    Ring<NSLOT, 2> key_slot;
    bool ok = true;
    while (ok && cur.left > 0) {
      const int take = cur.part(), hk = cur.hk, kbeg = cur.first() * TILE;   // kbeg < len
      auto window = [&](int w) -> int {
        const long long key = kbeg + static_cast<long long>(32 * w + lane) * box;
        if (key >= cur.len || 32 * w + lane >= take * nbox) return -1;
        return __ldcg(p.block_table + static_cast<size_t>(cur.b) * p.max_pages + (key >> p.page_shift));
      };
      int win = window(0), win_next = window(1);
      for (int i = 0; ok && i < take; ++i, ++n, key_slot.next()) {
        if (i > 0 && ((i * nbox) & 31) == 0) {
          win = win_next;
          win_next = window(i * nbox / 32 + 1);
        }
        const int box_at = (i * nbox) & 31;
        const int phys = __shfl_sync(0xffffffffu, win, (box_at + lane) & 31);
        const long long key = static_cast<long long>(kbeg) + i * TILE + lane * box;
        const bool wanted = lane < nbox && key < cur.len;
        const bool good = wanted && phys >= 0 && phys < p.num_pages;
        if (wanted && !good) atomicCAS(p.status, 0, kDevBadSeqlens);
        const unsigned there = __ballot_sync(0xffffffffu, good);
        const int off = static_cast<int>(key) & (p.page_size - 1);
        for (int kv = warp - C::LOAD; kv < 2; kv += C::LW) {
          const int slot = key_slot.at + kv;
          const bool free = n < NSLOT / 2 || mbar_wait(&kv_empty[slot], key_slot.phase ^ 1u, ab, kDevTimeoutLoad);
          if (!__all_sync(0xffffffffu, free)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            if (kv == 0) there_sh[slot / 2] = there;
            mbar_arrive_expect_tx(&kv_full[slot], __popc(there) * box * (D / 2));
            issued_sh[kv] = n + 1;
          }
          __syncwarp();
          if (good)
            tma_load_4d(sKV + slot * C::SLOT + lane * (box / KP) * 128, kv ? &tmV : &tmK, &kv_full[slot], 0, off / KP, hk, phys);
          if (kv == 0) {
            uint8_t* dst = sDesc + slot / 2 * 4 * TILE;
#pragma unroll
            for (int c = lane; c < TILE / 4; c += 32) {          // 16 bytes: keys' first, then values'
              const int tok = c % (TILE / 8) * 8, x = tok >> box_shift;
              const int page = __shfl_sync(0xffffffffu, phys, x);
              const size_t row = ((static_cast<size_t>(page) * p.H_kv + hk) << p.page_shift) +
                                 ((kbeg + i * TILE + tok) & (p.page_size - 1));
              if ((there >> x) & 1u) copy16_async(dst + c * 16, p.descale[c / (TILE / 8)] + row, true);
            }
            copies_arrive(&kv_full[slot]);
          }
        }
      }
      cur.next_part(p);
    }
  } else if (warp == C::MMA_S) {
    // ------------------------------------------------------------ S^T = K^ Q^T
    // S(n) into buffer n % SB, which the softmax has read: it hands a key slot back when it has
    // read that tile's scores, so a key tile that came into a slot used before says so for all
    // tiles before the slot's last one.
    if (lane == 0) {
      constexpr uint32_t id = idesc_e2m1_e4m3(128, C::NS, false, false);
      const uint64_t qdesc0 = sdesc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t kdesc0 = sdesc_sw128(smem_u32(sKV), 16, 1024);
      bool ok = true;
      int n = 0;
      Ring<NSLOT, 2> key, old;              // old: the keys of tile n - SB
      Ring<C::SB> buf;
      for (int part = 0; ok && cur.left > 0; ++part) {
        const int take = cur.part();
        if (!(ok = mbar_wait(&q_full[part & 1], (part >> 1) & 1, ab, kDevTimeoutMma))) break;
        const uint64_t qdesc = opaque(sdesc_add(qdesc0, (part & 1) * C::Q_STEP));
        for (int i = 0; i < take; ++i, ++n, key.next(), buf.next()) {
          if (!(ok = mbar_wait(&kv_full[key.at], key.phase, ab, kDevTimeoutMma))) break;
          if (C::SB < NSLOT / 2 && n >= C::SB) {
            if (!(ok = mbar_wait(&kv_empty[old.at], old.phase, ab, kDevTimeoutMma))) break;
            old.next();
          }
          tc_fence_after_sync();
          const uint64_t kdesc = opaque(sdesc_add(kdesc0, key.at * C::SLOT));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            // d = 64: two 32-column steps for the even tokens, two for the odd ones
            constexpr int steps = D / 32;
            mma_f8_ss(tmem + C::S_COL(buf.at) + kk / steps * C::NS, sdesc_add(kdesc, kk * 32),
                      sdesc_add(qdesc, kk % steps * 32), id, kk % steps > 0 ? 1u : 0u);
          }
          mma_commit(&s_full[buf.at]);
        }
        if (ok) mma_commit(&q_empty[part & 1]);
        cur.next_part(p);
      }
    }
  } else if (warp == C::MMA_PV) {
    // ------------------------------------------------------------ O^T += V^^T P'^T
    if (lane == 0) {
      constexpr uint32_t id = idesc_e2m1_e4m3(128, C::NPV, true, true);
      const uint64_t pdesc0 = sdesc_mn_plain(smem_u32(sP), 128 * 16, 128);     // MN-major
      const uint64_t vdesc0 = sdesc_sw128(smem_u32(sKV), C::SLOT, 1024);
      bool ok = true;
      Ring<NSLOT, 2> val;                   // (the odd slot behind)
      Ring<C::PB> pb;
      for (int part = 0; ok && cur.left > 0; ++part) {
        const int take = cur.part();
        const uint32_t o_col = C::O_COL(part & 1);
        for (int i = 0; i < take; ++i, val.next(), pb.next()) {
          if (!(ok = mbar_wait(&kv_full[val.at + 1], val.phase, ab, kDevTimeoutMma))) break;
          const uint64_t vdesc = opaque(sdesc_add(vdesc0, (val.at + 1) * C::SLOT));
          if (!(ok = mbar_wait(&p_full[pb.at], pb.phase, ab, kDevTimeoutMma))) break;
          // the buffer's output of two parts ago has been read
          if (i == 0 && part >= 2 && !(ok = mbar_wait(&o_empty[part & 1], ((part >> 1) - 1) & 1, ab, kDevTimeoutMma))) break;
          tc_fence_after_sync();
          const uint64_t pdesc = sdesc_add(pdesc0, pb.at * C::P_TILE);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f8_ss(tmem + o_col, sdesc_add(vdesc, kk * 32 * 128), sdesc_add(pdesc, kk * 32 * 16), id,
                      (i > 0 || kk > 0) ? 1u : 0u);
          mma_commit(&kv_empty[val.at + 1]);  // every use of a value slot gets its phase
          if (i == take - 1) mma_commit(&o_full[part & 1]);
        }
        cur.next_part(p);
      }
    }
  } else if (warp >= C::QUERY) {
    // ------------------------------------------------------------ query rows as e4m3 terms
    // d / 16 lanes hold a row, 16 neighbouring columns each.
    constexpr int L = D / 16, PER = 32 / L, PASSES = (NR + PER - 1) / PER / C::QW;
    const int u = lane % L, first_row = (warp - C::QUERY) * PASSES * PER;
    float4 sgn[4];
    if constexpr (SIGNS) {
#pragma unroll
      for (int i = 0; i < 4; ++i) sgn[i] = __ldcg(reinterpret_cast<const float4*>(p.signs + 16 * u) + i);
    }
    bool ok = true;
    int4 crossing = make_int4(0, 0, 0, -1);            // a segment that this share begins and does not end
    for (int part = 0; ok && cur.left > 0; ++part) {
      const int buf = part & 1;
      if (part >= 2 && __any_sync(0xffffffffu, !mbar_wait(&q_empty[buf], ((part >> 1) - 1) & 1, ab, kDevTimeoutLoad))) {
        ok = false;
        break;
      }
      const int row0 = cur.qt * 16;
      const size_t at0 = (static_cast<size_t>(cur.b) * p.H_kv + cur.hk) * p.rows + row0;
      const int rows_here = min(NR, p.rows - row0);
      uint4 raw[PASSES][2];
#pragma unroll
      for (int x = 0; x < PASSES; ++x) {
        const int r = first_row + x * PER + lane / L;
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (at0 + (r < rows_here ? r : 0)) * D + 16 * u);
        raw[x][0] = __ldcg(src);
        raw[x][1] = __ldcg(src + 1);
      }
#pragma unroll
      for (int pass = 0; pass < PASSES; ++pass) {
        const int r = first_row + pass * PER + lane / L;
        const bool live = r < rows_here;
        float x[16];
        {
          float lo[8], hi[8];
          unpack16<FP16>(raw[pass][0], lo);
          unpack16<FP16>(raw[pass][1], hi);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = live ? lo[i] : 0.f, x[8 + i] = live ? hi[i] : 0.f;
        }
        if constexpr (SIGNS) {
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            // of x / d, so that the sums stay in range, and sqrt(d) at their end: the same bits
            const float4 s = sgn[i / 4];
            const uint64_t down = pack2(1.f / D, 1.f / D);
            const uint64_t a = fmul2(fmul2(pack2(x[i], x[i + 1]), pack2(s.x, s.y)), down);
            const uint64_t b = fmul2(fmul2(pack2(x[i + 2], x[i + 3]), pack2(s.z, s.w)), down);
            x[i] = lo2(a), x[i + 1] = hi2(a), x[i + 2] = lo2(b), x[i + 3] = hi2(b);
          }
#pragma unroll
          for (int h = 1; h < 16; h <<= 1)
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if ((i & h) == 0) {
                const float a = x[i], b = x[i + h];
                x[i] = a + b;
                x[i + h] = a - b;
              }
#pragma unroll
          for (int m = 1; m < L; m <<= 1) {
            const float minus = (u & m) ? -1.f : 1.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = fmaf(minus, x[i], __shfl_xor_sync(0xffffffffu, x[i], m));
          }
          const float root = D == 128 ? 11.313708498984761f : 8.f;      // sqrt(d)
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] *= root;
        }
        uint32_t top = 0u;
#pragma unroll
        for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
        for (int m = 1; m < L; m <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
        // times f = 2^(7 - floor(log2 top)), at most 2^126, so that 1 / f is a normal number too; a row with an
        // infinity or a NaN gets a coefficient of NaN
        const int e = static_cast<int>(top >> 23);
        const int up = top == 0u ? 127 : min(261 - e, 253);
        const float f = __uint_as_float(static_cast<uint32_t>(up) << 23);
        const float back = e == 255 ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float(static_cast<uint32_t>(254 - up) << 23);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] *= f;
#pragma unroll
        for (int k = 0; k < TQ; ++k) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a = e4m3_pair(x[4 * i], x[4 * i + 1]), b = e4m3_pair(x[4 * i + 2], x[4 * i + 3]);
            w[i] = a | (b << 16);
            if (k + 1 < TQ) {
              const float2 fa = __half22float2(as_half2(e4m3_halves(a))), fb = __half22float2(as_half2(e4m3_halves(b)));
              const uint64_t up = pack2(1 << kPStep, 1 << kPStep), down = pack2(-(1 << kPStep), -(1 << kPStep));
              const uint64_t ra = ffma2(pack2(x[4 * i], x[4 * i + 1]), up, fmul2(pack2(fa.x, fa.y), down));
              const uint64_t rb = ffma2(pack2(x[4 * i + 2], x[4 * i + 3]), up, fmul2(pack2(fb.x, fb.y), down));
              x[4 * i] = lo2(ra), x[4 * i + 1] = hi2(ra), x[4 * i + 2] = lo2(rb), x[4 * i + 3] = hi2(rb);
            }
          }
          const int col = k * NR + r;
          if (r < NR) {
            const int piece = KP == 2 ? 4 * buf + u : u;         // of the row's eight
            uint8_t* tile = KP == 2 ? sQ : sQ + buf * C::Q_STEP;
            st_shared_v4(smem_u32(tile + col * 128 + ((piece ^ (col & 7)) << 4)), w[0], w[1], w[2], w[3]);
          }
        }
        if (u == 0 && r < NR) {
          cq_sh[buf][r] = p.scale_log2 * back;
          vend_sh[buf][r] = live ? max(p.causal ? min(cur.len, cur.len - p.n_q + (row0 + r) % p.n_q + 1) : cur.len, 0) : 0;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[buf]);
      if (p.cluster == 0 && cur.first() == 0 && cur.part() < cur.tiles()) {
        // the CTA whose share holds the segment's last unit
        const int last = g0 + (total - cur.left) - cur.at + cur.tiles() + extra - 1;
        crossing = make_int4(static_cast<int>(at0), rows_here, Shares(T, gridDim.x).owner(last),
                             static_cast<int>(2 * blockIdx.x + (part > 0 ? 1 : 0)));
      }
      cur.next_part(p);
    }
    if (lane == 0 && warp == C::QUERY && p.cluster == 0) p.crossing[blockIdx.x] = crossing;
    // batch entries without tokens: O = 0, LSE = -inf (a cluster's joining finds them)
    for (int b = blockIdx.x; p.cluster == 0 && warp == C::QUERY && b < p.B; b += gridDim.x) {
      if (tokens_of(p, b) != 0) continue;
      const size_t rows_b = static_cast<size_t>(p.H) * p.n_q;
      uint4* dst = reinterpret_cast<uint4*>(p.o + b * rows_b * D);
      for (size_t i = lane; i < rows_b * (D / 8); i += 32) dst[i] = make_uint4(0u, 0u, 0u, 0u);
      for (size_t i = lane; i < rows_b; i += 32) p.lse[b * rows_b + i] = -INFINITY;
    }
  } else {
    // ------------------------------------------------------------ softmax
    // Thread (quarter, lane): tile row t, of KP tokens; query rows [r0, r0 + NRW); in O^T
    // the lane t of those rows' columns.
    const int t = (warp & 3) * 32 + lane, cg = warp >> 2, r0 = cg * NRW;
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t bar = 1 + cg;          // of the four warps that have the same query rows
    constexpr uint32_t MEMBERS = 128;
    const int box_shift = min(p.page_shift, KP == 2 ? 8 : 7);
    const unsigned all_boxes = 0xFFFFu >> (16 - (TILE >> box_shift));
    const int o_half = KP == 2 && (warp & 2) ? NR * TP : 0;    // columns that hold this lane's sums
    // A wait that gives up sets the CTA's abort flag, on which all others end at once; these
    // warps go on through their barriers, and what they write is reported as invalid.
    // output of a finished part: where it goes, and its rows' references
    struct Done {
      int part, rows;
      bool whole;
      size_t at0;
    } done;
    done.part = -1;
    // Every softmax thread comes here at the same point, also after giving up (the barriers).
    auto write_out = [&]() {
      const int buf = done.part & 1;
      mbar_wait(&o_full[buf], (done.part >> 1) & 1, ab, kDevTimeoutEpilogue);
      __syncwarp();
      tc_fence_after_sync();
      float o[NRW];
#pragma unroll
      for (int i = 0; i < NRW; ++i) o[i] = 0.f;
      uint32_t raw[TP][NRW];
#pragma unroll
      for (int k = 0; k < TP; ++k) tmem_ld_cols<NRW>(tmem + lane_addr + C::O_COL(buf) + o_half + k * NR + r0, raw[k]);
      tmem_ld_wait();
#pragma unroll
      for (int k = TP - 1; k >= 0; --k)
#pragma unroll
        for (int i = 0; i < NRW; ++i) o[i] = fmaf(o[i], 1.f / (1 << kPStep), __uint_as_float(raw[k][i]));
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_empty[buf]);
      if (KP == 2 && (warp & 2)) {
#pragma unroll
        for (int i = 0; i < NRW; ++i) xch_sh[KP == 2 ? r0 + i : 0][KP == 2 ? t - 64 : 0] = o[i];
      }
      named_bar_sync(bar, MEMBERS);                            // the sums of rows are there, too
      if (KP == 1 || !(warp & 2)) {
        // lane i: factor and log-sum-exp of row i
        const int mine = r0 + (lane & (NRW - 1));
        const float4 l4 = *reinterpret_cast<const float4*>(l_sh[buf][mine]);
        const float l = ((l4.x + l4.y) + l4.z) + l4.w;
        const float2 ref = ref_sh[buf][mine];
        // (a NaN among the scores or the descales that all rows see is in o by now, and stays)
        const float f = nan_sh[done.part & 3][mine] == done.part + 1 ? __uint_as_float(0x7FFFFFFFu)
                        : l == 0.f                                   ? 0.f
                                                                     : __fdividef(__fdividef(1.f, ref.x), l);   // (all below 2^126)
        const float lse = l == 0.f ? -INFINITY : (lg2(l) - ref.y) * 0.69314718055994530942f;
        // (a cluster's partial results: in its ring's place, which is free by then)
        const size_t at = done.whole ? done.at0 : p.cluster > 0 ? 0 : (2ull * blockIdx.x + (done.part > 0 ? 1 : 0)) * p.seg_rows;
        if ((warp & 3) == 0 && lane < NRW && mine < done.rows)
          (done.whole ? p.lse : p.cluster > 0 ? part_lse : p.lse_part)[at + mine] = lse;
#pragma unroll
        for (int i = 0; i < NRW; ++i) {
          if constexpr (KP == 2) o[i] += xch_sh[r0 + i][t];
          o[i] *= __shfl_sync(0xffffffffu, f, i);
        }
        const int rows = done.rows - r0;
        if (done.whole) {
          uint16_t* const dst = p.o + (at + r0) * D + t;
#pragma unroll
          for (int i = 0; i < NRW; ++i)
            if (i < rows) dst[i * D] = static_cast<uint16_t>(FP16 ? cvt_pack_f16(o[i], 0.f) : cvt_pack_bf16(o[i], 0.f));
        } else {
          float* const dst = (p.cluster > 0 ? reinterpret_cast<float*>(sKV) : p.o_part) + (at + r0) * D + t;
#pragma unroll
          for (int i = 0; i < NRW; ++i)
            if (i < rows) dst[i * D] = o[i];
        }
      }
      if constexpr (KP == 2) named_bar_sync(bar, MEMBERS);     // xch_sh has been read
    };

    int n = 0;
    // SAME: scores and P' of a tile are in the buffers of its slot's number
    constexpr bool SAME = C::SB == NSLOT / 2 && C::PB == NSLOT / 2;
    Ring<NSLOT, 2> key, last, used;         // last: tile n - 1; used: tile n - PB
    Ring<C::SB> sb;
    Ring<C::PB> pb;
    for (int part = 0; cur.left > 0; ++part) {
      const int take = cur.part(), len = cur.len, first_tile = cur.first();
      mbar_wait(&q_full[part & 1], (part >> 1) & 1, ab, kDevTimeoutSoftmax);
      __syncwarp();
      // mm = -M, at first so large that any finite score moves it.
      float c[NRW], mm[NRW], lsum[NRW];
#pragma unroll
      for (int i = 0; i < NRW; ++i) {
        c[i] = 1.f;
        mm[i] = kFar;
        lsum[i] = 0.f;
      }
      const unsigned vis_all = max(p.causal ? len - p.n_q + 1 : len, 0);   // seen by every row
      for (int i = 0; i < take; ++i, ++n) {
        const int kslot = key.at, sbuf = SAME ? kslot / 2 : sb.at;
        // (the keys' barrier is complete then: what came with them is seen)
        const bool ready = mbar_test_wait(&s_full[sbuf], SAME ? key.phase : sb.phase), seen_too = mbar_test_wait(&kv_full[kslot], key.phase);
        if (!(ready && seen_too)) {
          mbar_wait(&s_full[sbuf], SAME ? key.phase : sb.phase, ab, kDevTimeoutSoftmax);
          mbar_test_wait(&kv_full[kslot], key.phase);
        }
        __syncwarp();
        tc_fence_after_sync();
        constexpr int LD = C::CW == 1 ? C::NS : TQ * NRW;      // columns read
        uint32_t raw[KP][LD];
#pragma unroll
        for (int h = 0; h < KP; ++h) {
          const uint32_t at = tmem + lane_addr + C::S_COL(sbuf) + h * C::NS;
          if constexpr (C::CW == 1) {
            tmem_ld_cols<LD>(at, raw[h]);
          } else {
#pragma unroll
            for (int k = 0; k < TQ; ++k) tmem_ld_cols<NRW>(at + k * NR + r0, *reinterpret_cast<uint32_t(*)[NRW]>(&raw[h][k * NRW]));
          }
        }
        uint32_t ks2, vs2;         // descales of the thread's tokens (d = 64: two)
        const uint8_t* desc = sDesc + kslot / 2 * 4 * TILE;
        if constexpr (KP == 2) {
          ks2 = *reinterpret_cast<const uint32_t*>(desc + 4 * t);
          vs2 = *reinterpret_cast<const uint32_t*>(desc + 2 * TILE + 4 * t);
        } else {
          ks2 = *reinterpret_cast<const uint16_t*>(desc + 2 * t);
          vs2 = *reinterpret_cast<const uint16_t*>(desc + 2 * TILE + 2 * t);
        }
        const unsigned tile0 = static_cast<unsigned>(first_tile + i) * TILE, key0 = tile0 + KP * t;
        const unsigned boxes = there_sh[kslot / 2];
        const bool there = (boxes >> (KP * t >> box_shift)) & 1u;
        const bool open = tile0 + TILE <= vis_all && boxes == all_boxes;
        tmem_ld_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&kv_empty[kslot]);
        // scores in log2 units
        float s[KP][NRW], sv[KP];
#pragma unroll
        for (int h = 0; h < KP; ++h) {
          const float ks = h ? __uint_as_float(ks2 & 0xFFFF0000u) : bf16_bits(ks2);
          sv[h] = h ? __uint_as_float(vs2 & 0xFFFF0000u) : bf16_bits(vs2);
          const uint64_t ks_2 = pack2(ks, ks), step = pack2(1.f / (1 << kPStep), 1.f / (1 << kPStep));
#pragma unroll
          for (int e = 0; e < NRW; e += 2) {
            auto pair = [&](int k) {
              const int c = k * (C::CW == 1 ? NR : NRW) + e;
              return pack2(__uint_as_float(raw[h][c]), __uint_as_float(raw[h][c + 1]));
            };
            uint64_t x = pair(TQ - 1);
#pragma unroll
            for (int k = TQ - 2; k >= 0; --k) x = ffma2(x, step, pair(k));
            const float2 cq = *reinterpret_cast<const float2*>(&cq_sh[part & 1][r0 + e]);
            x = fmul2(x, fmul2(pack2(cq.x, cq.y), ks_2));
            s[h][e] = lo2(x), s[h][e + 1] = hi2(x);
          }
          if (!open) {
            // (a slot without a token may hold any descale)
            if (!there || key0 + h >= static_cast<unsigned>(len)) sv[h] = 0.f;
            // 0 times NaN is NaN: of a token that only some rows see, NaN goes to those when they are written
            if (__builtin_expect(key0 + h >= vis_all && sv[h] != sv[h], 0)) {
              mark_nan(&nan_sh[part & 3][r0], &vend_sh[part & 1][r0], key0 + h, NRW, part + 1);
              sv[h] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < NRW; ++e) {
              const bool seen = there && key0 + h < vend_sh[part & 1][r0 + e];
              s[h][e] = seen ? s[h][e] : -INFINITY;
            }
          }
        }
        uint64_t pr[KP][NRW / 2], pv[KP][NRW / 2];             // p and P'
        bool need = false;
        auto weigh = [&]() {
          need = false;
#pragma unroll
          for (int h = 0; h < KP; ++h)
#pragma unroll
            for (int e = 0; e < NRW; e += 2) {
              const uint64_t a = fadd2(pack2(s[h][e], s[h][e + 1]), pack2(mm[e], mm[e + 1]));
              pr[h][e / 2] = pack2(ex2_approx(lo2(a)), ex2_approx(hi2(a)));
              // (c s^v may overflow where p is 0; p s^v, once p is 1 at most, does not)
              pv[h][e / 2] = fmul2(fmul2(pr[h][e / 2], pack2(sv[h], sv[h])), pack2(c[e], c[e + 1]));
              need |= fmaxf(lo2(pv[h][e / 2]), hi2(pv[h][e / 2])) > kPTop || fmaxf(lo2(a), hi2(a)) > 64.f;
            }
        };
        if (i > 0) weigh();
        if (i == 0 || any_of(bar, MEMBERS, need)) {
          // references move to the maxima over the tile
          float lv[KP];
#pragma unroll
          for (int h = 0; h < KP; ++h) lv[h] = lg2(sv[h]);
#pragma unroll
          for (int e = 0; e < NRW; ++e) {
            float my = s[0][e] + lv[0], ms = s[0][e];
            if constexpr (KP == 2) {
              my = fmaxf(my, s[KP - 1][e] + lv[KP - 1]);
              ms = fmaxf(ms, s[KP - 1][e]);
            }
            asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(my) : "f"(my));
            asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(ms) : "f"(ms));
            if (lane == 0) {
              red_sh[n & 1][0][r0 + e][warp & 3] = my;
              red_sh[n & 1][1][r0 + e][warp & 3] = ms;
            }
          }
          named_bar_sync(bar, MEMBERS);
          // lane x: row x % NRW
          const int mine = lane & (NRW - 1);
          float m_old = mm[0], c_old = c[0];
#pragma unroll
          for (int e = 1; e < NRW; ++e) {
            m_old = mine == e ? mm[e] : m_old;
            c_old = mine == e ? c[e] : c_old;
          }
          const float4 y4 = *reinterpret_cast<const float4*>(red_sh[n & 1][0][r0 + mine]);
          const float4 m4 = *reinterpret_cast<const float4*>(red_sh[n & 1][1][r0 + mine]);
          const float ty = fmaxf(fmaxf(y4.x, y4.y), fmaxf(y4.z, y4.w));
          const float m_new = fminf(m_old, -fmaxf(fmaxf(m4.x, m4.y), fmaxf(m4.z, m4.w)));
          const bool none = m_new == kFar;                       // no token yet
          const float by = ex2_approx(m_new - m_old);            // 0 at the first token
          const float t_old = m_old == kFar ? -INFINITY : kPShift - m_old - lg2(c_old);
          const float t_new = fmaxf(fmaxf(t_old, ty), kPShift - kMostC - m_new);
          const float c_new = none ? 1.f : ex2_approx(kPShift - m_new - t_new);
          const float alpha = by * __fdividef(c_new, c_old);     // (c: 2^-123 .. 2^120)
          const bool grew = __any_sync(0xffffffffu, !none && t_new > t_old);
#pragma unroll
          for (int e = 0; e < NRW; ++e) {
            mm[e] = __shfl_sync(0xffffffffu, m_new, e);
            c[e] = __shfl_sync(0xffffffffu, c_new, e);
            lsum[e] *= __shfl_sync(0xffffffffu, by, e);
          }
          weigh();
          if (i > 0 && grew) {
            // O^T times alpha once P' V(n - 1) is in it (the phase of its value slot's empty barrier)
            mbar_wait(&kv_empty[last.at + 1], last.phase, ab, kDevTimeoutSoftmax);
            __syncwarp();
            tc_fence_after_sync();
#pragma unroll
            for (int k = 0; k < TP; ++k) {
              uint32_t o[NRW];
              const uint32_t at = tmem + lane_addr + C::O_COL(part & 1) + o_half + k * NR + r0;
              tmem_ld_cols<NRW>(at, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < NRW; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * __shfl_sync(0xffffffffu, alpha, e));
              tmem_st_cols<NRW>(at, o);
            }
            tmem_st_wait();
          }
        }
        if (n >= C::PB) {
          // P' of tile n - PB has been multiplied
          if constexpr (SAME) {
            mbar_wait(&kv_empty[kslot + 1], key.phase ^ 1u, ab, kDevTimeoutSoftmax);
          } else {
            mbar_wait(&kv_empty[used.at + 1], used.phase, ab, kDevTimeoutSoftmax);
            used.next();
          }
        }
        // probabilities as e4m3 terms: column (h TP + k) NR + row, four of them a word
        uint32_t w[KP][TP][NRW / 4];
#pragma unroll
        for (int h = 0; h < KP; ++h)
#pragma unroll
          for (int e = 0; e < NRW; e += 2) {
            lsum[e] += lo2(pr[h][e / 2]);
            lsum[e + 1] += hi2(pr[h][e / 2]);
            __half2 x = as_half2(cvt_pack_f16(lo2(pv[h][e / 2]), hi2(pv[h][e / 2])));
#pragma unroll
            for (int k = 0; k < TP; ++k) {
              const uint32_t code = e4m3_pair_h(half2_bits(x));
              if (k + 1 < TP) x = __hmul2(__hsub2(x, as_half2(e4m3_halves(code))), __float2half2_rn(1 << kPStep));
              w[h][k][e / 4] = e & 2 ? w[h][k][e / 4] | (code << 16) : code;
            }
          }
        {
          const uint32_t at = smem_u32(sP + (SAME ? key.at / 2 : pb.at) * C::P_TILE) + t * 16;
          if constexpr (C::CW == 1) {
            // all columns of the key: words 4 i .. 4 i + 3 are its i-th 16
            constexpr int n_words = KP * TP * NR / 4;
            const uint32_t* const ws = &w[0][0][0];
#pragma unroll
            for (int i = 0; i < n_words; i += 4) {
              const uint32_t dst = at + i / 4 * 128 * 16;
              if (n_words - i >= 4) st_shared_v4(dst, ws[i], ws[i + 1], ws[i + 2], ws[i + 3]);
              else if (n_words - i == 3) st_shared_v4(dst, ws[i], ws[i + 1], ws[i + 2], 0u);
              else st_shared_v2(dst, ws[i], ws[i + 1]);
            }
          } else {
#pragma unroll
            for (int h = 0; h < KP; ++h)
#pragma unroll
              for (int k = 0; k < TP; ++k) st_shared_v2(at + (h * TP + k) * 128 * 16 + r0, w[h][k][0], w[h][k][1]);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[SAME ? key.at / 2 : pb.at]);
        last = key;
        key.next();
        if constexpr (!SAME) {
          sb.next();
          pb.next();
        }
        // the part before this one, while this tile's products run
        if (i == 0 && part > 0) write_out();
      }
      // this part's row sums, and what its output needs
      int which;
      const float row_sum = warp_sums<NRW>(lsum, lane, &which);
      l_sh[part & 1][r0 + which][warp & 3] = row_sum;          // (several lanes, the same value)
      float c_mine = c[0], mm_mine = mm[0];
#pragma unroll
      for (int e = 1; e < NRW; ++e) {
        c_mine = (lane & (NRW - 1)) == e ? c[e] : c_mine;
        mm_mine = (lane & (NRW - 1)) == e ? mm[e] : mm_mine;
      }
      ref_sh[part & 1][r0 + (lane & (NRW - 1))] = make_float2(c_mine, mm_mine);
      // the part's coefficients and ends have been read
      if (lane == 0) mbar_arrive(&q_empty[part & 1]);
      done.part = part;
      done.rows = min(NR, p.rows - cur.qt * 16);
      done.whole = p.cluster == 0 && take == cur.tiles();
      done.at0 = (static_cast<size_t>(cur.b) * p.H_kv + cur.hk) * p.rows + cur.qt * 16;
      cur.next_part(p);
    }
    if (done.part >= 0) write_out();
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before_sync();
  __syncthreads();
  if (abort_sh) {
    // let every copy and product this CTA issued land before the memory goes away
    if (warp == C::LOAD && lane < 2) {
      const int kv = lane, n = issued_sh[kv];
      for (int i = n - 1; i >= 0 && i >= n - NSLOT / 2; --i)
        mbar_wait_drain(&kv_full[2 * (i % (NSLOT / 2)) + kv], (i / (NSLOT / 2)) & 1);
    }
    if ((warp == C::MMA_S || warp == C::MMA_PV) && lane == 0) {
      uint64_t* bar = &drain_bar[warp == C::MMA_S ? 0 : 1];
      mma_commit(bar);
      mbar_wait_drain(bar, 0);
    }
    __syncthreads();
  }
  if (warp == C::MMA_S) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, C::TMEM);
  }
  if (p.cluster > 0) {
    // Every thread of every CTA comes here, after an abort too.  The cluster's threads share the
    // segment's rows, four columns each.
    if (begin.left <= 0 && threadIdx.x < NR) part_lse[threadIdx.x] = -INFINITY;
    cluster_sync();
    const int row0 = begin.qt * 16;
    const size_t at0 = (static_cast<size_t>(begin.b) * p.H_kv + begin.hk) * p.rows + row0;
    const int items = min(NR, p.rows - row0) * (D / 4);
    for (int x = rank * C::THREADS + static_cast<int>(threadIdx.x); x < items; x += ranks * C::THREADS) {
      const int r = x / (D / 4), c4 = x % (D / 4);
      float lse[8], m = -INFINITY;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        lse[i] = i < ranks ? ld_cluster_f32(smem_u32(part_lse + r), i) : -INFINITY;
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
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const uint2 pk = FP16 ? make_uint2(cvt_pack_f16(acc.x * inv, acc.y * inv), cvt_pack_f16(acc.z * inv, acc.w * inv))
                            : make_uint2(cvt_pack_bf16(acc.x * inv, acc.y * inv), cvt_pack_bf16(acc.z * inv, acc.w * inv));
      *reinterpret_cast<uint2*>(p.o + (at0 + r) * D + 4 * c4) = pk;
      if (c4 == 0) p.lse[at0 + r] = sum == 0.f ? -INFINITY : m + logf(sum);
    }
    cluster_sync();                                  // the others may still be reading here
  }
}

// Segments that cross shares: LSE = log sum_c exp(lse_c), O = sum_c exp(lse_c - LSE) O_c over
// CTAs c0 .. c1, whose partial results are c0's slot and the others' first ones.  A block for
// every CTA that left a segment unfinished (4 rows of it), D / 4 threads per row.
constexpr int kMergeThreads = 128;
template <int D, bool FP16>
__global__ void __launch_bounds__(kMergeThreads) decode_fp4_merge_kernel(const KParams p) {
  release_dependents();
  wait_for_previous_kernel();
  const int4 seg = __ldcg(p.crossing + blockIdx.x);
  const int r = blockIdx.y * (kMergeThreads / (D / 4)) + threadIdx.x / (D / 4), col = threadIdx.x % (D / 4) * 4;
  if (seg.w < 0 || r >= seg.y) return;
  float m = -INFINITY, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto take = [&](int c, auto some) {                // the results of CTAs c .. c + some - 1
    constexpr int N = decltype(some)::value;
    float lse[N];
    float4 o[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      lse[i] = -INFINITY;
      o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c + i <= seg.z) {
        const size_t at = static_cast<size_t>(c + i == static_cast<int>(blockIdx.x) ? seg.w : 2 * (c + i)) * p.seg_rows + r;
        lse[i] = __ldcg(p.lse_part + at);
        o[i] = __ldcg(reinterpret_cast<const float4*>(p.o_part + at * D + col));
      }
    }
    float m_new = m;
#pragma unroll
    for (int i = 0; i < N; ++i) m_new = fmaxf(m_new, lse[i]);
    const float keep = m == -INFINITY ? 0.f : expf(m - m_new);
    sum *= keep;
    acc = make_float4(acc.x * keep, acc.y * keep, acc.z * keep, acc.w * keep);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float w = lse[i] == -INFINITY ? 0.f : expf(lse[i] - m_new);
      sum += w;
      acc.x = fmaf(w, o[i].x, acc.x);
      acc.y = fmaf(w, o[i].y, acc.y);
      acc.z = fmaf(w, o[i].z, acc.z);
      acc.w = fmaf(w, o[i].w, acc.w);
    }
    m = m_new;
  };
  int c = blockIdx.x;
  for (; seg.z - c >= 4; c += 16) take(c, std::integral_constant<int, 16>());
  if (c <= seg.z) take(c, std::integral_constant<int, 4>());
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const size_t at = static_cast<size_t>(seg.x) + r;
  const uint2 pk = FP16 ? make_uint2(cvt_pack_f16(acc.x * inv, acc.y * inv), cvt_pack_f16(acc.z * inv, acc.w * inv))
                          : make_uint2(cvt_pack_bf16(acc.x * inv, acc.y * inv), cvt_pack_bf16(acc.z * inv, acc.w * inv));
  *reinterpret_cast<uint2*>(p.o + at * D + col) = pk;
  if (col == 0) p.lse[at] = sum == 0.f ? -INFINITY : m + logf(sum);
}

// CTAs of the cluster that takes a segment, or 0: all segments' tiles dealt out in one line.  The
// smaller modelled time, in microseconds, fitted to 4 and 16 rows of d = 128, 1 to 32 sequences of 500 to
// 16384 tokens (8 rows and d = 64 take it as it is): a start and an end, the tiles of one CTA (less with an SM to itself), and for the line
// the joining of a segment's CTAs (of 34 shapes one took 11 % more than the other way, the rest at
// most 4).  One sequence of 4096 tokens, 8 heads: 8.5 by clusters, 12.3 in line; of 16384 14.7 and 15.9;
// 16 of 8192 in line 29.7.  Clusters only as far as all of them run at a time (with one CTA to an SM
// and with two: a multiprocessor group's SMs are not a multiple of every size).
inline int cluster_of(int B, int segs, int tiles, int per_sm) {
  constexpr int at_a_time[2][9] = {{0, 152, 76, 46, 36, 28, 23, 15, 15}, {0, 304, 152, 97, 74, 58, 46, 38, 36}};
  const double n = static_cast<double>(B) * segs, ctas = 152.0 * per_sm, tile = per_sm == 1 ? 0.9 : 0.7;
  int best = 0;
  double least = 8.6 + tile * std::ceil(n * tiles / ctas) + 0.1 * std::min<double>(tiles, ctas / n);
  for (int c = 1; c <= 8; ++c) {
    if (n > at_a_time[per_sm - 1][c]) break;
    const double each = per_sm == 1 ? 0.9 : n * c <= 152 ? 0.52 : 0.8;
    const double t = (per_sm == 1 ? 7.0 : 6.3) + each * ((tiles + c - 1) / c);
    if (t < least) {
      least = t;
      best = c;
    }
  }
  return best;
}

template <int D, int NR, int TQ, int TP, bool FP16, bool SIGNS>
attn_status_t launch_t(const Fp4DecodeParams& a, KParams p, int ctas, cudaStream_t stream) {
  using C = Cfg<D, NR, TQ, TP>;
  p.cluster = cluster_of(p.B, p.segs, (a.max_seqlen - 1) / C::TILE + 1, C::CTAS);
  p.solo = a.max_seqlen <= C::TILE ? 1 : 0;
  if (p.cluster > 0) ctas = p.B * p.segs * p.cluster;
  else if (ctas > 152 * C::CTAS) ctas = 152 * C::CTAS;
  auto kern = decode_fp4_kernel<D, NR, TQ, TP, FP16, SIGNS>;
  attn_status_t s = set_smem(reinterpret_cast<const void*>(kern), C::SMEM);
  if (s != ATTN_OK) return s;
  // {128 codes of one or two tokens, rows of a page, heads, pages}
  CUtensorMap tk, tv;
  const int box = (p.page_size < C::TILE ? p.page_size : C::TILE) / C::KP;
  const uint64_t head_b = static_cast<uint64_t>(p.page_size) * (D / 2);
  if ((s = make_tmap_fp4(&tk, a.k_cache, p.page_size / C::KP, p.H_kv, p.num_pages, 64, head_b, head_b * p.H_kv, box)) != ATTN_OK)
    return s;
  if ((s = make_tmap_fp4(&tv, a.v_cache, p.page_size / C::KP, p.H_kv, p.num_pages, 64, head_b, head_b * p.H_kv, box)) != ATTN_OK)
    return s;
  cudaError_t e = launch_dependent(kern, dim3(ctas), C::THREADS, C::SMEM, stream, p.cluster, tk, tv, p);
  if (e != cudaSuccess) return fail_cuda(e, "4-bit decode kernel launch");
  if (ctas == 1 || p.cluster > 0 || p.solo) return ATTN_OK;            // no segment crosses shares
  constexpr int rows = kMergeThreads / (D / 4);
  e = launch_dependent(decode_fp4_merge_kernel<D, FP16>, dim3(ctas, (p.seg_rows + rows - 1) / rows), kMergeThreads, 0, stream,
                       0, p);
  return e == cudaSuccess ? ATTN_OK : fail_cuda(e, "4-bit decode merge kernel launch");
}

template <int D, int NR>
attn_status_t launch_r(const Fp4DecodeParams& a, const KParams& p, int ctas, cudaStream_t stream) {
  if (a.fp16)
    return p.signs ? launch_t<D, NR, 4, 3, true, true>(a, p, ctas, stream) : launch_t<D, NR, 3, 3, true, false>(a, p, ctas, stream);
  return p.signs ? launch_t<D, NR, 4, 2, false, true>(a, p, ctas, stream) : launch_t<D, NR, 2, 2, false, false>(a, p, ctas, stream);
}

template <int D>
attn_status_t launch_d(const Fp4DecodeParams& a, const KParams& p, int ctas, cudaStream_t stream) {
  return p.rows <= 4 ? launch_r<D, 4>(a, p, ctas, stream) : p.rows <= 8 ? launch_r<D, 8>(a, p, ctas, stream)
                                                                         : launch_r<D, 16>(a, p, ctas, stream);
}

}  // namespace

attn_status_t launch_decode_fp4(const Fp4DecodeParams& p, cudaStream_t stream) {
  int* status = device_status_word();
  if (!status) return fail(ATTN_ERR_CUDA, "status word unavailable");
  const Fp4DecodePlan plan = fp4_decode_plan(p.B, p.H, p.H_kv, p.n_q, p.d, p.max_seqlen);
  const int rows = p.H / p.H_kv * p.n_q;
  const size_t part_rows = 2ull * plan.ctas * plan.seg_rows;
  char* ws = static_cast<char*>(p.workspace);
  char* const lse_part = ws + align_up(part_rows * p.d * sizeof(float), 256);
  char* const crossing = lse_part + align_up(part_rows * sizeof(float), 256);
  const int most = static_cast<int>(std::min(2147483647ll, static_cast<long long>(p.max_pages) * p.page_size));
  const KParams kp{static_cast<const uint16_t*>(p.q), {p.k_descale, p.v_descale}, p.signs,
                   p.block_table, p.seq_lens, static_cast<uint16_t*>(p.o), p.lse, reinterpret_cast<float*>(ws),
                   reinterpret_cast<float*>(lse_part), reinterpret_cast<int4*>(crossing), status, p.B, p.H, p.H_kv, p.n_q,
                   rows, plan.qtiles, p.H_kv * plan.qtiles, plan.seg_rows, p.num_pages, p.page_size,
                   page_shift_of(p.page_size), p.max_pages, p.causal, 0, 0, most, p.scale * 1.4426950408889634f};
  return p.d == 64 ? launch_d<64>(p, kp, plan.ctas, stream) : launch_d<128>(p, kp, plan.ctas, stream);
}

}  // namespace attn
