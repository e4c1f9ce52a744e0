// Decode attention over a paged 4-bit cache (fp4.cuh): n_q new query tokens per sequence,
// grouped-query heads, keys optionally stored transformed.
//
//   S_ij = scale q_i . (k^_j s^k_j),   O_i = sum_j softmax(S)_ij (v^_j s^v_j),
// with k^, v^ the e2m1 values of a row and s^k, s^v its descales.  A step reads d + 4
// bytes per token and head and has to turn them into operands at HBM's rate: per SM some 45
// bytes a nanosecond, 24 codes a clock of each, so what bounds this kernel besides HBM is
// the number of instructions per code.
//
//  * Codes go from shared memory to the registers of mma.sync as float16 (exact) by one
//    conversion per two codes.  No dequantised tile is written to shared memory: as 16-bit
//    operands of tcgen05.mma the tiles would be written and read at four times the bytes of
//    their codes.  The products are small (16 keys x 8 query rows x 16), and take a third of
//    what the legacy tensor path gives.
//  * S^T = K Q^T with the keys on the M side and 8 query rows on N; the order of the d
//    columns within a product is free, so lane t of a group takes the quarter [t d / 4, + d / 4)
//    of its key rows with one load.  O^T += V^T P^T: its operand pairs neighbouring keys, so
//    two rows' conversions are joined by two byte permutes.  P^T comes out of the
//    accumulators of S^T through movmatrix.
//  * Queries are scaled by a power of two to [2^14, 2^15) and held as float16: exact for
//    bfloat16 and float16 queries (up to values 2^-28 below a row's largest).  Transformed
//    ones are held as the sum of two float16 (LO): one would put 2^-12 of each component
//    into the scores, which shows in the log-sum-exps of short sequences.
//  * P is held as float16 of 2^(s + log2 s^v - T + 12), T a running reference of that sum: the
//    value descale is part of the exponent, as in the e4m3 decode, so it is the tokens that
//    count for the result which have float16's eleven bits, however their descales differ.  One
//    whose product is 2^-26 of the largest or less loses bits (an error of 2^-37 of that one).
//    The row sums are float32 sums of 2^(s - M) with a reference of their own, since s^v may
//    be 0.  References move only when a value exceeds T by 3 or M by 64.
//  * Every warp walks alone: its own ring of blocks of 32 keys, filled by bulk copies that it
//    issues itself, its own statistics and accumulators; no barrier in the loop.  A CTA's
//    four warps take the blocks of a part of a segment in turn and join at its end.
//  * A segment is up to 16 query rows of a key/value head with all keys of a sequence.  The
//    128-key tiles of all segments stand in one line, dealt out evenly to the CTAs; segments
//    that cross shares are joined by a second, dependent kernel from float32 partial results
//    (at most two per CTA).
#include <cmath>

#include "common.h"
#include "fp4.cuh"
#include "rope.cuh"

namespace attn {
namespace {

constexpr int W = 4;                    // warps of a CTA
constexpr int kThreads = 32 * W;
constexpr int BK = 32;                  // keys of a block
constexpr float kPShift = 12.f;         // P' is 2^12 at the reference, 2^15 at most

template <int D>
struct Cfg {
  static constexpr int CODES = BK * D / 2;              // of a block's keys or values
  static constexpr int KD = 2 * CODES;                  // key descales, then value descales
  static constexpr int STAGE = 2 * CODES + 4 * BK;
  static constexpr int VPL = D / 4;                     // columns of a lane in S^T
  static constexpr int VB = D / 16;                     // bytes of a lane's value rows in O^T
};
// Ring depth by what fits beside the other CTAs of an SM.
template <int D, int NT>
constexpr int kStages = (NT == 1 ? 3 : 4) * (D == 64 ? 2 : 1);

struct KParams {
  const uint16_t* q;
  const uint8_t* codes[2];
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
  int num_pages, page_size, page_shift, max_pages, causal, fp16;
  float scale_log2;
};

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// D (16 x 8, float32) += A (16 x 16, float16) B (16 x 8, float16)
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// Tokens of a sequence; one out of range counts as none.
__device__ __forceinline__ int tokens_of(const KParams& p, int b) {
  const int n = __ldcg(p.seq_lens + b);
  return n < 0 || n > static_cast<long long>(p.max_pages) * p.page_size ? 0 : n;
}
__device__ __forceinline__ int tiles_of(int len) { return (len + kFp4Tile - 1) / kFp4Tile; }

// First tile of CTA c's share of T tiles (at most T CTAs get one).
__device__ __forceinline__ long long share_start(long long c, int C, long long T) {
  const long long n = T < C ? T : C;
  return c >= n ? T : c * T / n;
}

// A walk over the parts of segments in a share.
struct Cursor {
  int b, y, j;           // sequence, segment of it, first tile
  int len;
  long long left;        // tiles of the share from here on
  __device__ __forceinline__ int tiles() const { return tiles_of(len); }
  __device__ __forceinline__ int part() const {
    const int rest = tiles() - j;
    return left < rest ? static_cast<int>(left) : rest;
  }
  __device__ __forceinline__ void next_part(const KParams& p) {
    left -= part();
    if (left <= 0) return;
    j = 0;
    if (++y == p.segs) {
      y = 0;
      do {
        len = tokens_of(p, ++b);
      } while (len == 0);
    }
  }
};

// The warp's side that fills its ring, ahead of the side that reads it.
template <int D, int S>
struct Feeder {
  using C = Cfg<D>;
  Cursor cur;
  int kbeg, kend, n;       // keys of the current part, next of this warp's blocks in it
  int issued;
  int win, win_next;       // table entries of this warp's next 32 >> split blocks, and of those behind
  uint8_t* ring;
  uint64_t* full;
  int* flags;              // per stage: pieces that were copied
  int warp, lane, split;   // split: 1 where a block lies on two pages (of 16)

  // lane: entry of the window's block base + lane >> split
  __device__ __forceinline__ int window(const KParams& p, int base) const {
    const int key = kbeg + BK * (warp + W * (base + (lane >> split))) + ((lane & split) << 4);
    if (key >= kend) return -1;
    return __ldcg(p.block_table + static_cast<size_t>(cur.b) * p.max_pages + (key >> p.page_shift));
  }
  __device__ __forceinline__ void enter(const KParams& p) {
    kbeg = cur.j * kFp4Tile;
    kend = min((cur.j + cur.part()) * kFp4Tile, cur.len);
    n = 0;
    if (kbeg + BK * warp < kend) {
      win = window(p, 0);
      win_next = window(p, 32 >> split);
    }
  }
  // One more block of this warp into its ring stage, if the share has one.
  __device__ __forceinline__ void issue(const KParams& p) {
    while (cur.left > 0 && kbeg + BK * (warp + W * n) >= kend) {
      cur.next_part(p);
      if (cur.left > 0) enter(p);
    }
    if (cur.left <= 0) return;
    const int key0 = kbeg + BK * (warp + W * n);
    const int stage = issued % S;
    const int piece = lane & split, kind = lane >> split;        // kind: codes and descales of K and V
    const int rows = BK >> split, at = piece * rows;
    const int in_win = n & ((32 >> split) - 1);
    const int phys = __shfl_sync(0xffffffffu, win, (in_win << split) + piece);
    const bool wanted = kind < 4 && key0 + at < kend;
    const bool ok = wanted && phys >= 0 && phys < p.num_pages;
    if (wanted && !ok && kind == 0) atomicCAS(p.status, 0, kDevBadSeqlens);
    const uint32_t copied = __ballot_sync(0xffffffffu, ok) & ((1u << (1 << split)) - 1u);
    uint8_t* const dst = ring + stage * C::STAGE;
    if (lane == 0) {
      flags[stage] = static_cast<int>(copied);
      mbar_arrive_expect_tx(&full[stage], __popc(copied) * rows * (D + 4));
    }
    __syncwarp();
    if (ok) {
      const int hk = cur.y / p.qtiles;
      const size_t row = (static_cast<size_t>(phys) * p.H_kv + hk) * p.page_size + ((key0 + at) & (p.page_size - 1));
      const int kv = kind & 1;
      if (kind < 2) bulk_load(dst + kv * C::CODES + at * (D / 2), p.codes[kv] + row * (D / 2), rows * (D / 2), &full[stage]);
      else bulk_load(dst + C::KD + 2 * BK * kv + 2 * at, p.descale[kv] + row, 2 * rows, &full[stage]);
    }
    ++issued;
    ++n;
    if ((n & ((32 >> split) - 1)) == 0) {
      win = win_next;
      win_next = window(p, n + (32 >> split));
    }
  }
};

// Key of row r (0 .. 7) of an 8-row half of a product's M side: with this order the four
// value rows that the lanes of a group read at a time, and the key rows of neighbouring
// groups, lie in different banks as far as rows of 64 bytes allow (of 32 bytes: wholly).
__device__ __forceinline__ int key_row(int r) { return r < 4 ? r : r ^ 1; }

template <int D, int NT, bool LO>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 4 : 3)
    decode_fp4_kernel(const KParams p) {
  using C = Cfg<D>;
  constexpr int S = kStages<D, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full[W][S];
  __shared__ int flags[W][S];
  __shared__ float stat_t[W][16], stat_m[W][16], stat_l[W][16];
  __shared__ int buf_sh[W];
  __shared__ long long warp_sum[W], start_sh[2];      // prefix sums; first batch entry and tile in its line
  __shared__ __align__(16) float signs[LO ? D : 4];
  __shared__ int abort_sh;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane >> 2, t = lane & 3;
  if (threadIdx.x == 0) {
    for (int w = 0; w < W; ++w)
      for (int s = 0; s < S; ++s) mbar_init(&full[w][s], 1);
    abort_sh = 0;
    fence_mbar_init();
  }
  wait_for_previous_kernel();
  release_dependents();
  const Abort ab{&abort_sh, p.status};
  if (LO && threadIdx.x < D / 4)
    *reinterpret_cast<float4*>(signs + 4 * threadIdx.x) = __ldcg(reinterpret_cast<const float4*>(p.signs) + threadIdx.x);

  // ---- tiles of one segment of the entries before each; this CTA's share
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = min(static_cast<int>(threadIdx.x) * per, p.B), b1 = min(b0 + per, p.B);
  long long sum = 0;
  for (int b = b0; b < b1; ++b) {
    const int len = tokens_of(p, b);
    if (len == 0 && blockIdx.x == 0 && __ldcg(p.seq_lens + b) != 0) atomicCAS(p.status, 0, kDevBadSeqlens);
    sum += tiles_of(len);
  }
  long long scan = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += x;
  }
  if (lane == 31) warp_sum[warp] = scan;
  __syncthreads();
  long long base = scan - sum, all = 0;
  for (int w = 0; w < W; ++w) {
    if (w < warp) base += warp_sum[w];
    all += warp_sum[w];
  }
  const long long T = all * p.segs;
  const long long g0 = share_start(blockIdx.x, gridDim.x, T);
  const long long total = share_start(blockIdx.x + 1ll, gridDim.x, T) - g0;
  if (total > 0 && base * p.segs <= g0 && g0 < (base + sum) * p.segs) {
    int b = b0;
    while (true) {
      const int n = tiles_of(tokens_of(p, b));
      if (g0 < (base + n) * p.segs) break;
      base += n;
      ++b;
    }
    start_sh[0] = b;
    start_sh[1] = g0 - base * p.segs;
  }
  __syncthreads();

  // batch entries without tokens: O = 0, LSE = -inf
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (tokens_of(p, b) != 0) continue;
    const size_t rows_b = static_cast<size_t>(p.H) * p.n_q;
    uint4* dst = reinterpret_cast<uint4*>(p.o + b * rows_b * D);
    for (size_t i = threadIdx.x; i < rows_b * (D / 8); i += kThreads) dst[i] = make_uint4(0u, 0u, 0u, 0u);
    for (size_t i = threadIdx.x; i < rows_b; i += kThreads) p.lse[b * rows_b + i] = -INFINITY;
  }
  int4 crossing = make_int4(0, 0, 0, -1);
  if (total == 0) {
    if (threadIdx.x == 0) p.crossing[blockIdx.x] = crossing;
    return;
  }

  Cursor cur;
  cur.b = static_cast<int>(start_sh[0]);
  cur.len = tokens_of(p, cur.b);
  cur.left = total;
  {
    const int n = cur.tiles();
    cur.y = static_cast<int>(start_sh[1] / n);
    cur.j = static_cast<int>(start_sh[1] - static_cast<long long>(cur.y) * n);
  }
  uint8_t* const ring = smem + warp * S * C::STAGE;
  Feeder<D, S> feed;
  feed.cur = cur;
  feed.issued = 0;
  feed.ring = ring;
  feed.full = full[warp];
  feed.flags = flags[warp];
  feed.warp = warp;
  feed.lane = lane;
  feed.split = p.page_size < BK ? 1 : 0;
  feed.enter(p);
#pragma unroll 1
  for (int i = 0; i < S; ++i) feed.issue(p);

  int used = 0;                 // blocks that this warp has read
  bool ok = true;
  bool first_part = true;
  long long at_tile = g0;
  while (cur.left > 0) {
    const int take = cur.part(), nt_tiles = cur.tiles(), len = cur.len;
    const int kbeg = cur.j * kFp4Tile, kend = min((cur.j + take) * kFp4Tile, len);
    const int hk = cur.y / p.qtiles, row0 = (cur.y - hk * p.qtiles) * 16;
    // rows of a key/value head are contiguous in [B, H, n_q]
    const size_t at0 = (static_cast<size_t>(cur.b) * p.H_kv + hk) * p.rows + row0;
    const int rows_here = min(16, p.rows - row0);

    // ---- query rows as operands: lane (g, t) of tile x the columns [t VPL, + VPL) of row 8 x + g
    uint32_t qh[NT][D / 16][2], ql[LO ? NT : 1][LO ? D / 16 : 1][2];
    float cq[NT][2];             // score coefficient of the lane's two query columns
    int vend[NT][2];             // keys [0, vend) visible to them
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      float v[C::VPL];
      const int r = 8 * x + g;
      const uint4* src = reinterpret_cast<const uint4*>(p.q + (at0 + (r < rows_here ? r : 0)) * D + t * C::VPL);
#pragma unroll
      for (int i = 0; i < C::VPL / 8; ++i) {
        const uint4 w = __ldcg(src + i);
        float f[8];
        if (p.fp16) unpack16<true>(w, f);
        else unpack16<false>(w, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[8 * i + e] = r < rows_here ? f[e] : 0.f;
      }
      if constexpr (LO) {
#pragma unroll
        for (int i = 0; i < C::VPL; i += 4) {
          const float4 s = *reinterpret_cast<const float4*>(signs + t * C::VPL + i);
          v[i] *= s.x, v[i + 1] *= s.y, v[i + 2] *= s.z, v[i + 3] *= s.w;
        }
#pragma unroll
        for (int h = 1; h < C::VPL; h <<= 1)
#pragma unroll
          for (int i = 0; i < C::VPL; ++i)
            if ((i & h) == 0) {
              const float a = v[i], b = v[i + h];
              v[i] = a + b;
              v[i + h] = a - b;
            }
#pragma unroll
        for (int m = 1; m < 4; m <<= 1) {
          const float sgn = (t & m) ? -1.f : 1.f;
#pragma unroll
          for (int i = 0; i < C::VPL; ++i) v[i] = fmaf(sgn, v[i], __shfl_xor_sync(0xffffffffu, v[i], m));
        }
        const float isd = D == 128 ? 0.08838834764831845f : 0.125f;
#pragma unroll
        for (int i = 0; i < C::VPL; ++i) v[i] *= isd;
      }
      uint32_t top = 0u;
#pragma unroll
      for (int i = 0; i < C::VPL; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // times 2^(14 - floor(log2 top)): an infinity stays one
      const int e = static_cast<int>(top >> 23);
      const int up = top == 0u ? 127 : min(268 - e, 254);
      const float f = __uint_as_float(static_cast<uint32_t>(up) << 23);
      const float back = __uint_as_float(static_cast<uint32_t>(max(254 - up, 1)) << 23);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float a = v[4 * kk + 2 * i] * f, b = v[4 * kk + 2 * i + 1] * f;
          const uint32_t h = cvt_pack_f16(a, b);
          qh[x][kk][i] = h;
          if constexpr (LO) {
            const float2 hf = __half22float2(*reinterpret_cast<const __half2*>(&h));
            ql[x][kk][i] = cvt_pack_f16(a - hf.x, b - hf.y);
          }
        }
      const float c_row = p.scale_log2 * back;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        cq[x][i] = __shfl_sync(0xffffffffu, c_row, (2 * t + i) * 4);
        const int rr = 8 * x + 2 * t + i, tq = (row0 + rr) % p.n_q;
        vend[x][i] = rr < rows_here ? (p.causal ? min(len, len - p.n_q + tq + 1) : len) : 0;
      }
    }

    float o[C::VB][NT][4];
    float tref[NT][2], mref[NT][2], lsum[NT][2];
#pragma unroll
    for (int x = 0; x < NT; ++x) {
#pragma unroll
      for (int i = 0; i < C::VB; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][x][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) tref[x][e] = mref[x][e] = -INFINITY, lsum[x][e] = 0.f;
    }

    bool owed = false;            // the last block's stage is refilled after the part's end
    for (int key0 = kbeg + BK * warp; key0 < kend; key0 += BK * W) {
      if (owed && ok) {
        __syncwarp();
        feed.issue(p);
      }
      const int stage = used % S;
      if (__any_sync(0xffffffffu, !mbar_wait(&full[warp][stage], (used / S) & 1, ab, kDevTimeoutLoad))) ok = false;
      ++used;
      owed = true;
      if (!ok) continue;
      const uint8_t* blk = ring + stage * C::STAGE;
      const int got = flags[warp][stage];
      // ---- S^T of the block's two halves of 16 keys
      float acc[2][NT][4];
#pragma unroll
      for (int mb = 0; mb < 2; ++mb) {
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[mb][x][e] = 0.f;
        const uint8_t* ra = blk + (16 * mb + key_row(g)) * (D / 2) + t * (C::VPL / 2);
        uint32_t wa[C::VPL / 8], wb[C::VPL / 8];
        if constexpr (D == 128) {
          const uint4 a = *reinterpret_cast<const uint4*>(ra), b = *reinterpret_cast<const uint4*>(ra + 8 * (D / 2));
          wa[0] = a.x, wa[1] = a.y, wa[2] = a.z, wa[3] = a.w;
          wb[0] = b.x, wb[1] = b.y, wb[2] = b.z, wb[3] = b.w;
        } else {
          const uint2 a = *reinterpret_cast<const uint2*>(ra), b = *reinterpret_cast<const uint2*>(ra + 8 * (D / 2));
          wa[0] = a.x, wa[1] = a.y;
          wb[0] = b.x, wb[1] = b.y;
        }
#pragma unroll
        for (int i = 0; i < C::VPL / 8; ++i) {
          uint32_t ha[4], hb[4];
          e2m1_halves(wa[i], ha);
          e2m1_halves(wb[i], hb);
#pragma unroll
          for (int k2 = 0; k2 < 2; ++k2)
#pragma unroll
            for (int x = 0; x < NT; ++x) {
              const int kk = 2 * i + k2;
              mma_16816(acc[mb][x], ha[2 * k2], hb[2 * k2], ha[2 * k2 + 1], hb[2 * k2 + 1], qh[x][kk][0], qh[x][kk][1]);
              if constexpr (LO)
                mma_16816(acc[mb][x], ha[2 * k2], hb[2 * k2], ha[2 * k2 + 1], hb[2 * k2 + 1], ql[x][kk][0],
                          ql[x][kk][1]);
            }
        }
      }
      // ---- scores in log2 units, and with the value descale's logarithm
      float y[2][NT][4];
      const uint16_t* sd = reinterpret_cast<const uint16_t*>(blk + C::KD);
      bool need = false;
#pragma unroll
      for (int mb = 0; mb < 2; ++mb)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int kr = 16 * mb + 8 * r + key_row(g);
          const float ks = bf16_bits(sd[kr]), lv = lg2(bf16_bits(sd[BK + kr]));
          const bool there = feed.split ? (got >> mb) & 1 : got != 0;
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const bool seen = there && key0 + kr < vend[x][e];
              const float s = seen ? acc[mb][x][2 * r + e] * (cq[x][e] * ks) : -INFINITY;
              acc[mb][x][2 * r + e] = s;
              y[mb][x][2 * r + e] = seen ? s + lv : -INFINITY;
              need |= y[mb][x][2 * r + e] > tref[x][e] + 3.f || s > mref[x][e] + 64.f;
            }
        }
      if (__any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float ty = fmaxf(fmaxf(y[0][x][e], y[0][x][2 + e]), fmaxf(y[1][x][e], y[1][x][2 + e]));
            float ms = fmaxf(fmaxf(acc[0][x][e], acc[0][x][2 + e]), fmaxf(acc[1][x][e], acc[1][x][2 + e]));
#pragma unroll
            for (int m = 4; m < 32; m <<= 1) {
              ty = fmaxf(ty, __shfl_xor_sync(0xffffffffu, ty, m));
              ms = fmaxf(ms, __shfl_xor_sync(0xffffffffu, ms, m));
            }
            ty = fmaxf(ty, tref[x][e]);
            ms = fmaxf(ms, mref[x][e]);
            const float at = tref[x][e] == -INFINITY ? 0.f : ex2_approx(tref[x][e] - ty);
            const float am = mref[x][e] == -INFINITY ? 0.f : ex2_approx(mref[x][e] - ms);
            tref[x][e] = ty;
            mref[x][e] = ms;
            lsum[x][e] *= am;
#pragma unroll
            for (int i = 0; i < C::VB; ++i) {
              o[i][x][e] *= at;
              o[i][x][2 + e] *= at;
            }
          }
      }
      // ---- probabilities, transposed into operands
      uint32_t pb[2][NT][2];
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        float tr[2], mr[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          tr[e] = kPShift - (tref[x][e] == -INFINITY ? 0.f : tref[x][e]);
          mr[e] = mref[x][e] == -INFINITY ? 0.f : mref[x][e];
        }
#pragma unroll
        for (int mb = 0; mb < 2; ++mb) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            lsum[x][0] += ex2_approx(acc[mb][x][2 * r] - mr[0]);
            lsum[x][1] += ex2_approx(acc[mb][x][2 * r + 1] - mr[1]);
            pb[mb][x][r] = transpose8x8(
                cvt_pack_f16(ex2_approx(y[mb][x][2 * r] + tr[0]), ex2_approx(y[mb][x][2 * r + 1] + tr[1])));
          }
        }
      }
      // ---- O^T += V^T P^T
#pragma unroll
      for (int mb = 0; mb < 2; ++mb) {
        const uint8_t* rv = blk + C::CODES + 16 * mb * (D / 2) + g * C::VB;
        const int r0 = key_row(2 * t) * (D / 2), r1 = key_row(2 * t + 1) * (D / 2);
        uint32_t w[4][C::VB / 4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint8_t* src = rv + (r & 1 ? r1 : r0) + (r >> 1) * 8 * (D / 2);
          if constexpr (D == 128) {
            const uint2 a = *reinterpret_cast<const uint2*>(src);
            w[r][0] = a.x, w[r][1] = a.y;
          } else {
            w[r][0] = *reinterpret_cast<const uint32_t*>(src);
          }
        }
#pragma unroll
        for (int i = 0; i < C::VB / 4; ++i) {
          uint32_t h[4][4];
#pragma unroll
          for (int r = 0; r < 4; ++r) e2m1_halves(w[r][i], h[r]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t a0 = __byte_perm(h[0][e], h[1][e], 0x5410), a1 = __byte_perm(h[0][e], h[1][e], 0x7632);
            const uint32_t a2 = __byte_perm(h[2][e], h[3][e], 0x5410), a3 = __byte_perm(h[2][e], h[3][e], 0x7632);
#pragma unroll
            for (int x = 0; x < NT; ++x) mma_16816(o[4 * i + e][x], a0, a1, a2, a3, pb[mb][x][0], pb[mb][x][1]);
          }
        }
      }
    }

    // ---- the part's end: the warps' results joined.  Each leaves its output in the stage it
    // read last, 8 rows at a time, 16-byte pieces exchanged within a row so that the four
    // lanes of a group write to different banks.
    const int nw = min(W, (kend - kbeg + BK - 1) / BK);          // warps that had a block
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int m = 4; m < 32; m <<= 1) lsum[x][e] += __shfl_xor_sync(0xffffffffu, lsum[x][e], m);
        if (g == 0) {
          const int r = 8 * x + 2 * t + e;
          stat_t[warp][r] = tref[x][e];
          stat_m[warp][r] = mref[x][e];
          stat_l[warp][r] = lsum[x][e];
        }
      }
    if (lane == 0) buf_sh[warp] = (used + S - 1) % S;
    const bool whole = take == nt_tiles;
    const size_t slot = 2ull * blockIdx.x + (first_part ? 0 : 1);
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      __syncthreads();                        // statistics are there; the round before has been read
      if (warp < nw) {
        float4* dst = reinterpret_cast<float4*>(ring + ((used + S - 1) % S) * C::STAGE);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 2 * t + e;
          float top = -INFINITY;
          for (int w = 0; w < nw; ++w) top = fmaxf(top, stat_t[w][8 * x + r]);
          const float f = tref[x][e] == -INFINITY ? 0.f : ex2_approx(tref[x][e] - top);
#pragma unroll
          for (int i = 0; i < C::VB / 2; ++i) {
            const float4 val = make_float4(o[2 * i][x][e] * f, o[2 * i][x][2 + e] * f, o[2 * i + 1][x][e] * f,
                                           o[2 * i + 1][x][2 + e] * f);
            dst[r * (D / 4) + ((g * (C::VB / 2) + i) ^ t)] = val;
          }
        }
      }
      __syncthreads();
      const int real = min(8, rows_here - 8 * x);
      for (int it = threadIdx.x; it < real * (D / 4); it += kThreads) {
        const int r = it / (D / 4), c4 = it % (D / 4);
        float top_t = -INFINITY, top_m = -INFINITY, l = 0.f;
        for (int w = 0; w < nw; ++w) {
          top_t = fmaxf(top_t, stat_t[w][8 * x + r]);
          top_m = fmaxf(top_m, stat_m[w][8 * x + r]);
        }
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < nw; ++w) {
          const float m = stat_m[w][8 * x + r];
          if (m != -INFINITY) l += stat_l[w][8 * x + r] * ex2_approx(m - top_m);
          const float4 v = *(reinterpret_cast<const float4*>(smem + w * S * C::STAGE + buf_sh[w] * C::STAGE) +
                             r * (D / 4) + (c4 ^ (r >> 1)));
          a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
        }
        // (a NaN among the scores or descales is in a by now, and stays)
        const float f = l == 0.f || top_t == -INFINITY ? 0.f : ex2_approx(top_t - top_m - kPShift) / l;
        a.x *= f, a.y *= f, a.z *= f, a.w *= f;
        const float lse = l == 0.f ? -INFINITY : (top_m + lg2(l)) * 0.69314718055994530942f;
        if (whole) {
          const uint2 pk = p.fp16 ? make_uint2(cvt_pack_f16(a.x, a.y), cvt_pack_f16(a.z, a.w))
                                  : make_uint2(cvt_pack_bf16(a.x, a.y), cvt_pack_bf16(a.z, a.w));
          *reinterpret_cast<uint2*>(p.o + (at0 + 8 * x + r) * D + 4 * c4) = pk;
          if (c4 == 0) p.lse[at0 + 8 * x + r] = lse;
        } else {
          const size_t pr = slot * p.seg_rows + 8 * x + r;
          *reinterpret_cast<float4*>(p.o_part + pr * D + 4 * c4) = a;
          if (c4 == 0) p.lse_part[pr] = lse;
        }
      }
    }
    if (!whole && cur.j == 0) {
      // CTA whose share holds the segment's last tile: the last c with c T / n <= it
      const long long n = T < gridDim.x ? T : gridDim.x, last = at_tile + nt_tiles - 1;
      crossing = make_int4(static_cast<int>(at0), rows_here, static_cast<int>(((last + 1) * n - 1) / T),
                           static_cast<int>(slot));
    }
    fence_proxy_async_smem();                 // before copies land in the stages again
    __syncthreads();
    if (owed && ok) feed.issue(p);
    first_part = false;
    at_tile += take;
    cur.next_part(p);
  }
  if (threadIdx.x == 0) p.crossing[blockIdx.x] = crossing;
  if (!ok)       // let the copies in flight land before the memory goes away
    for (int i = max(0, feed.issued - S); i < feed.issued; ++i) mbar_wait_drain(&full[warp][i % S], (i / S) & 1);
}

// Segments that cross shares: LSE = log sum_c exp(lse_c), O = sum_c exp(lse_c - LSE) O_c over
// CTAs c0 .. c1, whose partial results are c0's slot and the others' first ones.  A block for
// every CTA that left a segment unfinished (4 rows of it), D / 4 threads per row.
constexpr int kMergeThreads = 128;
template <int D>
__global__ void __launch_bounds__(kMergeThreads) decode_fp4_merge_kernel(const KParams p) {
  wait_for_previous_kernel();
  const int4 seg = __ldcg(p.crossing + blockIdx.x);
  const int r = blockIdx.y * (kMergeThreads / (D / 4)) + threadIdx.x / (D / 4), col = threadIdx.x % (D / 4) * 4;
  if (seg.w < 0 || r >= seg.y) return;
  float m = -INFINITY, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = blockIdx.x; c <= seg.z; c += 4) {
    float lse[4];
    float4 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lse[i] = -INFINITY;
      o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c + i <= seg.z) {
        const size_t at = static_cast<size_t>(c + i == static_cast<int>(blockIdx.x) ? seg.w : 2 * (c + i)) * p.seg_rows + r;
        lse[i] = __ldcg(p.lse_part + at);
        o[i] = __ldcg(reinterpret_cast<const float4*>(p.o_part + at * D + col));
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
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const size_t at = static_cast<size_t>(seg.x) + r;
  const uint2 pk = p.fp16 ? make_uint2(cvt_pack_f16(acc.x * inv, acc.y * inv), cvt_pack_f16(acc.z * inv, acc.w * inv))
                          : make_uint2(cvt_pack_bf16(acc.x * inv, acc.y * inv), cvt_pack_bf16(acc.z * inv, acc.w * inv));
  *reinterpret_cast<uint2*>(p.o + at * D + col) = pk;
  if (col == 0) p.lse[at] = sum == 0.f ? -INFINITY : m + logf(sum);
}

template <int D, int NT, bool LO>
attn_status_t launch_t(const KParams& p, int ctas, cudaStream_t stream) {
  constexpr int smem = W * kStages<D, NT> * Cfg<D>::STAGE;
  static_assert(Cfg<D>::STAGE >= 8 * D * 4, "a stage holds the output of 8 rows");
  auto kern = decode_fp4_kernel<D, NT, LO>;
  const attn_status_t s = set_smem(reinterpret_cast<const void*>(kern), smem);
  if (s != ATTN_OK) return s;
  cudaError_t e = launch_dependent(kern, dim3(ctas), kThreads, smem, stream, 0, p);
  if (e != cudaSuccess) return fail_cuda(e, "4-bit decode kernel launch");
  if (ctas == 1) return ATTN_OK;
  constexpr int rows = kMergeThreads / (D / 4);
  e = launch_dependent(decode_fp4_merge_kernel<D>, dim3(ctas, (p.seg_rows + rows - 1) / rows), kMergeThreads, 0, stream,
                       0, p);
  return e == cudaSuccess ? ATTN_OK : fail_cuda(e, "4-bit decode merge kernel launch");
}

template <int D>
attn_status_t launch_d(const KParams& p, int ctas, cudaStream_t stream) {
  if (p.rows <= 8) return p.signs ? launch_t<D, 1, true>(p, ctas, stream) : launch_t<D, 1, false>(p, ctas, stream);
  return p.signs ? launch_t<D, 2, true>(p, ctas, stream) : launch_t<D, 2, false>(p, ctas, stream);
}

}  // namespace

attn_status_t launch_decode_fp4(const Fp4DecodeParams& p, cudaStream_t stream) {
  int* status = device_status_word();
  if (!status) return fail(ATTN_ERR_CUDA, "status word unavailable");
  const Fp4DecodePlan plan = fp4_decode_plan(p.B, p.H, p.H_kv, p.n_q, p.max_seqlen);
  const int rows = p.H / p.H_kv * p.n_q;
  const size_t part_rows = 2ull * plan.ctas * plan.seg_rows;
  char* ws = static_cast<char*>(p.workspace);
  char* const lse_part = ws + align_up(part_rows * p.d * sizeof(float), 256);
  char* const crossing = lse_part + align_up(part_rows * sizeof(float), 256);
  const KParams kp{static_cast<const uint16_t*>(p.q), {p.k_cache, p.v_cache}, {p.k_descale, p.v_descale}, p.signs,
                   p.block_table, p.seq_lens, static_cast<uint16_t*>(p.o), p.lse, reinterpret_cast<float*>(ws),
                   reinterpret_cast<float*>(lse_part), reinterpret_cast<int4*>(crossing), status, p.B, p.H, p.H_kv, p.n_q,
                   rows, plan.qtiles, p.H_kv * plan.qtiles, plan.seg_rows, p.num_pages, p.page_size,
                   page_shift_of(p.page_size), p.max_pages, p.causal, p.fp16, p.scale * 1.4426950408889634f};
  return p.d == 64 ? launch_d<64>(kp, plan.ctas, stream) : launch_d<128>(kp, plan.ctas, stream);
}

}  // namespace attn
