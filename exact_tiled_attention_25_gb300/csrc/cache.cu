// Upkeep of a paged key/value cache: block tables and slot maps built from
// request lengths, and new keys and values written to the cache, in 16 bits or
// as e4m3 codes with one scale per (page, key/value head).  "FlashAttention 3
// Hardware Acceleration: Hopper GPU Strategies for Long-Context Enterprise
// Inference Optimization", section "Memory Fragmentation", describes the cache
// in fixed-size blocks; the paged decode (decode.cu) reads what these write.
#include <cmath>

#include "common.h"
#include "fp8_row.cuh"
#include "rope.cuh"

namespace attn {
namespace {

// ============================================================ block tables ====
constexpr int kTabThreads = 512;
constexpr int kTabMaxB = 16384;   // 12 bytes of shared memory per request

// Exclusive prefix sums of new tokens and new pages over all requests, in every
// block (the requests' lengths are a few KB of L2 hits, cheaper than a second
// launch), then this block's share of the outputs.  Request b has old_lens[b]
// tokens in ceil(old / page_size) pages; its new pages take consecutive entries
// of the free list, requests in order.  New table entries are taken from the
// free list directly, so no block reads what another writes.
// Bound: latency -- a launch, the lengths, the scan's barriers, and per token a binary
// search in shared memory, a table entry and the stores.
// A dependent launch: it reads past the L1 cache.
__global__ void __launch_bounds__(kTabThreads)
    block_tables_kernel(const TablesParams p, int* status, int page_shift) {
  extern __shared__ int tab_sh[];
  int* cu = tab_sh;                  // [B + 1] first new token of each request
  int* pg = cu + p.B + 1;            // [B + 1] first free-list entry of each request
  int* old_sh = pg + p.B + 1;        // [B] tokens in the cache
  __shared__ long long warp_sum[2][kTabThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int page = p.page_size;
  const long long room = static_cast<long long>(p.max_pages) * page;
  auto pages_of = [&](long long n) { return static_cast<int>((n + page - 1) >> page_shift); };
  bool bad = false;
  wait_for_previous_kernel();
#pragma unroll 4
  for (int b = threadIdx.x; b < p.B; b += kTabThreads) {
    int old = __ldcg(p.old_lens + b), add = __ldcg(p.new_lens + b);
    if (old < 0 || old > room || add < 0 || old + static_cast<long long>(add) > room) {
      bad = true;
      old = old < 0 || old > room ? 0 : old;
      add = 0;
    }
    old_sh[b] = old;
    cu[b] = add;
    pg[b] = pages_of(old + static_cast<long long>(add)) - pages_of(old);
  }
  __syncthreads();
  // each thread's own requests, one after the other, then those of the threads before
  const int per = (p.B + kTabThreads - 1) / kTabThreads;
  const int b0 = min(static_cast<int>(threadIdx.x) * per, p.B), b1 = min(b0 + per, p.B);
  long long tok = 0, pages = 0;
  for (int b = b0; b < b1; ++b) {
    tok += cu[b];
    pages += pg[b];
  }
  long long ts = tok, ps = pages;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, ts, o), q = __shfl_up_sync(0xffffffffu, ps, o);
    if (lane >= o) {
      ts += t;
      ps += q;
    }
  }
  if (lane == 31) {
    warp_sum[0][warp] = ts;
    warp_sum[1][warp] = ps;
  }
  __syncthreads();
  long long tok_all = 0, pages_sum = 0;
  ts -= tok;
  ps -= pages;
#pragma unroll
  for (int w = 0; w < kTabThreads / 32; ++w) {
    const long long t = warp_sum[0][w], q = warp_sum[1][w];
    if (w < warp) {
      ts += t;
      ps += q;
    }
    tok_all += t;
    pages_sum += q;
  }
  auto clamp = [](long long x) { return static_cast<int>(x < 2147483647LL ? x : 2147483647LL); };
  for (int b = b0; b < b1; ++b) {
    const int add = cu[b], need = pg[b];
    if (blockIdx.x == 0) p.seq_lens[b] = old_sh[b] + add;
    cu[b] = clamp(ts);
    pg[b] = clamp(ps);
    ts += add;
    ps += need;
  }
  const int total = clamp(tok_all), pages_all = clamp(pages_sum);
  if (threadIdx.x == 0) {
    cu[p.B] = total;
    pg[p.B] = pages_all;
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b <= p.B; b += kTabThreads) p.cu_seqlens[b] = cu[b];
    if (threadIdx.x == 0) p.used[0] = min(pages_all, p.n_free);
    if (bad || (threadIdx.x == 0 && (tok_all > p.capacity || pages_sum > p.n_free)))
      atomicCAS(status, 0, kDevBadTables);
  }
  // request that owns index x of a list whose request b starts at first[b]: the
  // last b with first[b] <= x (requests without entries are passed over)
  auto owner = [&](const int* first, int x) {
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= x) lo = mid;
      else hi = mid;
    }
    return lo;
  };
  const int step = gridDim.x * kTabThreads;
  const int me = blockIdx.x * kTabThreads + threadIdx.x;
  bool lost = false;                 // a new token whose page the table or the free list lacks
  for (long long t = me; t < p.capacity; t += step) {
    long long slot = -1;
    int pos = -1;
    if (t < total) {
      const int b = owner(cu, static_cast<int>(t));
      const int old = old_sh[b];
      pos = old + (static_cast<int>(t) - cu[b]);
      const int lp = pos >> page_shift;
      const int have = pages_of(old);
      int phys;
      if (lp < have) {
        phys = __ldcg(p.block_table + static_cast<size_t>(b) * p.max_pages + lp);
      } else {
        const long long e = static_cast<long long>(pg[b]) + (lp - have);
        phys = e < p.n_free ? __ldcg(p.free_pages + e) : -1;
      }
      if (phys >= 0) slot = static_cast<long long>(phys) * page + (pos & (page - 1));
      else lost = true;
    }
    p.slots[t] = slot;
    p.positions[t] = pos;
  }
  if (lost) atomicCAS(status, 0, kDevBadTables);
  for (long long e = me; e < pages_all; e += step) {
    const int b = owner(pg, static_cast<int>(e));
    p.block_table[static_cast<size_t>(b) * p.max_pages + pages_of(old_sh[b]) + (e - pg[b])] =
        e < p.n_free ? __ldcg(p.free_pages + e) : -1;
  }
}

// ========================================================== e4m3 append ====
// For every page that receives tokens and every plane of it (a key/value head,
// keys or values), the page's new rows are rotated and transformed (keys); their
// amax gives
//   descale' = max(descale, amax / 448)       (a page whose first token is among
//                                              the new ones starts from 0; at least
//                                              2^-90, and 1 where all is 0),
// codes = e4m3_rn_satfinite(x / descale'); when the descale grows, the codes of
// the page's older tokens become e4m3_rn(code * (descale / descale')); the
// unused rest of a page that starts here is cleared, so the decode never meets
// another request's codes or a NaN there.  One owner per page and plane: no
// atomics, and no order on which the result could depend.
//
// Eight lanes hold a row: lane u the columns 8u .. 8u + 7 and 64 + 8u .. 64 + 8u +
// 7 (two 16-byte loads), so a full-width rotation pairs values of one lane and
// only three of the transform's seven stages cross lanes (12 shuffles a row; a
// warp per row takes 24).  Stages run in the pre-pass's order: same bits.
constexpr int kF8Threads = 64;     // of the few-rows variant
constexpr int kF8MaxThreads = 512;

template <bool FP16>
__device__ __forceinline__ void widen16(const uint4& a, const uint4& b, float (&x)[16]) {
  float lo[8], hi[8];
  unpack16<FP16>(a, lo);
  unpack16<FP16>(b, hi);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = lo[i];
    x[8 + i] = hi[i];
  }
}

// Eight table values from column i of a row's table entries.
__device__ __forceinline__ void load8(const float* t, size_t at, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(t + at));
  const float4 b = __ldg(reinterpret_cast<const float4*>(t + at) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// What happens to a key row before it is quantised, fixed per kernel.
enum : int {
  kPlain = 0,          // not rotated
  kHalves = 1,         // all 128 columns, column c with c + 64
  kHalvesPart = 2,     // the first rot < 128 columns, column c with c + rot / 2
  kNeighbours = 3,     // the first rot columns, column 2 c with 2 c + 1
};

// A key row held by eight lanes: rotated by the tables' row `pos`, then (SIGNS)
// transformed by M = diag(signs) H_128 / sqrt(128), the signs in shared memory.
// Every lane of the warp takes part.
template <int MODE, bool SIGNS>
__device__ __forceinline__ void key_row(float (&x)[16], const AppendFp8Params& p, int pos, int u,
                                        const float* signs) {
  if constexpr (MODE != kPlain) {
    const bool inside = pos < p.max_pos;
    const size_t row = static_cast<size_t>(inside ? pos : 0) * (MODE == kHalves ? 64 : p.rot / 2);
    if constexpr (MODE == kNeighbours) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int col = 64 * w + 8 * u;
        if (!inside || col >= p.rot) continue;
        const float4 c = __ldg(reinterpret_cast<const float4*>(p.cos + row + col / 2));
        const float4 s = __ldg(reinterpret_cast<const float4*>(p.sin + row + col / 2));
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a = x[8 * w + 2 * e], b = x[8 * w + 2 * e + 1];
          x[8 * w + 2 * e] = fmaf(-b, ss[e], a * cc[e]);
          x[8 * w + 2 * e + 1] = fmaf(a, ss[e], b * cc[e]);
        }
      }
    } else if constexpr (MODE == kHalves) {
      // both columns of a pair are in this lane
      float c[8], s[8];
      load8(p.cos, row + 8 * u, c);
      load8(p.sin, row + 8 * u, s);
      if (inside) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float a = x[e], b = x[8 + e];
          x[e] = fmaf(-b, s[e], a * c[e]);
          x[8 + e] = fmaf(a, s[e], b * c[e]);
        }
      }
    } else {
      // vector j (columns 8j .. 8j + 7) pairs with vector j +- rot / 16
      const int nv = p.rot / 16;
      float other[16];
      bool turn[2], lower[2];
      int at[2];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int j = u + 8 * w;
        turn[w] = j < 2 * nv;
        lower[w] = j < nv;
        at[w] = lower[w] ? j : j - nv;               // vector of the table row
        const int pj = turn[w] ? (lower[w] ? j + nv : j - nv) : j;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float a = __shfl_sync(0xffffffffu, x[e], pj & 7, 8);
          const float b = __shfl_sync(0xffffffffu, x[8 + e], pj & 7, 8);
          other[8 * w + e] = pj < 8 ? a : b;
        }
      }
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        if (!turn[w] || !inside) continue;
        float c[8], s[8];
        load8(p.cos, row + 8 * at[w], c);
        load8(p.sin, row + 8 * at[w], s);
        const float sg = lower[w] ? -1.f : 1.f;      // x c - y s, and y c + x s
#pragma unroll
        for (int e = 0; e < 8; ++e)
          x[8 * w + e] = fmaf(sg * other[8 * w + e], s[e], x[8 * w + e] * c[e]);
      }
    }
  }
  if constexpr (SIGNS) {
    uint64_t y[8];                                   // pairs of neighbouring columns
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 sg = *reinterpret_cast<const float4*>(signs + (i < 2 ? 8 * u + 4 * i : 64 + 8 * u + 4 * (i - 2)));
      const uint64_t a = fmul2(pack2(x[4 * i], x[4 * i + 1]), pack2(sg.x, sg.y));
      const uint64_t c = fmul2(pack2(x[4 * i + 2], x[4 * i + 3]), pack2(sg.z, sg.w));
      y[2 * i] = pack2(lo2(a) + hi2(a), lo2(a) - hi2(a));           // span 1
      y[2 * i + 1] = pack2(lo2(c) + hi2(c), lo2(c) - hi2(c));
    }
    const uint64_t neg = pack2(-1.f, -1.f);
    auto in_lane = [&](int i, int j) {
      const uint64_t a = y[i], b = y[j];
      y[i] = fadd2(a, b);
      y[j] = ffma2(neg, b, a);
    };
    in_lane(0, 1), in_lane(2, 3), in_lane(4, 5), in_lane(6, 7);   // span 2
    in_lane(0, 2), in_lane(1, 3), in_lane(4, 6), in_lane(5, 7);   // span 4
#pragma unroll
    for (int m = 1; m < 8; m <<= 1) {                // spans 8, 16, 32: across lanes
      const float sg = (u & m) ? -1.f : 1.f;
      const uint64_t sg2 = pack2(sg, sg);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        y[i] = ffma2(sg2, y[i], pack2(__shfl_xor_sync(0xffffffffu, lo2(y[i]), m),
                                      __shfl_xor_sync(0xffffffffu, hi2(y[i]), m)));
    }
    const uint64_t isd2 = pack2(0.08838834764831845f, 0.08838834764831845f);   // 1 / sqrt(128)
#pragma unroll
    for (int i = 0; i < 4; ++i) in_lane(i, i + 4);   // span 64
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = fmul2(y[i], isd2);
      x[2 * i] = lo2(y[i]);
      x[2 * i + 1] = hi2(y[i]);
    }
  }
}

// One page and plane: where its new rows come from and its codes go.
struct AppendSite {
  bool ok;                // it receives rows
  bool is_v;
  int page0;              // position of the page's first row
  int first, end;         // page rows [first, end) are new
  const uint16_t* src;    // row x of the page: src + x * st
  long long st;
  uint8_t* dst;           // row x: dst + x * dstep (the caller adds its lanes' columns to both)
  size_t dstep;
  float* descale;
  float before;
};

// Request b's pages are units cu[b] / page_size + 2 b and on: at least as many units
// as its cu[b + 1] - cu[b] tokens can touch pages.  Its pages with more than kFewRows new
// rows (MANY) are units cu[b] / (kFewRows + 1) and on: the first page that has as many, and
// those behind it.  The owner of a unit is found by an eight-way search in every group of
// eight lanes.
constexpr int kFewRows = 8;
template <bool MANY>
__device__ __forceinline__ AppendSite append_site(const AppendFp8Params& p, long long unit, int hv,
                                                  int page_shift, int u) {
  constexpr int D = 128;
  auto first_unit = [&](int b, int cu) -> long long {
    return MANY ? cu / (kFewRows + 1) : (static_cast<long long>(cu) >> page_shift) + 2ll * b;
  };
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = p.B;
  while (__any_sync(0xffffffffu, hi - lo > 1)) {
    const int step = (hi - lo + 7) / 8;
    const int at = lo + u * step;
    const bool below = u == 0 || (at < hi && first_unit(at, p.cu_seqlens[at]) <= unit);
    const uint32_t m = __ballot_sync(0xffffffffu, below) >> (lane & 24) & 0xffu;
    if (hi - lo > 1) {
      lo += (31 - __clz(m)) * step;
      hi = min(hi, lo + step);
    }
  }
  AppendSite s;
  s.ok = false;
  s.is_v = hv >= p.H_kv;
  s.first = s.end = 0;
  const int b = lo;
  const int c0 = p.cu_seqlens[b], c1 = p.cu_seqlens[b + 1];
  const int len = p.seq_lens[b];
  const int add = c1 - c0;
  const bool bad = c0 < 0 || c1 < c0 || c1 > p.total || len < add ||
                   len > static_cast<long long>(p.max_pages) * p.page_size;
  if (bad) {
    if (u == 0) atomicCAS(p.status, 0, kDevBadTables);
    return s;
  }
  const int start = len - add;                       // first new position
  long long lp = (start >> page_shift) + (unit - first_unit(b, c0));
  if (MANY && p.page_size - (start & (p.page_size - 1)) <= kFewRows) ++lp;
  if (add == 0 || lp < (start >> page_shift) || (lp << page_shift) >= len) return s;
  const int phys = p.block_table[static_cast<size_t>(b) * p.max_pages + lp];
  if (phys < 0 || phys >= p.num_pages) {
    if (u == 0) atomicCAS(p.status, 0, kDevBadTables);
    return s;
  }
  const int h = s.is_v ? hv - p.H_kv : hv;
  s.page0 = static_cast<int>(lp << page_shift);
  s.first = max(start, s.page0) - s.page0;
  s.end = min(len - s.page0, p.page_size);
  s.ok = !MANY || s.end - s.first > kFewRows;
  s.st = s.is_v ? p.vt : p.kt;
  // row x of the page is token c0 + (page0 + x - start)
  s.src = static_cast<const uint16_t*>(s.is_v ? p.v : p.k) + (s.is_v ? p.vh : p.kh) * h +
          s.st * (c0 + (s.page0 - start));
  s.dst = (s.is_v ? p.v_cache : p.k_cache) +
          (static_cast<size_t>(phys) * p.page_size * p.H_kv + h) * D;
  s.dstep = static_cast<size_t>(p.H_kv) * D;
  s.descale = (s.is_v ? p.v_descale : p.k_descale) + static_cast<size_t>(phys) * p.H_kv + h;
  s.before = s.first == 0 ? 0.f : *s.descale;
  if (p.cos && !s.is_v && u == 0 && s.page0 + s.end > p.max_pos) atomicCAS(p.status, 0, kDevBadTables);
  return s;
}

// Offsets of request i that do not fit are reported here: where they decrease, the search for
// a unit's owner may pass their request, and tokens of others, over.
__device__ __forceinline__ void check_offsets(const AppendFp8Params& p, long long i) {
  if (i >= p.B) return;
  const int c0 = __ldg(p.cu_seqlens + i), c1 = __ldg(p.cu_seqlens + i + 1);
  if (c0 < 0 || c1 < c0 || c1 > p.total) atomicCAS(p.status, 0, kDevBadTables);
}

struct Raw16 {
  uint4 a, b;
};
__device__ __forceinline__ Raw16 load_row(const AppendSite& s, int x) {
  const uint4* at = reinterpret_cast<const uint4*>(s.src + s.st * x);
  return {__ldg(at), __ldg(at + 8)};
}

__device__ __forceinline__ float amax16(const float (&x)[16]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; i += 2) m = fmax3(m, fabsf(x[i]), fabsf(x[i + 1]));
  return m;
}

// The least descale of a page that holds anything but zeros, 2^-90.  1 / descale and the
// quotients' residuals stay normal float32 numbers (from amax = 1.3e-36 down 1 / descale was
// infinite, and every code NaN), and so do the decode's sums of p / descale over any number of
// keys.  What it costs: values are off by up to 2^-100.
constexpr float kMinPageDescale = 0x1p-90f;

__device__ __forceinline__ float new_descale(float before, float amax) {
  const float after = fmaxf(before, __fdiv_rn(amax, 448.f));
  return after == 0.f ? 1.f : fmaxf(after, kMinPageDescale);
}

// Codes of a row, with the quotients rounded as divisions by `after`.
__device__ __forceinline__ void store_row(const AppendSite& s, int x, const float (&v)[16], uint64_t y2,
                                          uint64_t nb2) {
  uint2* at = reinterpret_cast<uint2*>(s.dst + s.dstep * x);
#pragma unroll
  for (int w = 0; w < 2; ++w)
    at[8 * w] = make_uint2(
        quantise4(pack2(v[8 * w], v[8 * w + 1]), pack2(v[8 * w + 2], v[8 * w + 3]), y2, nb2),
        quantise4(pack2(v[8 * w + 4], v[8 * w + 5]), pack2(v[8 * w + 6], v[8 * w + 7]), y2, nb2));
}

// Two e4m3 codes as exact float32 values.
__device__ __forceinline__ float2 widen_e4m3x2(uint32_t codes) {
  uint32_t h2;
  const uint16_t c = static_cast<uint16_t>(codes);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(c));
  return __half22float2(*reinterpret_cast<const __half2*>(&h2));
}
__device__ __forceinline__ uint32_t scale_codes(uint32_t w, float ratio) {
  const float2 a = widen_e4m3x2(w & 0xffffu), c = widen_e4m3x2(w >> 16);
  return cvt_pack_e4m3x4(a.x * ratio, a.y * ratio, c.x * ratio, c.y * ratio);
}

// The page's other rows, row x = from, from + by, ...: cleared behind the new ones of
// a page that starts here, requantised before them when the descale grew.  Lane u of the
// eight takes codes 16 u .. 16 u + 15.  Bound: the latency of a load and its store, row by row
// (the next load may not pass the store: some 0.16 us a row where one group of lanes walks a page).
__device__ __forceinline__ void other_rows(const AppendSite& s, float after, int page_size, int from, int by, int u) {
  uint8_t* const at = s.dst + 8 * u;                 // s.dst is at column 8 u
  if (s.first == 0) {
#pragma unroll 4
    for (int x = s.end + from; x < page_size; x += by)
      *reinterpret_cast<uint4*>(at + s.dstep * x) = make_uint4(0u, 0u, 0u, 0u);
  } else if (after > s.before) {
    const float ratio = __fdiv_rn(s.before, after);
#pragma unroll 4
    for (int x = from; x < s.first; x += by) {
      uint4* const row = reinterpret_cast<uint4*>(at + s.dstep * x);
      const uint4 c = *row;
      *row = make_uint4(scale_codes(c.x, ratio), scale_codes(c.y, ratio), scale_codes(c.z, ratio),
                        scale_codes(c.w, ratio));
    }
  }
}

// Largest magnitude of a raw row's sixteen values, in packed 16-bit maxima (exact).
template <bool FP16>
__device__ __forceinline__ float raw_amax(const Raw16& r) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
  float2 m;
  if (FP16) {
    __half2 t = __habs2(*reinterpret_cast<const __half2*>(&w[0]));
#pragma unroll
    for (int i = 1; i < 8; ++i) t = __hmax2(t, __habs2(*reinterpret_cast<const __half2*>(&w[i])));
    m = __half22float2(t);
  } else {
    __nv_bfloat162 t = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[0]));
#pragma unroll
    for (int i = 1; i < 8; ++i) t = __hmax2(t, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i])));
    m = __bfloat1622float2(t);
  }
  return fmaxf(m.x, m.y);
}

// Many rows per page: one block per page and plane, eight threads per row and a quarter
// of the page (8 to 64 rows) at a time: up to four such sweeps are copied into shared
// memory at once, every thread its own values.  A key row's transform costs some 300
// instructions per 4 rows, which bounds this kernel, so it runs once: all sweeps but the
// last staged one go back to shared memory as float32, that one stays in registers until
// the amax is known (transforming twice measured 62 us against 41 for 16 K rows of 8
// heads).  Rows of pages beyond 256 are read and transformed again, from L2.
// Small blocks for small pages, so that an SM holds many in different phases.  8 prompts
// of 2048 in pages of 16, 32, 64, 128: 65, 58, 59, 66 us; with a sweep as large as the page
// allows (up to 512 threads) 8 to 30 us more.  256 requests that bring 3 or 60 tokens each:
// 28 and 68.  (Clusters of such blocks for pages of 256: 13 us more than one
// of 512 threads.)
// Query rows are rotated by q_blocks other blocks, bound by DRAM and spread among
// these.  One of them has to keep HBM busy beside a page's block, so its rows too come
// through shared memory, seven heads in flight, two neighbouring heads of a token at a
// time (512 bytes in a piece; 2 x 8192 tokens, 32 heads: 73.4 us one by one, 68.6 so, 72.3 by fours).
constexpr int kQHeads = 2;
constexpr int kSweeps = 4;
// 16-byte words of shared memory per thread: three sweeps as float32, the last one raw
constexpr int kStagedWords = 3 * 4 + 2;
static_assert(kStagedWords == 7 * 2, "seven slots of the rotation");

template <bool FP16, int MODE, bool SIGNS, bool MANY>
__global__ void __launch_bounds__(kF8MaxThreads, 2)
    append_fp8_pages_kernel(const AppendFp8Params p, int page_shift, const RopeKParams q, unsigned q_blocks,
                            unsigned q_columns) {
  extern __shared__ uint4 stage[];                   // sweep i: words [(4 i + part) blockDim + thread]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int u = lane & 7;
  const int by = blockDim.x >> 3, mine = threadIdx.x >> 3;
  __shared__ float warp_max[kF8MaxThreads / 32];
  __shared__ __align__(16) float signs[128];
  __shared__ AppendSite site_sh;
  // query blocks among the first blockIdx.x blocks, and among one more
  const unsigned before_q = static_cast<unsigned>(static_cast<unsigned long long>(blockIdx.x) * q_blocks / gridDim.x);
  const unsigned with_q = static_cast<unsigned>((blockIdx.x + 1ull) * q_blocks / gridDim.x);
  if (with_q > before_q) {
    rope_block<FP16, MODE == kNeighbours, false, 2, 7, kQHeads>(q, before_q % q_columns, before_q / q_columns, stage);
    return;
  }
  const unsigned at_site = blockIdx.x - before_q;
  // (MANY: the few-rows kernel beside it checks them)
  if (!MANY && threadIdx.x == blockDim.x - 1) check_offsets(p, at_site);
  if (warp == 0) {
    const AppendSite found = append_site<MANY>(p, at_site / (2 * p.H_kv), at_site % (2 * p.H_kv), page_shift, u);
    if (lane == 0) site_sh = found;
  } else if (SIGNS && warp == 1) {
    *reinterpret_cast<float4*>(signs + 4 * lane) = __ldg(reinterpret_cast<const float4*>(p.signs) + lane);
  }
  __syncthreads();
  AppendSite s = site_sh;
  // MANY: a dependent launch beside the few-rows kernel, which writes other pages; only its
  // end has to be waited for
  if constexpr (MANY) {
    if (!s.ok) wait_for_previous_kernel();
  }
  if (!s.ok) return;                                 // the same for the whole block
  s.src += 8 * u;
  s.dst += 8 * u;
  uint4* const my = stage + threadIdx.x;
  const int step = blockDim.x, slot = 4 * step;
#pragma unroll
  for (int i = 0; i < kSweeps; ++i) {
    const int x = s.first + mine + i * by;
    const bool valid = x < s.end;
    const uint4* at = reinterpret_cast<const uint4*>(s.src + s.st * (valid ? x : s.first));
    copy16_async(my + i * slot, at, valid);
    copy16_async(my + i * slot + step, at + 8, valid);
    copies_commit();
  }
  const int warp_first = s.first + (warp << 2);      // first row of the warp's first sweep
  const int sweeps = warp_first < s.end ? (s.end - warp_first + by - 1) / by : 0;   // of this warp
  float v[16];
  // row s.first + mine + i * by, zeros past the new rows (the transform's shuffles are
  // warp-wide, so those lanes go along)
  auto raw_row = [&](int i) -> Raw16 {
    const int x = s.first + mine + i * by;
    return x < s.end ? load_row(s, x) : Raw16{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  };
  auto finish = [&](int i, const Raw16& r) {
    widen16<FP16>(r.a, r.b, v);
    if (!s.is_v) key_row<MODE, SIGNS>(v, p, s.page0 + s.first + mine + i * by, u, signs);
  };
  float amax = 0.f;
  const int held = min(sweeps, kSweeps) - 1;         // the last staged sweep stays in v
  auto staged = [&](int at) {
    const Raw16 r{my[at * slot], my[at * slot + step]};
    if (s.is_v) {
      amax = fmaxf(amax, raw_amax<FP16>(r));         // values are widened when stored
      return;
    }
    finish(at, r);
    amax = fmaxf(amax, amax16(v));
    if (at == held) return;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      my[at * slot + e * step] = make_uint4(__float_as_uint(v[4 * e]), __float_as_uint(v[4 * e + 1]),
                                            __float_as_uint(v[4 * e + 2]), __float_as_uint(v[4 * e + 3]));
  };
  copies_wait<3>();
  if (sweeps > 0) staged(0);
  copies_wait<2>();
  if (sweeps > 1) staged(1);
  copies_wait<1>();
  if (sweeps > 2) staged(2);
  copies_wait<0>();
  // rows beyond the staged ones before the last staged sweep
  for (int i = kSweeps; i < sweeps; ++i) {
    finish(i, raw_row(i));
    amax = fmaxf(amax, amax16(v));
  }
  if (sweeps > 3) staged(3);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (lane == 0) warp_max[warp] = amax;
  __syncthreads();                                   // also: every thread has read the old descale
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) amax = fmaxf(amax, warp_max[w]);
  const float after = new_descale(s.before, amax);
  if (threadIdx.x == 0) *s.descale = after;
  const float rcp = __fdiv_rn(1.f, after);
  const uint64_t y2 = pack2(rcp, rcp), nb2 = pack2(-after, -after);
  auto store = [&](int at) {
    const int x = s.first + mine + at * by;
    if (x < s.end) store_row(s, x, v, y2, nb2);
  };
  if (held >= 0) {
    if (s.is_v) widen16<FP16>(my[held * slot], my[held * slot + step], v);
    store(held);
  }
  for (int at = 0; at < held; ++at) {
    if (s.is_v) {
      widen16<FP16>(my[at * slot], my[at * slot + step], v);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint4 w = my[at * slot + e * step];
        v[4 * e] = __uint_as_float(w.x), v[4 * e + 1] = __uint_as_float(w.y);
        v[4 * e + 2] = __uint_as_float(w.z), v[4 * e + 3] = __uint_as_float(w.w);
      }
    }
    store(at);
  }
  for (int i = kSweeps; i < sweeps; ++i) {
    finish(i, raw_row(i));
    store(i);
  }
  other_rows(s, after, p.page_size, mine, by, u);
  if constexpr (MANY) wait_for_previous_kernel();
}

// Few rows per page (a decode step): eight lanes per page and plane, so the planes
// of a page share a block and its lookups; blocks behind them rotate query rows.  Pages with
// more than most_rows new rows are left to append_fp8_pages_kernel.  Small blocks spread a
// few requests' pages, which may have to be cleared or requantised, over the machine (64
// requests, pages of 64 and of 256, some cleared and none requantised: 5.6 and 7.7 us; in blocks
// of 256 threads 5.7 and 11.7).  A page whose descale grows has its older rows requantised by
// its eight lanes, one after the other, and the slowest sets the kernel's time: with descales of
// N(0, 1) rows, some 16 of the 64 requests' planes growing in a step, 10.5 and 48 us.
template <bool FP16, int MODE, bool SIGNS>
__global__ void __launch_bounds__(kF8Threads)
    append_fp8_rows_kernel(const AppendFp8Params p, int page_shift, long long sites, unsigned site_blocks,
                           const RopeKParams q, unsigned q_columns, int most_rows) {
  __shared__ __align__(16) float signs[128];
  if (most_rows < p.page_size) release_dependents();
  if (blockIdx.x >= site_blocks) {
    const unsigned at = blockIdx.x - site_blocks;
    rope_block<FP16, MODE == kNeighbours, false>(q, at % q_columns, at / q_columns);
    return;
  }
  const int u = threadIdx.x & 7;
  const long long site = static_cast<long long>(blockIdx.x) * (kF8Threads / 8) + (threadIdx.x >> 3);
  const int planes = 2 * p.H_kv;
  // past the last site: a unit that no request reaches
  AppendSite s = append_site<false>(p, site < sites ? site / planes : 0, static_cast<int>(site % planes), page_shift, u);
  check_offsets(p, static_cast<long long>(blockIdx.x) * kF8Threads + threadIdx.x);
  if (site >= sites || s.end - s.first > most_rows) s.ok = false;
  if (!s.ok) s.first = s.end = 0;
  s.src += 8 * u;
  s.dst += 8 * u;
  if constexpr (SIGNS) {
    if (threadIdx.x < 32)
      *reinterpret_cast<float4*>(signs + 4 * threadIdx.x) = __ldg(reinterpret_cast<const float4*>(p.signs) + threadIdx.x);
    __syncthreads();
  }
  const int rows = s.end - s.first;
  const int most = __reduce_max_sync(0xffffffffu, rows);
  float v[16];
  auto finish = [&](int i) {
    const int x = s.first + i;
    const Raw16 r = i < rows ? load_row(s, x) : Raw16{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    widen16<FP16>(r.a, r.b, v);
    // lanes of values go along (the transform's shuffles are warp-wide)
    float k[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) k[e] = v[e];
    key_row<MODE, SIGNS>(k, p, i < rows ? s.page0 + x : 0, u, signs);
    if (!s.is_v) {
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = k[e];
    }
  };
  float amax = 0.f;
  for (int i = 0; i < most; ++i) {
    finish(i);
    if (i < rows) amax = fmaxf(amax, amax16(v));
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float after = new_descale(s.before, amax);
  const float rcp = __fdiv_rn(1.f, after);
  const uint64_t y2 = pack2(rcp, rcp), nb2 = pack2(-after, -after);
  for (int i = 0; i < most; ++i) {
    if (most > 1) finish(i);
    if (i < rows) store_row(s, s.first + i, v, y2, nb2);
  }
  __syncwarp();                                      // every lane has read the old descale
  if (s.ok) {
    if (u == 0) *s.descale = after;
    other_rows(s, after, p.page_size, 0, 1, u);
  }
}

int shift_of(int page_size) {
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

template <bool FP16, int MODE, bool SIGNS>
attn_status_t launch_append_t(const AppendFp8Params& p, RopeKParams q, int page_shift, long long sites,
                              cudaStream_t stream) {
  q.status = p.status;
  // Three ways: all pages by eight lanes per plane; all by blocks per plane; or the first for
  // pages of few new rows and the second for the others.  The times are fitted to 16 to 256 rows
  // a page, 1 to 1024 requests and 8 heads.  Eight lanes: a start and the page's other rows, the
  // rows one after the other (which page they stand in is not known here; one a page is
  // assumed where there are no more tokens than requests), and their number.  Blocks: as
  // many as fit at a time, those of pages that no token reaches among them.
  // Pages of 64 whose descales do not grow, us by lanes, by blocks, by both: 64 requests with a token each 5.5, 7.7, -;
  // 256: 6.7, 22, -; 256 with 4 each 12, 24, 15; 16 of which two bring up to 30 33, 5.4, -; 256 of
  // which 32 bring up to 20 26, 24, 13.
  const int quarter = p.page_size / 4 * 8;           // threads of a sweep of a quarter of the page
  const int page_threads = quarter < 64 ? 64 : quarter > kF8MaxThreads ? kF8MaxThreads : quarter;
  const double at_a_time = 152.0 * (1024 / page_threads);
  const long long many = p.total / (kFewRows + 1) * 2 * p.H_kv;
  const double lanes = 3.5 + 0.015 * p.page_size + 4.6e-4 * p.total * 2 * p.H_kv;
  const double blocks = 2.0 + (2.5 + 20.0 / p.page_size) * std::fmax(1.0, sites / at_a_time);
  const double both = lanes + 2.0 + 1.7 * (many / at_a_time);
  enum { kLanes, kBlocks, kBoth } how = p.total <= p.B ? lanes <= blocks ? kLanes : kBlocks
                                                       : both <= blocks ? kBoth : kBlocks;
  const int threads = how == kBlocks ? page_threads : kF8Threads;
  RopeGrid g{1, 0};
  if (q.heads[0] > 0) g = rope_grid(&q, threads, how == kBlocks ? 152 * 2 : 152 * 8, how == kBlocks ? kQHeads : 1);
  const long long q_blocks = g.columns * g.chunks;
  const long long own = how == kBlocks ? sites : (sites + kF8Threads / 8 - 1) / (kF8Threads / 8);
  if (own + q_blocks > 2147483647LL) return fail(ATTN_ERR_UNSUPPORTED, "grid dimension limit exceeded");
  const unsigned grid = static_cast<unsigned>(own + q_blocks), columns = static_cast<unsigned>(g.columns);
  const unsigned qb = static_cast<unsigned>(q_blocks);
  const int page_smem = kStagedWords * 16 * page_threads;
  cudaError_t e = cudaSuccess;
  if (how == kBlocks) {
    auto kern = append_fp8_pages_kernel<FP16, MODE, SIGNS, false>;
    const attn_status_t s = set_smem(reinterpret_cast<const void*>(kern), kStagedWords * 16 * kF8MaxThreads);
    if (s != ATTN_OK) return s;
    kern<<<grid, page_threads, page_smem, stream>>>(p, page_shift, q, qb, columns);
    e = cudaGetLastError();
  } else {
    const bool rest = how == kBoth && many > 0;
    append_fp8_rows_kernel<FP16, MODE, SIGNS><<<grid, threads, 0, stream>>>(
        p, page_shift, sites, static_cast<unsigned>(own), q, columns, rest ? kFewRows : p.page_size);
    e = cudaGetLastError();
    if (e == cudaSuccess && rest) {
      auto kern = append_fp8_pages_kernel<FP16, MODE, SIGNS, true>;
      const attn_status_t s = set_smem(reinterpret_cast<const void*>(kern), kStagedWords * 16 * kF8MaxThreads);
      if (s != ATTN_OK) return s;
      e = launch_dependent(kern, dim3(static_cast<unsigned>(many)), page_threads, page_smem, stream, 0, p, page_shift, q,
                           0u, 1u);
    }
  }
  if (e != cudaSuccess) return fail_cuda(e, "FP8 append kernel launch");
  return ATTN_OK;
}

template <bool FP16, int MODE>
attn_status_t launch_append_m(const AppendFp8Params& p, const RopeKParams& q, int page_shift, long long sites,
                              cudaStream_t stream) {
  return p.signs ? launch_append_t<FP16, MODE, true>(p, q, page_shift, sites, stream)
                 : launch_append_t<FP16, MODE, false>(p, q, page_shift, sites, stream);
}

template <bool FP16>
attn_status_t launch_append(const AppendFp8Params& p, const RopeKParams& q, int interleaved, int page_shift,
                            long long sites, cudaStream_t stream) {
  if (!p.cos) return launch_append_m<FP16, kPlain>(p, q, page_shift, sites, stream);
  if (interleaved) return launch_append_m<FP16, kNeighbours>(p, q, page_shift, sites, stream);
  return p.rot == 128 ? launch_append_m<FP16, kHalves>(p, q, page_shift, sites, stream)
                      : launch_append_m<FP16, kHalvesPart>(p, q, page_shift, sites, stream);
}

}  // namespace

attn_status_t launch_block_tables(const TablesParams& p, cudaStream_t stream) {
  if (p.B > kTabMaxB) return fail(ATTN_ERR_UNSUPPORTED, "block tables: at most 16384 requests");
  int* status = device_status_word();
  if (!status) return fail(ATTN_ERR_CUDA, "status word unavailable");
  const int smem = (3 * p.B + 2) * static_cast<int>(sizeof(int));
  if (smem > 48 * 1024) {
    const attn_status_t s = set_smem(reinterpret_cast<const void*>(block_tables_kernel), (3 * kTabMaxB + 2) * 4);
    if (s != ATTN_OK) return s;
  }
  // one thread per token, at most two blocks per SM
  long long blocks = (static_cast<long long>(p.capacity) + kTabThreads - 1) / kTabThreads;
  blocks = blocks < 1 ? 1 : blocks > 304 ? 304 : blocks;
  const cudaError_t e = launch_dependent(block_tables_kernel, dim3(static_cast<unsigned>(blocks)), kTabThreads, smem,
                                         stream, 0, p, status, shift_of(p.page_size));
  if (e != cudaSuccess) return fail_cuda(e, "block table kernel launch");
  return ATTN_OK;
}

attn_status_t launch_append_fp8(AppendFp8Params p, RopeKParams q, int fp16, int interleaved,
                                cudaStream_t stream) {
  p.status = device_status_word();
  if (!p.status) return fail(ATTN_ERR_CUDA, "status word unavailable");
  const int shift = shift_of(p.page_size);
  const long long units = (static_cast<long long>(p.total) >> shift) + 2ll * p.B;
  const long long sites = units * 2 * p.H_kv;
  if (sites > 2147483647LL) return fail(ATTN_ERR_UNSUPPORTED, "grid dimension limit exceeded");
  return fp16 ? launch_append<true>(p, q, interleaved, shift, sites, stream)
              : launch_append<false>(p, q, interleaved, shift, sites, stream);
}

}  // namespace attn
