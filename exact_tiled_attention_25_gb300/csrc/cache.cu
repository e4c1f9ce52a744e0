// Upkeep of a paged key/value cache: block tables and slot maps built from
// request lengths, and new keys and values written to the cache, in 16 bits or
// as e4m3 codes with one scale per (page, key/value head).  "FlashAttention 3
// Hardware Acceleration: Hopper GPU Strategies for Long-Context Enterprise
// Inference Optimization", section "Memory Fragmentation", describes the cache
// in fixed-size blocks; the paged decode (decode.cu) reads what these write.
#include "common.h"
#include "fp8_row.cuh"
#include "rope.cuh"

namespace attn {
namespace {

// ============================================================ block tables ====
constexpr int kTabThreads = 512;
constexpr int kTabMaxB = 16384;   // 8 bytes of shared memory per request

// Exclusive prefix sums of new tokens and new pages over all requests, in every
// block (the requests' lengths are a few KB of L2 hits, cheaper than a second
// launch), then this block's share of the outputs.  Request b has old_lens[b]
// tokens in ceil(old / page_size) pages; its new pages take consecutive entries
// of the free list, requests in order.  New table entries are taken from the
// free list directly, so no block reads what another writes.
// Bound: latency -- a launch, the scan's barriers and one dependent chain of
// loads (length, table entry, store).
__global__ void __launch_bounds__(kTabThreads)
    block_tables_kernel(const TablesParams p, int* status, int page_shift) {
  extern __shared__ int tab_sh[];
  int* cu = tab_sh;                  // [B + 1] first new token of each request
  int* pg = tab_sh + p.B + 1;        // [B + 1] first free-list entry of each request
  __shared__ long long warp_sum[2][kTabThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int page = p.page_size;
  const long long room = static_cast<long long>(p.max_pages) * page;
  bool bad = false;
  long long tok_base = 0, page_base = 0;
  for (int b0 = 0; b0 < p.B; b0 += kTabThreads) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    long long tok = 0, pages = 0;
    if (b < p.B) {
      int old = p.old_lens[b], add = p.new_lens[b];
      if (old < 0 || old > room || add < 0 || old + static_cast<long long>(add) > room) {
        bad = true;
        old = old < 0 || old > room ? 0 : old;
        add = 0;
      }
      tok = add;
      pages = ((old + static_cast<long long>(add) + page - 1) >> page_shift) -
              ((static_cast<long long>(old) + page - 1) >> page_shift);
      if (blockIdx.x == 0) p.seq_lens[b] = old + add;
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
    long long tw = 0, pw = 0, tall = 0, pall = 0;
#pragma unroll
    for (int w = 0; w < kTabThreads / 32; ++w) {
      if (w == warp) {
        tw = tall;
        pw = pall;
      }
      tall += warp_sum[0][w];
      pall += warp_sum[1][w];
    }
    if (b < p.B) {
      const long long t = tok_base + tw + ts - tok, q = page_base + pw + ps - pages;
      cu[b] = static_cast<int>(t < 2147483647LL ? t : 2147483647LL);
      pg[b] = static_cast<int>(q < 2147483647LL ? q : 2147483647LL);
    }
    tok_base += tall;
    page_base += pall;
    __syncthreads();
  }
  const int total = static_cast<int>(tok_base < 2147483647LL ? tok_base : 2147483647LL);
  const int pages_all = static_cast<int>(page_base < 2147483647LL ? page_base : 2147483647LL);
  if (threadIdx.x == 0) {
    cu[p.B] = total;
    pg[p.B] = pages_all;
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b <= p.B; b += kTabThreads) p.cu_seqlens[b] = cu[b];
    if (threadIdx.x == 0) p.used[0] = min(pages_all, p.n_free);
    if (bad || (threadIdx.x == 0 && (tok_base > p.capacity || page_base > p.n_free)))
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
  auto valid_old = [&](int b) {
    const int old = p.old_lens[b];
    return old < 0 || old > room ? 0 : old;
  };
  const int step = gridDim.x * kTabThreads;
  const int me = blockIdx.x * kTabThreads + threadIdx.x;
  for (long long t = me; t < p.capacity; t += step) {
    long long slot = -1;
    int pos = -1;
    if (t < total) {
      const int b = owner(cu, static_cast<int>(t));
      const int old = valid_old(b);
      pos = old + (static_cast<int>(t) - cu[b]);
      const int lp = pos >> page_shift;
      const int have = static_cast<int>((static_cast<long long>(old) + page - 1) >> page_shift);
      int phys;
      if (lp < have) {
        phys = p.block_table[static_cast<size_t>(b) * p.max_pages + lp];
      } else {
        const long long e = static_cast<long long>(pg[b]) + (lp - have);
        phys = e < p.n_free ? p.free_pages[e] : -1;
      }
      if (phys >= 0) slot = static_cast<long long>(phys) * page + (pos & (page - 1));
    }
    p.slots[t] = slot;
    p.positions[t] = pos;
  }
  for (long long e = me; e < pages_all; e += step) {
    const int b = owner(pg, static_cast<int>(e));
    const int have = static_cast<int>((static_cast<long long>(valid_old(b)) + page - 1) >> page_shift);
    p.block_table[static_cast<size_t>(b) * p.max_pages + have + (e - pg[b])] =
        e < p.n_free ? p.free_pages[e] : -1;
  }
}

// ========================================================== e4m3 append ====
// One block per (page that receives tokens, key/value head, keys or values).
// The page's new rows are rotated and transformed (keys), their amax gives
//   descale' = max(descale, amax / 448)       (a page whose first token is among
//                                              the new ones starts from 0),
// codes = e4m3_rn_satfinite(x / descale'); when the descale grows, the codes of
// the page's older tokens become e4m3_rn(code * (descale / descale')); the
// unused rest of a page that starts here is cleared, so the decode never meets
// another request's codes or a NaN there.  A page belongs to one block per head,
// so there are no atomics and the result does not depend on any order.
// A warp holds a row as 32 lanes x 4 values, as the FP8 pre-pass does.
constexpr int kF8MaxThreads = 256;
constexpr int kF8Rows = 8;         // rows a warp keeps in registers between the two passes

// Request whose pages include unit u: request b's units start at
// cu[b] / page_size + 2 b, which leaves it at least as many as the pages that
// its cu[b + 1] - cu[b] tokens can touch.  A 32-way search, in every warp.
__device__ __forceinline__ int unit_owner(const int* cu, int B, int page_shift, long long u, int lane) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const bool below = at < hi && (static_cast<long long>(cu[at]) >> page_shift) + 2ll * at <= u;
    const uint32_t m = __ballot_sync(0xffffffffu, below || lane == 0);
    lo += (31 - __clz(m)) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

template <bool FP16>
__device__ __forceinline__ float4 widen4(uint2 w) {
  if (FP16) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
    return make_float4(a.x, a.y, b.x, b.y);
  }
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                     __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}

// Row of keys in the lanes of a warp: rotated by the table row of `pos`, then
// transformed by M = diag(signs) H_128 / sqrt(128).
template <bool INTERLEAVED>
__device__ __forceinline__ float4 key_row(float4 v, const AppendFp8Params& p, int pos, int lane,
                                          const float4& s4) {
  if (p.cos) {
    const bool turn = 4 * lane < p.rot && pos < p.max_pos;
    const size_t row = static_cast<size_t>(turn ? pos : 0) * (p.rot / 2);
    if (INTERLEAVED) {
      if (turn) {
        const float2 c = __ldg(reinterpret_cast<const float2*>(p.cos + row) + lane);
        const float2 s = __ldg(reinterpret_cast<const float2*>(p.sin + row) + lane);
        v = make_float4(fmaf(-v.y, s.x, v.x * c.x), fmaf(v.x, s.x, v.y * c.x),
                        fmaf(-v.w, s.y, v.z * c.y), fmaf(v.z, s.y, v.w * c.y));
      }
    } else {
      const int half = p.rot / 8;                    // lanes of one half
      const bool lower = lane < half;
      const int other = turn ? (lower ? lane + half : lane - half) : lane;
      const float ox = __shfl_sync(0xffffffffu, v.x, other);
      const float oy = __shfl_sync(0xffffffffu, v.y, other);
      const float oz = __shfl_sync(0xffffffffu, v.z, other);
      const float ow = __shfl_sync(0xffffffffu, v.w, other);
      if (turn) {
        const int i = lower ? lane : lane - half;
        const float4 c = __ldg(reinterpret_cast<const float4*>(p.cos + row) + i);
        const float4 s = __ldg(reinterpret_cast<const float4*>(p.sin + row) + i);
        const float sg = lower ? -1.f : 1.f;         // x c - y s, and y c + x s
        v = make_float4(fmaf(sg * ox, s.x, v.x * c.x), fmaf(sg * oy, s.y, v.y * c.y),
                        fmaf(sg * oz, s.z, v.z * c.z), fmaf(sg * ow, s.w, v.w * c.w));
      }
    }
  }
  if (p.signs) {
    uint64_t p01 = fmul2(pack2(v.x, v.y), pack2(s4.x, s4.y));
    uint64_t p23 = fmul2(pack2(v.z, v.w), pack2(s4.z, s4.w));
    wht128_row(p01, p23, lane);
    const uint64_t isd2 = pack2(0.08838834764831845f, 0.08838834764831845f);   // 1 / sqrt(128)
    p01 = fmul2(p01, isd2);
    p23 = fmul2(p23, isd2);
    v = make_float4(lo2(p01), hi2(p01), lo2(p23), hi2(p23));
  }
  return v;
}

__device__ __forceinline__ float amax4(float m, const float4& v) {
  return fmax3(m, fmax3(fabsf(v.x), fabsf(v.y), fabsf(v.z)), fabsf(v.w));
}

// Two e4m3 codes as exact float32 values.
__device__ __forceinline__ float2 widen_e4m3x2(uint32_t codes) {
  uint32_t h2;
  const uint16_t c = static_cast<uint16_t>(codes);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(c));
  return __half22float2(*reinterpret_cast<const __half2*>(&h2));
}

template <bool FP16, bool INTERLEAVED>
__device__ __forceinline__ void append_fp8_block(const AppendFp8Params& p, long long unit, int hv,
                                                 int page_shift) {
  constexpr int D = 128;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = blockDim.x >> 5;
  __shared__ float warp_max[kF8MaxThreads / 32];
  const int b = unit_owner(p.cu_seqlens, p.B, page_shift, unit, lane);
  const int c0 = p.cu_seqlens[b], c1 = p.cu_seqlens[b + 1];
  const int len = p.seq_lens[b];
  const int add = c1 - c0;
  if (c0 < 0 || c1 < c0 || c1 > p.total || len < add ||
      len > static_cast<long long>(p.max_pages) * p.page_size) {
    if (threadIdx.x == 0) atomicCAS(p.status, 0, kDevBadTables);
    return;
  }
  const int start = len - add;                       // first new position
  const long long lp = (start >> page_shift) + (unit - ((static_cast<long long>(c0) >> page_shift) + 2ll * b));
  if (add == 0 || lp < 0 || lp << page_shift >= len) return;
  const int phys = p.block_table[static_cast<size_t>(b) * p.max_pages + lp];
  if (phys < 0 || phys >= p.num_pages) {
    if (threadIdx.x == 0) atomicCAS(p.status, 0, kDevBadTables);
    return;
  }
  const int page0 = static_cast<int>(lp << page_shift);
  const int first = max(start, page0) - page0;       // page rows [first, end) are new
  const int end = min(len - page0, p.page_size);
  const bool is_v = hv >= p.H_kv;
  const int h = is_v ? hv - p.H_kv : hv;
  const uint16_t* src = static_cast<const uint16_t*>(is_v ? p.v : p.k);
  const long long st = is_v ? p.vt : p.kt;
  // row x of the page is token c0 + (page0 + x - start)
  src += (is_v ? p.vh : p.kh) * h + st * (c0 + (page0 - start));
  uint8_t* dst = (is_v ? p.v_cache : p.k_cache) + (static_cast<size_t>(phys) * p.page_size * p.H_kv + h) * D;
  const size_t dstep = static_cast<size_t>(p.H_kv) * D;
  float* descale = (is_v ? p.v_descale : p.k_descale) + static_cast<size_t>(phys) * p.H_kv + h;
  const float before = first == 0 ? 0.f : *descale;
  float4 s4 = make_float4(1.f, 1.f, 1.f, 1.f);
  if (p.signs && !is_v) s4 = __ldg(reinterpret_cast<const float4*>(p.signs) + lane);
  if (p.cos && !is_v && threadIdx.x == 0 && page0 + end > p.max_pos) atomicCAS(p.status, 0, kDevBadTables);

  auto load = [&](int x) {
    return __ldg(reinterpret_cast<const uint2*>(src + st * x) + lane);
  };
  auto finish = [&](uint2 w, int x) {
    const float4 v = widen4<FP16>(w);
    return is_v ? v : key_row<INTERLEAVED>(v, p, page0 + x, lane, s4);
  };
  // pass 1: the rows' amax; a warp's first kF8Rows rows stay in registers
  float4 kept[kF8Rows];
  uint2 raw[kF8Rows];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kF8Rows; ++i) {
    const int x = first + warp + i * warps;
    raw[i] = x < end ? load(x) : make_uint2(0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < kF8Rows; ++i) {
    const int x = first + warp + i * warps;
    if (x < end) {                                   // the same for the whole warp
      kept[i] = finish(raw[i], x);
      amax = amax4(amax, kept[i]);
    }
  }
  for (int x = first + warp + kF8Rows * warps; x < end; x += warps) amax = amax4(amax, finish(load(x), x));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (lane == 0) warp_max[warp] = amax;
  __syncthreads();                                   // also: every thread has read the old descale
  for (int w = 0; w < warps; ++w) amax = fmaxf(amax, warp_max[w]);
  float after = fmaxf(before, __fdiv_rn(amax, 448.f));
  if (after == 0.f) after = 1.f;
  if (threadIdx.x == 0) *descale = after;
  const float rcp = __fdiv_rn(1.f, after);
  const uint64_t y2 = pack2(rcp, rcp), nb2 = pack2(-after, -after);
  // pass 2: codes
  auto store = [&](const float4& v, int x) {
    reinterpret_cast<uint32_t*>(dst + dstep * x)[lane] =
        quantise4(pack2(v.x, v.y), pack2(v.z, v.w), y2, nb2);
  };
#pragma unroll
  for (int i = 0; i < kF8Rows; ++i) {
    const int x = first + warp + i * warps;
    if (x < end) store(kept[i], x);
  }
  for (int x = first + warp + kF8Rows * warps; x < end; x += warps) store(finish(load(x), x), x);
  if (first == 0) {
    for (int x = end + warp; x < p.page_size; x += warps)
      reinterpret_cast<uint32_t*>(dst + dstep * x)[lane] = 0u;
  } else if (after > before) {
    const float ratio = __fdiv_rn(before, after);
#pragma unroll 4
    for (int x = warp; x < first; x += warps) {
      uint32_t* at = reinterpret_cast<uint32_t*>(dst + dstep * x) + lane;
      const uint32_t w = *at;
      const float2 a = widen_e4m3x2(w & 0xffffu), c = widen_e4m3x2(w >> 16);
      *at = cvt_pack_e4m3x4(a.x * ratio, a.y * ratio, c.x * ratio, c.y * ratio);
    }
  }
}

// Blocks [0, units * 2 H_kv): pages; the rest rotate query rows.
template <bool FP16, bool INTERLEAVED>
__global__ void __launch_bounds__(kF8MaxThreads)
    append_fp8_kernel(const AppendFp8Params p, int page_shift, long long page_blocks,
                      const RopeKParams q, unsigned q_columns) {
  const long long x = blockIdx.x;
  if (x >= page_blocks) {
    const unsigned at = static_cast<unsigned>(x - page_blocks);
    rope_block<FP16, INTERLEAVED>(q, at % q_columns, at / q_columns);
    return;
  }
  const int planes = 2 * p.H_kv;
  append_fp8_block<FP16, INTERLEAVED>(p, x / planes, static_cast<int>(x % planes), page_shift);
}

int shift_of(int page_size) {
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

}  // namespace

attn_status_t launch_block_tables(const TablesParams& p, cudaStream_t stream) {
  if (p.B > kTabMaxB) return fail(ATTN_ERR_UNSUPPORTED, "block tables: at most 16384 requests");
  int* status = device_status_word();
  if (!status) return fail(ATTN_ERR_CUDA, "status word unavailable");
  const int smem = 2 * (p.B + 1) * static_cast<int>(sizeof(int));
  attn_status_t s = set_smem(reinterpret_cast<const void*>(block_tables_kernel), 2 * (kTabMaxB + 1) * 4);
  if (s != ATTN_OK) return s;
  // one thread per token, at most two blocks per SM
  long long blocks = (static_cast<long long>(p.capacity) + kTabThreads - 1) / kTabThreads;
  blocks = blocks < 1 ? 1 : blocks > 304 ? 304 : blocks;
  block_tables_kernel<<<static_cast<unsigned>(blocks), kTabThreads, smem, stream>>>(p, status,
                                                                                   shift_of(p.page_size));
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail_cuda(e, "block table kernel launch");
  return ATTN_OK;
}

attn_status_t launch_append_fp8(AppendFp8Params p, RopeKParams q, int fp16, int interleaved,
                                cudaStream_t stream) {
  p.status = device_status_word();
  if (!p.status) return fail(ATTN_ERR_CUDA, "status word unavailable");
  const int shift = shift_of(p.page_size);
  const long long units = (static_cast<long long>(p.total) >> shift) + 2ll * p.B;
  const long long page_blocks = units * 2 * p.H_kv;
  RopeGrid g{1, 0};
  if (q.heads[0] > 0) g = rope_grid(&q);
  q.status = p.status;
  const long long blocks = page_blocks + g.columns * g.chunks;
  if (blocks > 2147483647LL) return fail(ATTN_ERR_UNSUPPORTED, "grid dimension limit exceeded");
  static_assert(kF8MaxThreads == kRopeThreads, "one block size for both roles");
  const int threads = kF8MaxThreads;
  const unsigned grid = static_cast<unsigned>(blocks);
#define ATTN_APPEND(F, I) append_fp8_kernel<F, I><<<grid, threads, 0, stream>>>( \
      p, shift, page_blocks, q, static_cast<unsigned>(g.columns))
  if (fp16) {
    if (interleaved) ATTN_APPEND(true, true);
    else ATTN_APPEND(true, false);
  } else {
    if (interleaved) ATTN_APPEND(false, true);
    else ATTN_APPEND(false, false);
  }
#undef ATTN_APPEND
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail_cuda(e, "FP8 append kernel launch");
  return ATTN_OK;
}

}  // namespace attn
