// Ranges of positions of a paged cache back as 16-bit rows: out of a 16-bit cache, an e4m3
// one (a descale per page and head) or a 4-bit one (fp4.cuh).  Keys that were stored
// transformed, x M with M = diag(signs) H_d / sqrt(d), come back as x: M is orthogonal, so
// x = (x M) M^T = ((x M) H_d / sqrt(d)) o signs.
//
// d / 16 lanes hold a row: lane u the columns 8 u .. 8 u + 7 and d / 2 + 8 u .., so that a
// store of the lanes together is whole sectors (with 16 neighbouring columns each, a store
// wrote every other half of them).
// Bound: DRAM, the writes above all (4 d bytes a key and value against d + 4 read from the
// 4-bit cache).  A dependent launch: it reads past the L1 cache.
#include "common.h"
#include "fp4.cuh"
#include "rope.cuh"

namespace attn {
namespace {

constexpr int kThreads = 128;

enum : int { k16 = 0, k8 = 1, k4 = 2 };

// Where a row of the output comes from.
struct Site {
  int phys;        // page; -1: the row is written as zeros
  int off;         // row of the page
};

// Position `pos` of request b, whose range has been checked against its length.
__device__ __forceinline__ Site site_of(const CacheReadParams& p, int b, int pos) {
  const int phys = __ldcg(p.block_table + static_cast<size_t>(b) * p.max_pages + (pos >> p.page_shift));
  if (phys < 0 || phys >= p.num_pages) {
    atomicCAS(p.status, 0, kDevBadTables);
    return {-1, 0};
  }
  return {phys, pos & (p.page_size - 1)};
}

// Length and first position of request b: {0, 0} (reported) for what does not fit.
__device__ __forceinline__ int2 range_of(const CacheReadParams& p, int b) {
  const int len = __ldcg(p.seq_lens + b), first = p.first ? __ldcg(p.first + b) : 0;
  if (len < 0 || len > static_cast<long long>(p.max_pages) * p.page_size || first < 0) {
    atomicCAS(p.status, 0, kDevBadTables);
    return make_int2(0, 0);
  }
  return make_int2(len, first);
}

template <int FORMAT>
struct Raw {
  uint4 a, b;
};
template <>
struct Raw<k8> {
  uint2 a, b;
  float s;
};
template <>
struct Raw<k4> {
  uint32_t a, b;
  float s;
};

template <int D, int FORMAT>
__device__ __forceinline__ Raw<FORMAT> load_raw(const CacheReadParams& p, bool is_v, int h, Site at, int u) {
  const uint8_t* cache = static_cast<const uint8_t*>(is_v ? p.v_cache : p.k_cache);
  if constexpr (FORMAT == k4) {
    const size_t row = (static_cast<size_t>(at.phys) * p.H_kv + h) * p.page_size + at.off;
    const uint16_t* s = static_cast<const uint16_t*>(is_v ? p.v_descale : p.k_descale);
    const uint32_t* x = reinterpret_cast<const uint32_t*>(cache + row * (D / 2)) + u;
    return {__ldcg(x), __ldcg(x + D / 16), bf16_bits(__ldcg(s + row))};
  } else {
    const size_t row = (static_cast<size_t>(at.phys) * p.page_size + at.off) * p.H_kv + h;
    if constexpr (FORMAT == k8) {
      const float* s = static_cast<const float*>(is_v ? p.v_descale : p.k_descale);
      const uint2* x = reinterpret_cast<const uint2*>(cache + row * D) + u;
      return {__ldcg(x), __ldcg(x + D / 16), __ldcg(s + static_cast<size_t>(at.phys) * p.H_kv + h)};
    } else {
      const uint4* x = reinterpret_cast<const uint4*>(cache + row * (2 * D)) + u;
      return {__ldcg(x), __ldcg(x + D / 16)};
    }
  }
}

template <int FORMAT>
__device__ __forceinline__ void widen(const Raw<FORMAT>& r, float (&x)[16]) {
  if constexpr (FORMAT == k4) {
    const uint32_t w[2] = {r.a, r.b};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t h[4];
      e2m1_halves(w[i], h);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[e]));
        x[8 * i + 2 * e] = f.x * r.s;
        x[8 * i + 2 * e + 1] = f.y * r.s;
      }
    }
  } else if constexpr (FORMAT == k8) {
    const uint32_t w[4] = {r.a.x, r.a.y, r.b.x, r.b.y};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t h2;
      const uint16_t c = static_cast<uint16_t>(w[i / 2] >> (i & 1 ? 16 : 0));
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(c));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
      x[2 * i] = f.x * r.s;
      x[2 * i + 1] = f.y * r.s;
    }
  }
}

// (x H_d / sqrt(d)) o signs of x / d, whose sums are in range for every x (a power of two: the
// same bits): spans 1, 2, 4 in the lane, 8 .. d / 4 across lanes, d / 2 in the lane.
template <int D>
__device__ __forceinline__ void restore_row(float (&x)[16], const float* signs, int u) {
#pragma unroll
  for (int h = 1; h < 8; h <<= 1)
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if ((i & h) == 0) {
        const float a = x[i], b = x[i + h];
        x[i] = a + b;
        x[i + h] = a - b;
      }
#pragma unroll
  for (int m = 1; m < D / 16; m <<= 1) {
    const float sgn = (u & m) ? -1.f : 1.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = fmaf(sgn, x[i], __shfl_xor_sync(0xffffffffu, x[i], m));
  }
  const float root = D == 128 ? 11.313708498984761f : 8.f;      // sqrt(d)
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    const float4 s = *reinterpret_cast<const float4*>(signs + 8 * u + i);
    const float4 r = *reinterpret_cast<const float4*>(signs + D / 2 + 8 * u + i);
    const float sv[4] = {s.x, s.y, s.z, s.w}, rv[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = x[i + e], b = x[8 + i + e];
      x[i + e] = (a + b) * (root * sv[e]);
      x[8 + i + e] = (a - b) * (root * rv[e]);
    }
  }
}

// A block: kThreads / (d / 16) rows, a row of a thread, of one request (padded output) or of the
// packed batch, in `per` planes: keys and values of head 0, of head 1, ...  What a row needs is
// looked up once for all of them, and a plane's row is loaded before the last one's is stored.
template <int D, int FORMAT, bool FP16, bool SIGNS>
__global__ void __launch_bounds__(kThreads)
    cache_read_kernel(const CacheReadParams p, int per) {
  constexpr int L = D / 16, G = kThreads / L;
  const int u = threadIdx.x % L;
  const long long row0 = static_cast<long long>(blockIdx.x) * G, i = row0 + threadIdx.x / L;
  size_t out0 = 8 * u;                                // of head 0's row i
  Site at{-1, 0};
  bool write = false;
  // What every row needs comes through shared memory: read from L2 by each warp, the lines
  // of the signs and the lengths bounded the kernel (571 us for 8 prefixes of up to 16384).
  __shared__ __align__(16) float signs[SIGNS ? D : 4];
  __shared__ int2 range_sh[kThreads];                 // of requests from `lo` on (packed)
  __shared__ int cu_sh[kThreads + 1];
  wait_for_previous_kernel();
  if (SIGNS && threadIdx.x < D / 4)
    *reinterpret_cast<float4*>(signs + 4 * threadIdx.x) = __ldcg(reinterpret_cast<const float4*>(p.signs) + threadIdx.x);
  if (p.cu_seqlens == nullptr) {
    const int b = blockIdx.z;
    if (threadIdx.x == kThreads - 1) range_sh[0] = range_of(p, b);
    __syncthreads();
    const int2 r = range_sh[0];
    out0 += (static_cast<size_t>(b) * p.H_kv * p.n + i) * D;
    write = i < p.n;
    if (write && r.y + i < r.x) at = site_of(p, b, static_cast<int>(r.y + i));
  } else {
    out0 += static_cast<size_t>(i) * p.H_kv * D;
    // the request that owns the block's first row, by a search with all threads until
    // kThreads requests are left; those are kept
    int lo = 0, hi = p.B;
    while (hi - lo > kThreads) {
      const int step = (hi - lo + kThreads - 1) / kThreads, probe = lo + static_cast<int>(threadIdx.x) * step;
      const int below = __syncthreads_count(threadIdx.x == 0 || (probe < hi && __ldcg(p.cu_seqlens + probe) <= row0));
      lo += (below - 1) * step;
      hi = min(hi, lo + step);
    }
    const int have = min(kThreads, p.B - lo);
    if (static_cast<int>(threadIdx.x) < have) {
      cu_sh[threadIdx.x] = __ldcg(p.cu_seqlens + lo + threadIdx.x);
      range_sh[threadIdx.x] = range_of(p, lo + threadIdx.x);
    }
    if (threadIdx.x == 0) cu_sh[have] = __ldcg(p.cu_seqlens + lo + have);
    __syncthreads();
    if (i < p.n) {
      // the last request that starts at or before row i
      int a = 0, z = have;
      while (z - a > 1) {
        const int mid = (a + z) >> 1;
        if (cu_sh[mid] <= i) a = mid;
        else z = mid;
      }
      int b = lo + a, c0 = cu_sh[a], c1 = cu_sh[a + 1];
      int2 r = range_sh[a];
      if (i >= c1 && lo + have < p.B) {
        // behind the requests at hand (many empty ones)
        int z2 = p.B;
        while (z2 - b > 1) {
          const int mid = (b + z2) >> 1;
          if (__ldcg(p.cu_seqlens + mid) <= i) b = mid;
          else z2 = mid;
        }
        c0 = __ldcg(p.cu_seqlens + b), c1 = __ldcg(p.cu_seqlens + b + 1);
        r = range_of(p, b);
      }
      write = i >= c0 && i < c1;                       // rows behind the last request stay
      if (write) {
        const long long pos = r.y + (i - c0);
        if (pos < r.x) at = site_of(p, b, static_cast<int>(pos));
        else atomicCAS(p.status, 0, kDevBadTables);
      }
    }
    // offsets that do not fit
    if (blockIdx.x == 0 && blockIdx.y == 0)
      for (int b = threadIdx.x; b < p.B; b += kThreads) {
        const int c0 = __ldcg(p.cu_seqlens + b), c1 = __ldcg(p.cu_seqlens + b + 1);
        if (c0 < 0 || c1 < c0 || c1 > p.n || (b == 0 && c0 != 0)) atomicCAS(p.status, 0, kDevBadTables);
      }
  }
  const size_t head = p.cu_seqlens == nullptr ? static_cast<size_t>(p.n) * D : D;
  const int plane0 = blockIdx.y * per, plane1 = min(plane0 + per, 2 * p.H_kv);
  const bool some = __any_sync(0xffffffffu, at.phys >= 0);
  Raw<FORMAT> next{};
  if (at.phys >= 0) next = load_raw<D, FORMAT>(p, plane0 & 1, plane0 >> 1, at, u);
  for (int plane = plane0; plane < plane1; ++plane) {
    const bool is_v = plane & 1;
    const Raw<FORMAT> raw = next;
    if (at.phys >= 0 && plane + 1 < plane1) next = load_raw<D, FORMAT>(p, (plane + 1) & 1, (plane + 1) >> 1, at, u);
    uint4 a, b;
    if constexpr (FORMAT == k16) {
      a = raw.a, b = raw.b;
    } else if (!some) {
      a = b = make_uint4(0u, 0u, 0u, 0u);
    } else {
      float x[16];
      Raw<FORMAT> part = raw;
      if (SIGNS && !is_v) part.s /= D;
      widen<FORMAT>(part, x);
      if (SIGNS && !is_v) restore_row<D>(x, signs, u);
      uint32_t w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        w[e] = FP16 ? cvt_pack_f16(x[2 * e], x[2 * e + 1]) : cvt_pack_bf16(x[2 * e], x[2 * e + 1]);
      a = make_uint4(w[0], w[1], w[2], w[3]);
      b = make_uint4(w[4], w[5], w[6], w[7]);
    }
    if (write) {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? p.v_out : p.k_out) + out0 + (plane >> 1) * head);
      dst[0] = a;
      dst[L] = b;
    }
  }
}

// A plane a block, and several where 152 x 16 blocks are left so: a threshold found by trying, not
// a wave (of 128 threads with 40 to 56 registers 9 to 12 blocks fit on an SM).  16,000 packed rows of 16
// requests, 8 heads: a plane each 30 us, so 24.0, with half of the blocks 27; 8 ranges of up to 16384
// tokens 100.8 (6.0 TB/s); one of 509 tokens 3.2; e4m3, 65,536 packed rows of 4 heads 37.0.  Four rows of a
// thread instead, a plane each, took 28, 102, 5.0 and 38.6.  The 8 ranges of a 16-bit cache 121.5, packed 82
// (6.6 and 6.3 TB/s).
template <int D, int FORMAT, bool FP16, bool SIGNS>
attn_status_t launch_t(const CacheReadParams& p, cudaStream_t stream) {
  constexpr int rows = kThreads / (D / 16);
  const long long columns = (p.n + rows - 1LL) / rows, entries = p.cu_seqlens ? 1 : p.B;
  int per = 1;
  while (per < 2 * p.H_kv && columns * entries * 2 * p.H_kv / (2 * per) >= 152 * 16) per *= 2;
  const dim3 grid(static_cast<unsigned>(columns), (2 * p.H_kv + per - 1) / per, static_cast<unsigned>(entries));
  const cudaError_t e = launch_dependent(cache_read_kernel<D, FORMAT, FP16, SIGNS>, grid, kThreads, 0, stream, 0, p, per);
  return e == cudaSuccess ? ATTN_OK : fail_cuda(e, "cache read kernel launch");
}

template <int D, int FORMAT>
attn_status_t launch_f(const CacheReadParams& p, int fp16, cudaStream_t stream) {
  if (p.signs) return fp16 ? launch_t<D, FORMAT, true, true>(p, stream) : launch_t<D, FORMAT, false, true>(p, stream);
  return fp16 ? launch_t<D, FORMAT, true, false>(p, stream) : launch_t<D, FORMAT, false, false>(p, stream);
}

}  // namespace

attn_status_t launch_cache_read(CacheReadParams p, int format_bits, int d, int fp16, cudaStream_t stream) {
  p.status = device_status_word();
  if (!p.status) return fail(ATTN_ERR_CUDA, "status word unavailable");
  // (a packed read's grid has no dimension for the requests)
  if (2LL * p.H_kv > 65535 || (p.cu_seqlens == nullptr && p.B > 65535))
    return fail(ATTN_ERR_UNSUPPORTED, "H_kv must be <= 32767, and B <= 65535 where the output is padded");
  p.page_shift = page_shift_of(p.page_size);
  if (format_bits == 4) return d == 64 ? launch_f<64, k4>(p, fp16, stream) : launch_f<128, k4>(p, fp16, stream);
  if (format_bits == 8) return launch_f<128, k8>(p, fp16, stream);
  return d == 64    ? launch_t<64, k16, false, false>(p, stream)      // moves bits: either type
         : d == 128 ? launch_t<128, k16, false, false>(p, stream)
                    : launch_t<256, k16, false, false>(p, stream);
}

}  // namespace attn
