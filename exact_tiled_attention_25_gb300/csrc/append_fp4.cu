// New keys and values into a 4-bit paged cache: rotation, the key transform and the
// quantiser of fp4.cuh in one pass.
//
// Each row (a token's key or value head) is quantised by itself, so an append only writes
// its own rows: nothing of the page is read, requantised or cleared, and tokens may come in
// any order (slots, as in the 16-bit append).
//
// A page holds its rows head by head, [num_pages, H_kv, page_size, d / 2]: the decode reads
// one head's rows of a page as one run of bytes (interleaved by token, 64-byte rows would
// leave the other half of each 128-byte line to another head).  What that costs here is
// nothing: a row is 64 bytes, two whole sectors, either way.
//
// d / 16 lanes hold a row: lane u the columns 8 u .. 8 u + 7 and d / 2 + 8 u .. (two 16-byte
// loads), so a full-width rotation pairs values of one lane.  The transform's stages run in
// the order of their spans, and the rotation's products are rounded one by one: a code
// depends on which side of a tie a quotient falls, and a fused product would move some 1e-7
// of the codes away from what the same float32 formula gives elsewhere.
#include "common.h"
#include "fp4.cuh"
#include "rope.cuh"

namespace attn {
namespace {

constexpr int kThreads = 128;

enum : int { kPlain = 0, kHalves = 1, kHalvesPart = 2, kNeighbours = 3 };

struct Turn {           // a lane's table entries
  float c[16], s[16];
};

__device__ __forceinline__ float turn_a(float a, float b, float c, float s) {
  return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}
__device__ __forceinline__ float turn_b(float a, float b, float c, float s) {
  return __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

__device__ __forceinline__ void load8(const float* t, float* x) {
  const float4 a = __ldcg(reinterpret_cast<const float4*>(t));
  const float4 b = __ldcg(reinterpret_cast<const float4*>(t) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// The entries that lane u's columns take from table row `row` (entry 0 of it).
template <int D, int MODE>
__device__ __forceinline__ void load_turn(Turn& t, const AppendFp4Params& p, size_t row, int u) {
  if constexpr (MODE == kHalves) {
    load8(p.cos + row + 8 * u, t.c);
    load8(p.sin + row + 8 * u, t.s);
  } else if constexpr (MODE == kHalvesPart) {
    const int nv = p.rot / 16;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int j = u + w * (D / 16);                 // vector of 8 columns
      if (j >= 2 * nv) continue;
      load8(p.cos + row + 8 * (j < nv ? j : j - nv), t.c + 8 * w);
      load8(p.sin + row + 8 * (j < nv ? j : j - nv), t.s + 8 * w);
    }
  } else if constexpr (MODE == kNeighbours) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int col = w * (D / 2) + 8 * u;
      if (col >= p.rot) continue;
      const float4 c = __ldcg(reinterpret_cast<const float4*>(p.cos + row + col / 2));
      const float4 s = __ldcg(reinterpret_cast<const float4*>(p.sin + row + col / 2));
      t.c[4 * w] = c.x, t.c[4 * w + 1] = c.y, t.c[4 * w + 2] = c.z, t.c[4 * w + 3] = c.w;
      t.s[4 * w] = s.x, t.s[4 * w + 1] = s.y, t.s[4 * w + 2] = s.z, t.s[4 * w + 3] = s.w;
    }
  }
}

// Every lane of the warp takes part (shuffles); `turn` false: the row is left unrotated.
template <int D, int MODE>
__device__ __forceinline__ void rotate_row(float (&x)[16], const Turn& t, int rot, bool turn, int u) {
  constexpr int L = D / 16;
  if constexpr (MODE == kHalves) {
    if (!turn) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float a = x[e], b = x[8 + e];
      x[e] = turn_a(a, b, t.c[e], t.s[e]);
      x[8 + e] = turn_b(a, b, t.c[e], t.s[e]);
    }
  } else if constexpr (MODE == kHalvesPart) {
    // vector j (columns 8 j .. 8 j + 7) pairs with vector j +- rot / 16
    const int nv = rot / 16;
    float other[16];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int j = u + w * L;
      const int pj = j < nv ? j + nv : j < 2 * nv ? j - nv : j;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float a = __shfl_sync(0xffffffffu, x[e], pj & (L - 1), L);
        const float b = __shfl_sync(0xffffffffu, x[8 + e], pj & (L - 1), L);
        other[8 * w + e] = pj < L ? a : b;
      }
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int j = u + w * L;
      if (!turn || j >= 2 * nv) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = 8 * w + e;
        x[i] = j < nv ? turn_a(x[i], other[i], t.c[i], t.s[i]) : turn_b(other[i], x[i], t.c[i], t.s[i]);
      }
    }
  } else if constexpr (MODE == kNeighbours) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      if (!turn || w * (D / 2) + 8 * u >= rot) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 8 * w + 2 * e;
        const float a = x[i], b = x[i + 1];
        x[i] = turn_a(a, b, t.c[4 * w + e], t.s[4 * w + e]);
        x[i + 1] = turn_b(a, b, t.c[4 * w + e], t.s[4 * w + e]);
      }
    }
  }
}

// x -> (x o signs) H_d / sqrt(d), stages by span: 1, 2, 4 in the lane, 8 .. d / 4 across lanes,
// d / 2 in the lane.  The sums are of x / d, in range for every x, and sqrt(d) comes last; a
// power of two either way, so the bits are those of the plain formula.
template <int D>      // signs_d: signs / d
__device__ __forceinline__ void transform_row(float (&x)[16], const float* signs_d, int u) {
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    const float4 s = *reinterpret_cast<const float4*>(signs_d + (i < 8 ? 0 : D / 2 - 8) + 8 * u + i);
    x[i] *= s.x, x[i + 1] *= s.y, x[i + 2] *= s.z, x[i + 3] *= s.w;
  }
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
  for (int i = 0; i < 8; ++i) {
    const float a = x[i], b = x[8 + i];
    x[i] = (a + b) * root;
    x[8 + i] = (a - b) * root;
  }
}

// One block: kThreads / (d / 16) tokens, heads [chunk * per, + per) of the keys or of the
// values.  Bound: DRAM (the rows read once; a quarter of their bytes written).  16 requests, 14 of one
// token and two with prompts of some 8170, 8 heads and 32 query heads rotated: 62.9 us (5.6 TB/s; 67.3 without
// the next head's row on its way, 66 to 70 with 5, 6 or 8 blocks to an SM instead of 7); 64 single tokens 3.1.
template <int D, bool FP16, int MODE, bool SIGNS>
__device__ __forceinline__ void append_block(const AppendFp4Params& p, long long unit, int per, int chunks) {
  constexpr int L = D / 16;
  const int u = threadIdx.x % L;
  // unit: planes fastest, so that neighbouring blocks are one of keys and one of values
  const bool is_v = unit & 1;
  unit >>= 1;
  const int chunk = static_cast<int>(unit % chunks);
  const long long t = unit / chunks * (kThreads / L) + threadIdx.x / L;
  const bool live = t < p.total;
  long long slot = -1;
  bool turn = false;
  Turn tab;
  if (live) {
    slot = __ldcg(p.slots + t);
    if (slot >= p.num_slots || slot < -1) {
      if (u == 0) atomicCAS(p.status, 0, kDevBadTables);
      slot = -1;
    }
    if (MODE != kPlain && !is_v) {
      const int pos = __ldcg(p.positions + t);
      if (pos >= p.max_pos && u == 0) atomicCAS(p.status, 0, kDevBadTables);
      turn = pos >= 0 && pos < p.max_pos;
      if (turn) load_turn<D, MODE>(tab, p, static_cast<size_t>(pos) * (p.rot / 2), u);
    }
  }
  __shared__ __align__(16) float signs_d[SIGNS ? D : 4];
  if (SIGNS && !is_v) {
    if (threadIdx.x < D / 4) {
      const float4 s = __ldcg(reinterpret_cast<const float4*>(p.signs) + threadIdx.x);
      *reinterpret_cast<float4*>(signs_d + 4 * threadIdx.x) = make_float4(s.x / D, s.y / D, s.z / D, s.w / D);
    }
    __syncthreads();
  }
  const int h0 = chunk * per, h1 = min(h0 + per, p.H_kv);
  const uint16_t* src = static_cast<const uint16_t*>(is_v ? p.v : p.k) + (is_v ? p.vt : p.kt) * (live ? t : 0) + 8 * u;
  const long long sh = is_v ? p.vh : p.kh;
  // slot -> page and row of it; a head's rows of a page are page_size apart
  const long long row0 = (slot >> p.page_shift) * p.H_kv * p.page_size + (slot & (p.page_size - 1));
  uint8_t* const codes = is_v ? p.v_cache : p.k_cache;
  uint16_t* const descale = is_v ? p.v_descale : p.k_descale;
  uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
  auto load = [&](int h) {
    if (live && h < h1) {
      a = __ldcg(reinterpret_cast<const uint4*>(src + sh * h));
      b = __ldcg(reinterpret_cast<const uint4*>(src + sh * h + D / 2));
    }
  };
  load(h0);
  for (int h = h0; h < h1; ++h) {
    float x[16];
    {
      float lo[8], hi[8];
      unpack16<FP16>(a, lo);
      unpack16<FP16>(b, hi);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = lo[i], x[8 + i] = hi[i];
    }
    load(h + 1);
    if (!is_v) {                                       // the same for the whole block
      rotate_row<D, MODE>(x, tab, p.rot, turn, u);
      if constexpr (SIGNS) transform_row<D>(x, signs_d, u);
    }
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int m = L / 2; m > 0; m >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
    const float s = row_descale(top);
    const bool any = s > 0.f;                          // false for 0 and for NaN
    const float y = any ? __fdiv_rn(1.f, s) : 0.f;
    float lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo[i] = any ? div_by_recip(x[i], s, y) : 0.f;
      hi[i] = any ? div_by_recip(x[8 + i], s, y) : 0.f;
    }
    if (slot >= 0) {
      const long long row = row0 + static_cast<long long>(h) * p.page_size;
      uint32_t* dst = reinterpret_cast<uint32_t*>(codes + row * (D / 2));
      dst[u] = e2m1_word(lo);
      dst[L + u] = e2m1_word(hi);
      if (u == 0) descale[row] = static_cast<uint16_t>(__float_as_uint(s) >> 16);
    }
  }
}

// Query rows are rotated by q_blocks other blocks, spread among these (they are bound by
// DRAM, the keys' transform by instructions).
template <int D, bool FP16, int MODE, bool SIGNS>
__global__ void __launch_bounds__(kThreads, 7)
    append_fp4_kernel(const AppendFp4Params p, int per, int chunks, const RopeKParams q, unsigned q_blocks,
                      unsigned q_columns) {
  wait_for_previous_kernel();      // a dependent launch: it reads past the L1 cache
  const unsigned before_q = static_cast<unsigned>(static_cast<unsigned long long>(blockIdx.x) * q_blocks / gridDim.x);
  const unsigned with_q = static_cast<unsigned>((blockIdx.x + 1ull) * q_blocks / gridDim.x);
  if constexpr (MODE != kPlain) {
    if (with_q > before_q) {
      rope_block<FP16, MODE == kNeighbours, true, 2>(q, before_q % q_columns, before_q / q_columns);
      return;
    }
  }
  append_block<D, FP16, MODE, SIGNS>(p, blockIdx.x - before_q, per, chunks);
}

template <int D, bool FP16, int MODE, bool SIGNS>
attn_status_t launch_t(const AppendFp4Params& p, RopeKParams q, cudaStream_t stream) {
  q.status = p.status;
  constexpr int tokens = kThreads / (D / 16);
  const long long columns = (static_cast<long long>(p.total) + tokens - 1) / tokens;
  // heads per block: all of a token's share its table entries, as long as the machine is
  // filled (152 x 8 blocks; an SM holds 7 at a time)
  int per = p.H_kv;
  while (per > 1 && columns * 2 * ((p.H_kv + per - 1) / per) < 152 * 8) per = (per + 1) / 2;
  const int chunks = (p.H_kv + per - 1) / per;
  RopeGrid g{1, 0};
  if (q.heads[0] > 0) g = rope_grid(&q, kThreads);
  const long long q_blocks = g.columns * g.chunks, own = columns * 2 * chunks;
  if (own + q_blocks > 2147483647LL) return fail(ATTN_ERR_UNSUPPORTED, "grid dimension limit exceeded");
  const cudaError_t e = launch_dependent(append_fp4_kernel<D, FP16, MODE, SIGNS>,
                                         dim3(static_cast<unsigned>(own + q_blocks)), kThreads, 0, stream, 0, p, per,
                                         chunks, q, static_cast<unsigned>(q_blocks), static_cast<unsigned>(g.columns));
  return e == cudaSuccess ? ATTN_OK : fail_cuda(e, "4-bit append kernel launch");
}

template <int D, bool FP16>
attn_status_t launch_d(const AppendFp4Params& p, const RopeKParams& q, int interleaved, cudaStream_t stream) {
  const bool sg = p.signs != nullptr;
#define ATTN_APPEND4(MODE) \
  return sg ? launch_t<D, FP16, MODE, true>(p, q, stream) : launch_t<D, FP16, MODE, false>(p, q, stream)
  if (!p.cos) ATTN_APPEND4(kPlain);
  if (interleaved) ATTN_APPEND4(kNeighbours);
  if (p.rot == D) ATTN_APPEND4(kHalves);
  ATTN_APPEND4(kHalvesPart);
#undef ATTN_APPEND4
}

}  // namespace

attn_status_t launch_append_fp4(AppendFp4Params p, const RopeKParams& q, int d, int fp16, int interleaved,
                                cudaStream_t stream) {
  p.status = device_status_word();
  if (!p.status) return fail(ATTN_ERR_CUDA, "status word unavailable");
  p.page_shift = page_shift_of(p.page_size);
  p.num_slots = static_cast<long long>(p.num_pages) * p.page_size;
  if (d == 64)
    return fp16 ? launch_d<64, true>(p, q, interleaved, stream) : launch_d<64, false>(p, q, interleaved, stream);
  return fp16 ? launch_d<128, true>(p, q, interleaved, stream) : launch_d<128, false>(p, q, interleaved, stream);
}

}  // namespace attn
