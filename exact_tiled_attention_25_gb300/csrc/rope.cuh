// Rotary rotation of 16-bit rows: the body shared by the rotary kernel and the
// kernels that append rotated keys to a paged cache.
//
// A row of d values holds rot / 2 pairs (rot <= d, both multiples of 16): the
// pair (x_i, x_{i + rot/2}) of the halves layout, or (x_{2i}, x_{2i+1}) of the
// interleaved one, becomes
//   (x c - y s, y c + x s),  c, s = cos[p][i], sin[p][i],  p = position of the row;
// the inverse (the backward pass: the rotation is orthogonal up to the tables'
// common factor, and its gradient is the transpose) takes -s.  Columns rot .. d
// are copied.  Products are formed in float32 and rounded once.
//
// Bound: DRAM traffic, every element read once and written once.  A thread owns
// 16 values of a row (two 16-byte vectors: both members of 8 pairs, in either
// layout with the same 8 table entries) and walks over heads with those entries
// in registers, so the tables are read once per token and head chunk; kHeads
// heads are loaded before the first one is stored, to keep loads in flight.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "rope.h"
#include "sm103_prims.cuh"

namespace attn {

constexpr int kRopeThreads = 256;

template <bool FP16>
__device__ __forceinline__ void unpack16(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (FP16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    } else {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

// Two neighbouring 16-bit values as a float32 pair, and back.
template <bool FP16>
__device__ __forceinline__ uint64_t widen2(uint32_t w) {
  if (FP16) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return pack2(f.x, f.y);
  }
  return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <bool FP16>
__device__ __forceinline__ uint32_t narrow2(uint64_t x) {
  return FP16 ? cvt_pack_f16(lo2(x), hi2(x)) : cvt_pack_bf16(lo2(x), hi2(x));
}

// Eight pairs: (a_i, b_i) of the two vectors, or neighbours within each (a: pairs 0 to
// 3, b: 4 to 7); cc, ss, ns: cos, sin and -sin of pairs (0, 1), (2, 3), ...
template <bool FP16, bool INTERLEAVED>
__device__ __forceinline__ void rotate16(uint4& a, uint4& b, const uint64_t (&cc)[4], const uint64_t (&ss)[4],
                                         const uint64_t (&ns)[4]) {
  uint32_t* wa = reinterpret_cast<uint32_t*>(&a);
  uint32_t* wb = reinterpret_cast<uint32_t*>(&b);
  if constexpr (INTERLEAVED) {
    auto turn = [](uint32_t w, float c, float s) {
      const uint64_t x = widen2<FP16>(w);
      return narrow2<FP16>(pack2(fmaf(-hi2(x), s, lo2(x) * c), fmaf(lo2(x), s, hi2(x) * c)));
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      wa[i] = turn(wa[i], i & 1 ? hi2(cc[i / 2]) : lo2(cc[i / 2]), i & 1 ? hi2(ss[i / 2]) : lo2(ss[i / 2]));
      wb[i] = turn(wb[i], i & 1 ? hi2(cc[2 + i / 2]) : lo2(cc[2 + i / 2]),
                   i & 1 ? hi2(ss[2 + i / 2]) : lo2(ss[2 + i / 2]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t x = widen2<FP16>(wa[i]), y = widen2<FP16>(wb[i]);
      wa[i] = narrow2<FP16>(ffma2(y, ns[i], fmul2(x, cc[i])));
      wb[i] = narrow2<FP16>(ffma2(x, ss[i], fmul2(y, cc[i])));
    }
  }
}

// A load; of a dependent launch (DEPENDENT), which may have started before its inputs were
// written, past the L1 cache.
template <bool DEPENDENT, typename T>
__device__ __forceinline__ T load_input(const T* p) {
  return DEPENDENT ? __ldcg(p) : *p;
}

// Work of one block: tokens of block column `bx`, heads of chunk `chunk`, kHeads of
// them at a time.  SLOTS > 0: rows of the first tensor (no other is given) come through
// shared memory, SLOTS heads in flight, every thread its own 32 bytes of each; for
// kernels that cannot give the loads registers (stage: SLOTS * 2 * blockDim words).
// HL neighbouring heads of a token are rotated at a time, by as many groups of lanes.
template <bool FP16, bool INTERLEAVED, bool DEPENDENT, int kHeads = 4, int SLOTS = 0, int HL = 1>
__device__ __forceinline__ void rope_block(const RopeKParams& p, long long bx, int chunk, uint4* stage = nullptr) {
  const int units = p.d / 16;                       // 4, 8 or 16: divides the block
  const int tokens = static_cast<int>(blockDim.x) / units / HL;
  const int u = static_cast<int>(threadIdx.x) % units;
  const int hsub = HL > 1 ? static_cast<int>(threadIdx.x) / units % HL : 0;
  const long long tk = bx * tokens + static_cast<int>(threadIdx.x) / units / HL;
  if (tk >= static_cast<long long>(p.B) * p.N) return;
  const long long b = tk / p.N, n = tk - b * p.N;
  bool turn = p.rotated > 0 && 16 * u < p.rot;
  float c[8] = {}, s[8] = {};
  if (p.rotated > 0) {
    int pos = static_cast<int>(n);
    if (p.positions) {
      pos = load_input<DEPENDENT>(p.positions + tk);
    } else if (p.cu_seqlens) {
      int lo = 0, hi = p.requests;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.cu_seqlens[mid] <= pos) lo = mid;
        else hi = mid;
      }
      // rows behind the last request are padding
      pos = pos < p.cu_seqlens[lo + 1] ? p.seq_lens[lo] - (p.cu_seqlens[lo + 1] - pos) : -1;
    }
    if (pos < 0 || pos >= p.max_pos) {
      // a negative position marks padding; one past the tables is an error
      if (pos >= p.max_pos && u == 0 && chunk == 0) atomicCAS(p.status, 0, kDevBadTables);
      turn = false;
    }
    if (turn) {
      const size_t at = static_cast<size_t>(pos) * (p.rot / 2) + 8 * u;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 cv = load_input<DEPENDENT>(reinterpret_cast<const float4*>(p.cos + at) + i);
        const float4 sv = load_input<DEPENDENT>(reinterpret_cast<const float4*>(p.sin + at) + i);
        c[4 * i] = cv.x, c[4 * i + 1] = cv.y, c[4 * i + 2] = cv.z, c[4 * i + 3] = cv.w;
        s[4 * i] = sv.x, s[4 * i + 1] = sv.y, s[4 * i + 2] = sv.z, s[4 * i + 3] = sv.w;
      }
      if (p.inverse) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = -s[i];
      }
    }
  }
  long long slot = 0;
  if (p.slots) {
    slot = load_input<DEPENDENT>(p.slots + n);
    if (slot >= p.num_slots || slot < -1) {
      if (u == 0 && chunk == 0) atomicCAS(p.status, 0, kDevBadTables);
      slot = -1;
    }
  }
  // columns of the thread's two vectors
  const bool halves = !INTERLEAVED && p.rotated > 0 && 16 * u < p.rot;
  const int off_a = halves ? 8 * u : 16 * u;
  const int off_b = halves ? p.rot / 2 + 8 * u : 16 * u + 8;
  // cos and sin of the pairs of two neighbouring elements
  uint64_t cc[4], ss[4], ns[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    cc[i] = pack2(c[2 * i], c[2 * i + 1]);
    ss[i] = pack2(s[2 * i], s[2 * i + 1]);
    ns[i] = pack2(-s[2 * i], -s[2 * i + 1]);
  }
  const int lo = chunk * p.heads_per_chunk, hi = lo + p.heads_per_chunk;
  int before = 0;                                   // heads of the tensors before
#pragma unroll
  for (int t = 0; t < 3; ++t) {
    const int h0 = max(lo - before, 0) + hsub, h1 = min(hi - before, p.heads[t]);
    before += p.heads[t];
    if (h0 >= h1 || (p.slots && t > 0 && slot < 0)) continue;
    const int nh = (h1 - h0 + HL - 1) / HL;          // heads h0, h0 + HL, ... of this thread
    const bool rotate = turn && t < p.rotated;
    const uint16_t* in = p.src[t] + b * p.sb[t] + n * p.st[t] + h0 * p.sh[t];
    const bool cache = p.slots && t > 0;
    uint16_t* out = cache ? p.dst[t] + (slot * p.heads[1] + h0) * p.d
                          : p.dst[t] + b * p.db[t] + n * p.dt[t] + h0 * p.dh[t];
    const long long step_in = p.sh[t] * HL, step_out = (cache ? p.d : p.dh[t]) * HL;
    if constexpr (SLOTS > 0) {
      const int words = static_cast<int>(blockDim.x);
      auto copy = [&](int k) {
        if (k < nh) {
          uint4* dst = stage + (k % SLOTS) * 2 * words + threadIdx.x;
          copy16_async(dst, in + k * step_in + off_a, true);
          copy16_async(dst + words, in + k * step_in + off_b, true);
        }
        copies_commit();
      };
#pragma unroll
      for (int k = 0; k < SLOTS; ++k) copy(k);
      for (int k = 0; k < nh; ++k) {
        copies_wait<SLOTS - 1>();
        const uint4* src = stage + (k % SLOTS) * 2 * words + threadIdx.x;
        uint4 va = src[0], vb = src[words];
        if (rotate) rotate16<FP16, INTERLEAVED>(va, vb, cc, ss, ns);
        *reinterpret_cast<uint4*>(out + k * step_out + off_a) = va;
        *reinterpret_cast<uint4*>(out + k * step_out + off_b) = vb;
        copy(k + SLOTS);
      }
      copies_wait<0>();
    } else {
      for (int k = 0; k < nh; k += kHeads) {
        uint4 va[kHeads], vb[kHeads];
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
          if (k + i >= nh) break;
          va[i] = load_input<DEPENDENT>(reinterpret_cast<const uint4*>(in + i * step_in + off_a));
          vb[i] = load_input<DEPENDENT>(reinterpret_cast<const uint4*>(in + i * step_in + off_b));
        }
        in += kHeads * step_in;
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
          if (k + i >= nh) break;
          if (rotate) rotate16<FP16, INTERLEAVED>(va[i], vb[i], cc, ss, ns);
          *reinterpret_cast<uint4*>(out + i * step_out + off_a) = va[i];
          *reinterpret_cast<uint4*>(out + i * step_out + off_b) = vb[i];
        }
        out += kHeads * step_out;
      }
    }
  }
}

// Blocks of rope_block: token columns, and head chunks of at least 4 so that a call of
// few tokens still fills the machine.
struct RopeGrid {
  long long columns;
  int chunks;
};
inline RopeGrid rope_grid(RopeKParams* p, int threads = kRopeThreads, int least_blocks = 152 * 8, int head_lanes = 1) {
  const int tokens = threads / (p->d / 16) / head_lanes;
  RopeGrid g;
  g.columns = (static_cast<long long>(p->B) * p->N + tokens - 1) / tokens;
  const int all = p->heads[0] + p->heads[1] + p->heads[2];
  int per = all;
  while (per > 4 && g.columns * ((all + per - 1) / per) < least_blocks) per = (per + 1) / 2;
  p->heads_per_chunk = per;
  g.chunks = (all + per - 1) / per;
  return g;
}

}  // namespace attn
