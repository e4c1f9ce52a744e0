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

template <bool FP16>
__device__ __forceinline__ uint4 pack16(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = FP16 ? cvt_pack_f16(x[2 * i], x[2 * i + 1]) : cvt_pack_bf16(x[2 * i], x[2 * i + 1]);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Work of one block: tokens of block column `bx`, heads of chunk `chunk`, kHeads of
// them at a time.
template <bool FP16, bool INTERLEAVED, int kHeads = 4>
__device__ __forceinline__ void rope_block(const RopeKParams& p, long long bx, int chunk) {
  const int units = p.d / 16;                       // 4, 8 or 16: divides the block
  const int tokens = static_cast<int>(blockDim.x) / units;
  const int u = static_cast<int>(threadIdx.x) % units;
  const long long tk = bx * tokens + static_cast<int>(threadIdx.x) / units;
  if (tk >= static_cast<long long>(p.B) * p.N) return;
  const long long b = tk / p.N, n = tk - b * p.N;
  bool turn = p.rotated > 0 && 16 * u < p.rot;
  float c[8], s[8];
  if (p.rotated > 0) {
    int pos = static_cast<int>(n);
    if (p.positions) {
      pos = p.positions[tk];
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
        const float4 cv = __ldg(reinterpret_cast<const float4*>(p.cos + at) + i);
        const float4 sv = __ldg(reinterpret_cast<const float4*>(p.sin + at) + i);
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
    slot = p.slots[n];
    if (slot >= p.num_slots || slot < -1) {
      if (u == 0 && chunk == 0) atomicCAS(p.status, 0, kDevBadTables);
      slot = -1;
    }
  }
  // columns of the thread's two vectors
  const bool halves = !INTERLEAVED && p.rotated > 0 && 16 * u < p.rot;
  const int off_a = halves ? 8 * u : 16 * u;
  const int off_b = halves ? p.rot / 2 + 8 * u : 16 * u + 8;
  const int all = p.heads[0] + p.heads[1] + p.heads[2];
  const int h_end = min(all, (chunk + 1) * p.heads_per_chunk);
  for (int h0 = chunk * p.heads_per_chunk; h0 < h_end; h0 += kHeads) {
    uint4 va[kHeads], vb[kHeads];
    uint16_t* out[kHeads];
    bool rot[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      out[i] = nullptr;
      int h = h0 + i;
      if (h >= h_end) continue;
      int t = 0;
      if (h >= p.heads[0]) {
        h -= p.heads[0];
        t = 1;
        if (h >= p.heads[1]) {
          h -= p.heads[1];
          t = 2;
        }
      }
      rot[i] = turn && t < p.rotated;
      // selects, not indexed parameter arrays: t is only known at run time
      const uint16_t* src = t == 0 ? p.src[0] : t == 1 ? p.src[1] : p.src[2];
      uint16_t* dst = t == 0 ? p.dst[0] : t == 1 ? p.dst[1] : p.dst[2];
      const long long sb = t == 0 ? p.sb[0] : t == 1 ? p.sb[1] : p.sb[2];
      const long long sh = t == 0 ? p.sh[0] : t == 1 ? p.sh[1] : p.sh[2];
      const long long st = t == 0 ? p.st[0] : t == 1 ? p.st[1] : p.st[2];
      if (p.slots && t > 0) {
        if (slot < 0) continue;
        out[i] = dst + (slot * p.heads[1] + h) * p.d;
      } else {
        const long long db = t == 0 ? p.db[0] : p.db[1];
        const long long dh = t == 0 ? p.dh[0] : p.dh[1];
        const long long dt = t == 0 ? p.dt[0] : p.dt[1];
        out[i] = dst + b * db + h * dh + n * dt;
      }
      const uint16_t* in = src + b * sb + h * sh + n * st;
      va[i] = *reinterpret_cast<const uint4*>(in + off_a);
      vb[i] = *reinterpret_cast<const uint4*>(in + off_b);
    }
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      if (!out[i]) continue;
      if (rot[i]) {
        float x[8], y[8];
        unpack16<FP16>(va[i], x);
        unpack16<FP16>(vb[i], y);
        if (INTERLEAVED) {
          // x: pairs 0 .. 3, y: pairs 4 .. 7 of the thread's eight
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x0 = x[2 * e], x1 = x[2 * e + 1], y0 = y[2 * e], y1 = y[2 * e + 1];
            x[2 * e] = fmaf(-x1, s[e], x0 * c[e]);
            x[2 * e + 1] = fmaf(x0, s[e], x1 * c[e]);
            y[2 * e] = fmaf(-y1, s[4 + e], y0 * c[4 + e]);
            y[2 * e + 1] = fmaf(y0, s[4 + e], y1 * c[4 + e]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float x0 = x[e], y0 = y[e];
            x[e] = fmaf(-y0, s[e], x0 * c[e]);
            y[e] = fmaf(x0, s[e], y0 * c[e]);
          }
        }
        va[i] = pack16<FP16>(x);
        vb[i] = pack16<FP16>(y);
      }
      *reinterpret_cast<uint4*>(out[i] + off_a) = va[i];
      *reinterpret_cast<uint4*>(out[i] + off_b) = vb[i];
    }
  }
}

// Blocks of rope_block: token columns, and head chunks so that a call of few
// tokens still fills the machine.
struct RopeGrid {
  long long columns;
  int chunks;
};
inline RopeGrid rope_grid(RopeKParams* p, int threads = kRopeThreads) {
  const int tokens = threads / (p->d / 16);
  RopeGrid g;
  g.columns = (static_cast<long long>(p->B) * p->N + tokens - 1) / tokens;
  const int all = p->heads[0] + p->heads[1] + p->heads[2];
  int per = all;
  while (per > 4 && g.columns * ((all + per - 1) / per) < 152 * 8) per = (per + 1) / 2;
  p->heads_per_chunk = per;
  g.chunks = (all + per - 1) / per;
  return g;
}

}  // namespace attn
