// Rotary position embedding: the rotation of Q and K rows, and the tables of
// cosines and sines it reads, stretched for long contexts.
//
// "FlashAttention-3: Hopper Asynchrony and FP8 Attention", section "FP8 accuracy
// controls", fuses the rotation with the Hadamard transform of the FP8 pre-pass
// (fp8.cu) and leaves its definition to the caller's tables; this is the same
// rotation for the 16-bit kernels, forward and inverse.
#include <cmath>

#include "common.h"
#include "rope.cuh"

namespace attn {
namespace {

constexpr double kTwoPi = 6.283185307179586476925;

// PER_SM: blocks that an SM is to hold.  Three (80 registers, a few spilled; three or two
// heads at a time need none and are slower) where there are more than 2 x 152 blocks: 53.8
// -> 52.3 us for 2 x 8192 tokens of 40 heads, d = 128; two (102) otherwise, for a step of 64
// requests 2.8 us, 3.0 with three.
template <bool FP16, bool INTERLEAVED, int PER_SM>
__global__ void __launch_bounds__(kRopeThreads, PER_SM) rope_kernel(const RopeKParams p) {
  wait_for_previous_kernel();      // a dependent launch: its start overlaps that one's end
  rope_block<FP16, INTERLEAVED, true>(p, blockIdx.x, blockIdx.y);
}

// Table row r holds position p = first + r.  Frequency theta_i = base^(-2i/rot)
// makes r_i = orig_len * theta_i / (2 pi) turns within the original context; it
// is kept where r_i >= high, divided by `factor` where r_i <= low, and blended
// linearly in r_i between (interpolation "by parts", section 3.2 of "YaRN:
// Efficient Context Window Extension of Large Language Models",
// arXiv:2309.00071); orig_len = 0 divides every frequency (position
// interpolation, arXiv:2306.15595).
//
// The angle p * theta reaches 1e6 rad, where a float32 angle would be off by
// 0.06, and float64 arithmetic runs at 1/64 of the float32 rate here.  So the
// frequency is held in turns per position as a 64-bit binary fraction F, which the
// host computes in float64 (at most 128 of them, passed by value): the product
// p * F modulo 2^64 is the angle modulo one turn, exactly, in integers.  Its upper
// 32 bits, as a signed number of half turns, are what sincospif takes.  F is off by
// at most 2^-53 of itself, the cut to 32 bits by 2^-33 of a turn, and the conversion
// to float32, the largest of the three, by 2^-26 of a turn (9.4e-8 rad).
//
// A thread owns a column.  Every eighth of its rows takes the sine and cosine of its
// own angle: off by that and half a step or two of the functions, 2^-22.5 in all.  The
// seven behind it take the sum formulas with those of 1 .. 7 row steps, computed once
// per thread: both angles' errors (1.9e-7 together), four entries' function errors
// (2 sqrt(2) 2^-24) and two roundings (2^-25 each): 2^-21.2.  (Of two million random
// pairs of angles, with exact functions: 2^-22 at most, 5e-8 rms.)
// Bound: the writes, 8 bytes per entry.  131072 x 64 entries: 238 us with float64
// angles, 17.4 us with a sine and cosine per entry, 12.2 us so (5.5 TB/s).
struct RopeTurns {
  unsigned long long f[128];
};

// cos and sin of an angle in turns, as a 64-bit binary fraction.
__device__ __forceinline__ float2 cos_sin_turns(unsigned long long angle) {
  // the nearest multiple of 2^-32 turns, as half turns in [-1, 1)
  const int half_turns = static_cast<int>((angle + 0x80000000ull) >> 32);
  float sn, cs;
  sincospif(static_cast<float>(half_turns) * 4.656612873077392578125e-10f, &sn, &cs);
  return make_float2(cs, sn);
}

__global__ void __launch_bounds__(256)
    rope_table_kernel(float* __restrict__ cos_out, float* __restrict__ sin_out, long long n, int half,
                      const __grid_constant__ RopeTurns turns, float attn_factor, unsigned first,
                      int rows_per_block) {
  constexpr int kRun = 8;
  const int lanes = 256 / half;                     // rows written at a time
  const int i = static_cast<int>(threadIdx.x) % half;
  const int sub = static_cast<int>(threadIdx.x) / half;
  if (sub >= lanes) {
    wait_for_previous_kernel();
    return;
  }
  const unsigned long long f = turns.f[i];
  const long long r0 = static_cast<long long>(blockIdx.x) * rows_per_block;
  const long long r1 = r0 + rows_per_block < n ? r0 + rows_per_block : n;
  const unsigned long long step = f * lanes;
  float2 by[kRun];
#pragma unroll
  for (int k = 1; k < kRun; ++k) by[k] = cos_sin_turns(step * k);
  unsigned long long angle = f * (static_cast<unsigned long long>(first) + r0 + sub);
  wait_for_previous_kernel();      // a dependent launch: it may still be reading the tables' memory
  for (long long r = r0 + sub; r < r1; r += kRun * lanes, angle += step * kRun) {
    float2 b = cos_sin_turns(angle);
    b = make_float2(b.x * attn_factor, b.y * attn_factor);
    float* c = cos_out + r * half + i;
    float* s = sin_out + r * half + i;
    *c = b.x;
    *s = b.y;
#pragma unroll
    for (int k = 1; k < kRun; ++k) {
      if (r + k * lanes >= r1) break;
      c[k * lanes * half] = fmaf(-b.y, by[k].y, b.x * by[k].x);
      s[k * lanes * half] = fmaf(b.x, by[k].y, b.y * by[k].x);
    }
  }
}

}  // namespace

attn_status_t launch_rope(RopeKParams p, int fp16, int interleaved, cudaStream_t stream) {
  p.status = device_status_word();
  if (!p.status) return fail(ATTN_ERR_CUDA, "status word unavailable");
  const RopeGrid g = rope_grid(&p);
  if (g.columns > 2147483647LL || g.chunks > 65535)
    return fail(ATTN_ERR_UNSUPPORTED, "grid dimension limit exceeded");
  const dim3 grid(static_cast<unsigned>(g.columns), g.chunks);
  const bool many = g.columns * g.chunks > 2 * 152;
  auto pick = [&](auto three, auto two) { return many ? three : two; };
  auto kern = fp16 ? interleaved ? pick(rope_kernel<true, true, 3>, rope_kernel<true, true, 2>)
                                 : pick(rope_kernel<true, false, 3>, rope_kernel<true, false, 2>)
                   : interleaved ? pick(rope_kernel<false, true, 3>, rope_kernel<false, true, 2>)
                                 : pick(rope_kernel<false, false, 3>, rope_kernel<false, false, 2>);
  const cudaError_t e = launch_dependent(kern, grid, kRopeThreads, 0, stream, 0, p);
  if (e != cudaSuccess) return fail_cuda(e, "rotary kernel launch");
  return ATTN_OK;
}

attn_status_t launch_rope_table(float* cos_out, float* sin_out, long long n, int rot, double base,
                                double factor, long long orig_len, double low, double high,
                                double attn_factor, long long first, cudaStream_t stream) {
  const int half = rot / 2;
  RopeTurns turns;
  for (int i = 0; i < half; ++i) {
    double theta = std::pow(base, -static_cast<double>(i) / half);
    double keep = 0.0;
    if (orig_len > 0) {
      keep = (static_cast<double>(orig_len) * theta / kTwoPi - low) / (high - low);
      keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
    }
    theta *= keep + (1.0 - keep) / factor;
    // below 1 / (2 pi) turns per position, times 2^64
    turns.f[i] = static_cast<unsigned long long>(std::ldexp(theta / kTwoPi, 64));
  }
  // four blocks per SM, at least 8 rows each
  long long rows = (n + 152 * 4 - 1) / (152 * 4);
  rows = rows < 8 ? 8 : rows;
  const long long blocks = (n + rows - 1) / rows;
  const cudaError_t e = launch_dependent(rope_table_kernel, dim3(static_cast<unsigned>(blocks)), 256, 0, stream, 0,
                                         cos_out, sin_out, n, half, turns, static_cast<float>(attn_factor),
                                         static_cast<unsigned>(first), static_cast<int>(rows));
  if (e != cudaSuccess) return fail_cuda(e, "rotary table launch");
  return ATTN_OK;
}

}  // namespace attn
