// A 128-value row in the lanes of a warp: the Hadamard transform and the e4m3
// quantiser shared by the FP8 pre-pass and the e4m3 cache append.
#pragma once

#include "sm103_prims.cuh"

namespace attn {

// Walsh-Hadamard butterfly (unnormalised) of a 128-value row held by a warp as
// 32 lanes x 4 values, packed as (columns 4 lane, 4 lane + 1) and (4 lane + 2,
// 4 lane + 3): the stages of span 1 and 2 inside the lane, then those of span
// 4 .. 64 across lanes (lane distance 1 .. 16), where the lane with bit m set
// takes partner - own and the other own + partner, both as one fused
// multiply-add by +-1 (exactly the add or the subtract).
__device__ __forceinline__ void wht128_row(uint64_t& p01, uint64_t& p23, int lane) {
  const float a = lo2(p01) + hi2(p01), b = lo2(p01) - hi2(p01);
  const float c = lo2(p23) + hi2(p23), e = lo2(p23) - hi2(p23);
  p01 = pack2(a + c, b + e);
  p23 = pack2(a - c, b - e);
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const float ox = __shfl_xor_sync(0xffffffffu, lo2(p01), m);
    const float oy = __shfl_xor_sync(0xffffffffu, hi2(p01), m);
    const float oz = __shfl_xor_sync(0xffffffffu, lo2(p23), m);
    const float ow = __shfl_xor_sync(0xffffffffu, hi2(p23), m);
    const float sg = (lane & m) ? -1.f : 1.f;
    const uint64_t sg2 = pack2(sg, sg);
    p01 = ffma2(sg2, p01, pack2(ox, oy));
    p23 = ffma2(sg2, p23, pack2(oz, ow));
  }
}

// code = e4m3(x / descale) for four values (two packed pairs), each quotient
// rounded as an IEEE division would: q0 = x y with y = 1 / descale, then
// q0 + (x - descale q0) y (the steps of div_by_recip on packed pairs).
__device__ __forceinline__ uint32_t quantise4(uint64_t x01, uint64_t x23, uint64_t y2, uint64_t nb2) {
  const uint64_t q01 = fmul2(x01, y2), q23 = fmul2(x23, y2);
  const uint64_t c01 = ffma2(ffma2(nb2, q01, x01), y2, q01);
  const uint64_t c23 = ffma2(ffma2(nb2, q23, x23), y2, q23);
  return cvt_pack_e4m3x4(lo2(c01), hi2(c01), lo2(c23), hi2(c23));
}

}  // namespace attn
