// gdn_rotary.cuh -- the angle of a rotary pair.
//
// A position's angle is p f radians with p up to a million and f near 1: in f32 the product is off by
// 0.06.  Counted in turns, modulo one, it is a fixed-point fraction: the frequency in units of 2^-64
// turns times the position, modulo 2^64, is exact.  Its upper 32 bits, as a signed number, are the turn
// in [-1/2, 1/2) to 2^-32, whose sine and cosine f32 gives to a few units.
#pragma once

#include "gdn_internal.h"

namespace gdn {

// (cos, sin) of position pos at `turns`, times scale.
__device__ __forceinline__ float2 rotary_turn(uint64_t turns, int pos, float scale) {
  const uint64_t t = turns * (uint64_t)(int64_t)pos;
  float s, c;
  sincospif((float)(int32_t)(t >> 32) * 0x1p-31f, &s, &c);
  return make_float2(c * scale, s * scale);
}

// (a, b) turned: the same two roundings in every kernel.
__device__ __forceinline__ float turned_a(float a, float b, float c, float s) { return fmaf(a, c, -__fmul_rn(b, s)); }
__device__ __forceinline__ float turned_b(float a, float b, float c, float s) { return fmaf(b, c, __fmul_rn(a, s)); }

}  // namespace gdn
