// Device side of rotary positions: the angle of a (position, pair) and the
// rotation of a pair.
#pragma once
#include "rope.h"

namespace pkv {

// cos and sin of `pos` times a table entry, times the amplitude. The product
// modulo 2^64 is the angle modulo a turn; its top 32 bits, rounded, are a
// signed fraction in [-1/2, 1/2) of a turn, which sincospif takes in half
// turns. Rounding to 2^-32 of a turn and then to a float's 24 bits leaves at
// most pi * 2^-24 radians, below the 32-bit products that follow.
__device__ __forceinline__ void rope_angle(uint64_t turn, int32_t pos, float amplitude, float& c, float& s) {
  const uint64_t phase = turn * (uint64_t)(int64_t)pos + 0x80000000ull;
  const float half_turns = (float)(int32_t)(uint32_t)(phase >> 32) * 4.656612873077392578125e-10f;   // 2^-31
  sincospif(half_turns, &s, &c);
  c *= amplitude;
  s *= amplitude;
}

__device__ __forceinline__ void rope_turn(float& a, float& b, float c, float s) {
  const float x = a * c - b * s;
  b = b * c + a * s;
  a = x;
}

}  // namespace pkv
