// Rotary positions: the frequency table of a kv_rope_t and its host-side
// construction. Plain C++17, no CUDA.
//
// Pair i of a token at position p turns by p * theta_i radians. The table
// holds theta_i / (2 pi) as a 64-bit binary fraction of a turn, so p times
// the entry modulo 2^64 is the angle modulo a whole turn, exactly: the range
// reduction of a far position is one integer product and loses nothing. (In
// 32-bit floats p * theta_i is off by p * 2^-24 radians, 0.06 at a position
// of a million.) The entry itself is within 2^-64 of a turn for theta_i up to
// 1 (2^-61 up to 64, the largest), which a position of 2^31 makes 2^-33
// (2^-30).
#pragma once
#include <stdint.h>

#include <string>

namespace pkv {

constexpr int kMaxRot = 256;   // largest rot_dim

// Travels in the kernel parameters, so a rope handle needs no device memory.
struct RopeTable {
  uint64_t turn[kMaxRot / 2];   // theta_i / (2 pi), in units of 2^-64 turns
  float amplitude;              // factor on the rotated values
  int32_t rot;                  // leading values of a head that are rotated (0: none)
  int32_t interleaved;          // pairs (2i, 2i + 1) instead of (i, i + rot / 2)
};

struct RopeSpec {
  int rot_dim, layout, scaling;
  double base, factor, original_context, low_turns, high_turns, amplitude;
};

// theta_0 .. theta_{rot_dim/2 - 1} of a spec into `theta`, and its amplitude
// (spec.amplitude, or the scaling's own for 0). KV_OK or KV_ERR_ARG, with
// `why`.
int rope_frequencies(const RopeSpec& s, double* theta, double* amplitude, std::string* why);
// The table of given frequencies.
int rope_table(int rot_dim, int layout, const double* theta, double amplitude, RopeTable* out, std::string* why);

}  // namespace pkv

struct kv_rope {
  pkv::RopeTable table;
  double theta[pkv::kMaxRot / 2];
  double amplitude;
  int layout;
};
