#include "rope.h"

#include <cmath>
#include <cstring>

#include "../../include/kv.h"

namespace pkv {

static int bad(std::string* why, const char* s) {
  *why = s;
  return KV_ERR_ARG;
}

static int check_shape(int rot_dim, int layout, std::string* why) {
  if (rot_dim < 2 || rot_dim > kMaxRot || rot_dim % 2 != 0) return bad(why, "rope: rot_dim must be even, 2..256");
  if (layout != KV_ROPE_HALF && layout != KV_ROPE_INTERLEAVED) return bad(why, "rope: unknown layout");
  return KV_OK;
}

int rope_frequencies(const RopeSpec& s, double* theta, double* amplitude, std::string* why) {
  const int rc = check_shape(s.rot_dim, s.layout, why);
  if (rc != KV_OK) return rc;
  if (!std::isfinite(s.base) || s.base <= 0) return bad(why, "rope: base must be positive");
  if (!std::isfinite(s.factor) || s.factor <= 0) return bad(why, "rope: factor must be positive");
  if (!std::isfinite(s.amplitude) || s.amplitude < 0) return bad(why, "rope: amplitude < 0");
  if (s.scaling == KV_ROPE_YARN) {
    if (!std::isfinite(s.original_context) || s.original_context <= 0)
      return bad(why, "rope: yarn scaling needs original_context > 0");
    if (!std::isfinite(s.low_turns) || !std::isfinite(s.high_turns) || s.high_turns <= s.low_turns)
      return bad(why, "rope: yarn scaling needs low_turns < high_turns");
  } else if (s.scaling != KV_ROPE_NONE && s.scaling != KV_ROPE_LINEAR && s.scaling != KV_ROPE_NTK) {
    return bad(why, "rope: unknown scaling");
  }
  const double two_pi = 6.283185307179586476925286766559;
  for (int i = 0; i < s.rot_dim / 2; ++i) {
    double t = std::pow(s.base, -2.0 * i / s.rot_dim);
    if (s.scaling == KV_ROPE_LINEAR) {
      t /= s.factor;
    } else if (s.scaling == KV_ROPE_NTK && i > 0) {
      // base * factor^(rot / (rot - 2)): the last pair turns `factor` times slower, the first one as before
      t *= std::pow(s.factor, -2.0 * i / (s.rot_dim - 2));
    } else if (s.scaling == KV_ROPE_YARN) {
      double keep = (s.original_context * t / two_pi - s.low_turns) / (s.high_turns - s.low_turns);
      keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
      t *= keep + (1 - keep) / s.factor;
    }
    theta[i] = t;
  }
  *amplitude = s.amplitude > 0 ? s.amplitude
               : s.scaling == KV_ROPE_YARN && s.factor > 1 ? 0.1 * std::log(s.factor) + 1
                                                           : 1;
  return KV_OK;
}

int rope_table(int rot_dim, int layout, const double* theta, double amplitude, RopeTable* out, std::string* why) {
  const int rc = check_shape(rot_dim, layout, why);
  if (rc != KV_OK) return rc;
  if (!std::isfinite((float)amplitude) || (float)amplitude <= 0)   // the kernels' own
    return bad(why, "rope: amplitude must be positive, and fit 32 bits");
  std::memset(out, 0, sizeof(*out));
  for (int i = 0; i < rot_dim / 2; ++i) {
    // Up to 64 the quotient's 64-bit mantissa leaves its fraction within
    // 2^-61 of a turn, 2^-30 at a position of 2^31; larger ones would lose
    // what the integer products keep.
    if (!std::isfinite(theta[i]) || std::fabs(theta[i]) > 64.0)
      return bad(why, "rope: a frequency is not finite or above 64 radians a position");
    long double turns = (long double)theta[i] / 6.283185307179586476925286766559005768L;
    turns -= floorl(turns);                                   // [0, 1)
    const long double scaled = turns * 18446744073709551616.0L;   // 2^64
    out->turn[i] = scaled >= 18446744073709551615.0L ? 0 : (uint64_t)scaled;
  }
  out->amplitude = (float)amplitude;
  out->rot = rot_dim;
  out->interleaved = layout == KV_ROPE_INTERLEAVED;
  return KV_OK;
}

}  // namespace pkv
