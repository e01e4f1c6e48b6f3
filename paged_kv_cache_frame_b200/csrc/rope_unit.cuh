// One unit of a rotated head: two packs of V values, V pairs. Neighbouring
// pairs (2i, 2i + 1) of unit u fill values [2uV, 2uV + 2V); pairs
// (i, i + rot / 2) lie in the packs at uV and uV + rot / 2, and the units
// behind the rotated part copy two packs each. Pairs at or past rot / 2 of
// the neighbouring layout are copied too.
//
// A block works the angles of its tokens out once, a thread a pair, into
// shared memory: every head of a token takes them from there.
#pragma once
#include "rope.cuh"
#include "token_access.cuh"

namespace pkv {

// Angle table of a block: [tokens][units][V] (cos, sin), laid out so that
// neighbouring units' 16 bytes lie next to each other.
template <int V>
__host__ __device__ constexpr int angle_at(int units, int token, int pair) {
  return V == 1 ? token * units + pair
                : token * units * V + (pair % V / 2 * units + pair / V) * 2 + pair % 2;
}

template <typename T, int V, bool kInter>
struct RopeUnit {
  using P = Pack<T, V>;
  int u;
  int at0, at1;        // first value of each pack
  bool turns;          // any pair of the unit is rotated
  bool second;         // the second pack lies inside the head

  // Unit u of a head of D values.
  __device__ __forceinline__ RopeUnit(int unit, int D, int rot) : u(unit) {
    if (kInter) {
      at0 = 2 * u * V;
      at1 = at0 + V;
      turns = at0 < rot;
    } else {
      turns = u * V < rot / 2;
      at0 = turns ? u * V : rot + 2 * (u * V - rot / 2);
      at1 = turns ? at0 + rot / 2 : at0 + V;
    }
    second = at1 < D;
  }

  // Rotates the packs by the angles of the block's token `token`.
  __device__ __forceinline__ void turn(P& x0, P& x1, const float2* table, int units, int token, int rot) const {
    float2 cs[V];
    if constexpr (V == 1) {
      cs[0] = table[angle_at<V>(units, token, u)];
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const float4 x = *reinterpret_cast<const float4*>(table + angle_at<V>(units, token, u * V + i));
        cs[i] = make_float2(x.x, x.y);
        cs[i + 1] = make_float2(x.z, x.w);
      }
    }
    if constexpr (V == 1) {
      float a = x0.get(0), b = x1.get(0);
      rope_turn(a, b, cs[0].x, cs[0].y);
      x0.set(a);
      x1.set(b);
    } else if constexpr (kInter) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        P& x = i < V / 2 ? x0 : x1;
        const int j = i % (V / 2);
        float a = x.get(2 * j), b = x.get(2 * j + 1);
        rope_turn(a, b, cs[i].x, cs[i].y);
        if (u * V + i < rot / 2) x.set2(j, a, b);   // the others keep their bits
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        float a = x0.get(i), b = x1.get(i), c = x0.get(i + 1), d = x1.get(i + 1);
        rope_turn(a, b, cs[i].x, cs[i].y);
        rope_turn(c, d, cs[i + 1].x, cs[i + 1].y);
        x0.set2(i / 2, a, c);
        x1.set2(i / 2, b, d);
      }
    }
  }
};

constexpr int kSms = 148;   // of a B200: sizes of blocks count on them, results do not

// Tokens a block takes: enough heads per thread to hide the angles, as long
// as every SM still gets two blocks.
inline int rope_tokens_per_block(int n_tokens, int heads, int units, int threads, int most) {
  int n = 1;
  while (2 * n <= most && 2LL * n * heads * units <= 8LL * threads && n_tokens / (2 * n) >= 2 * kSms) n *= 2;
  return n;
}

}  // namespace pkv
