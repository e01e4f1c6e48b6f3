// One unit of a rotated head: two packs of V values, V pairs. Neighbouring
// pairs (2i, 2i + 1) of unit u fill values [2uV, 2uV + 2V); pairs
// (i, i + rot / 2) lie in the packs at uV and uV + rot / 2, and the units
// behind the rotated part copy two packs each. Pairs at or past rot / 2 of
// the neighbouring layout are copied too.
#pragma once
#include "rope.cuh"
#include "token_access.cuh"

namespace pkv {

template <typename T, int V, bool kInter>
struct RopeUnit {
  int at0, at1;        // first value of each pack
  bool turns;          // any pair of the unit is rotated
  bool second;         // the second pack lies inside the head
  float c[V], s[V];

  // Unit u of a head of D values. No angle yet.
  __device__ __forceinline__ void place(int u, int D, int rot) {
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

  // The angles of a position, negated for the inverse.
  __device__ __forceinline__ void angles(const RopeTable& t, int u, int32_t pos, bool inverse) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int p = u * V + i;
      if (p < t.rot / 2) {
        rope_angle(t.turn[p], pos, t.amplitude, c[i], s[i]);
        if (inverse) s[i] = -s[i];
      } else {
        c[i] = 1.f;
        s[i] = 0.f;
      }
    }
  }

  __device__ __forceinline__ void turn(const Pack<T, V>& x0, const Pack<T, V>& x1, int u, int rot, Pack<T, V>& y0,
                                       Pack<T, V>& y1) const {
    if (kInter) {
      T x[2 * V], y[2 * V];
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = x0.v[i], x[V + i] = x1.v[i];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float a = to_f32(x[2 * i]), b = to_f32(x[2 * i + 1]);
        rope_turn(a, b, c[i], s[i]);
        const bool on = u * V + i < rot / 2;   // the others keep their bits
        y[2 * i] = on ? from_f32<T>(a) : x[2 * i];
        y[2 * i + 1] = on ? from_f32<T>(b) : x[2 * i + 1];
      }
#pragma unroll
      for (int i = 0; i < V; ++i) y0.v[i] = y[i], y1.v[i] = y[V + i];
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float a = to_f32(x0.v[i]), b = to_f32(x1.v[i]);
        rope_turn(a, b, c[i], s[i]);
        y0.v[i] = from_f32<T>(a);
        y1.v[i] = from_f32<T>(b);
      }
    }
  }
};

}  // namespace pkv
