// A head's channels over lanes, and the angles of its rotated pairs.
//
// A head of D channels belongs to D / 16 lanes, each with two runs of 8
// channels (16-byte loads in bf16), a and b, laid out so that both members of
// a rotated pair are the same lane's: with pairs (i, i + R / 2) the first
// R / 16 lanes hold 8 l .. and R / 2 + 8 l .., the others the two halves of the
// channels behind R in the same way; with pairs (2 i, 2 i + 1) the runs are
// 8 l .. and D / 2 + 8 l ...  So the rotation moves nothing between lanes, a lane
// needs the sines of 8 pairs at most, and neighbouring lanes' loads join.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_internal.h"

namespace kda {

template <int D, bool INTER>
struct HeadRuns {
  int a, b;            // first channels of the two runs
  bool turn_a, turn_b; // whether their pairs are rotated (the same unless INTER)

  __device__ __forceinline__ HeadRuns(int lane, int R) {
    if constexpr (INTER) {
      a = 8 * lane;
      b = D / 2 + 8 * lane;
      turn_a = a < R;
      turn_b = b < R;
    } else {
      const int first = R >> 4;
      turn_a = turn_b = lane < first;
      a = turn_a ? 8 * lane : R + 8 * (lane - first);
      b = turn_a ? (R >> 1) + 8 * lane : R + ((D - R) >> 1) + 8 * (lane - first);
    }
  }
  // The pair that sine e of a lane belongs to.
  __device__ __forceinline__ int pair(int e) const {
    if constexpr (INTER) return e < 4 ? (a >> 1) + e : (b >> 1) + e - 4;
    else return a + e;
  }
  __device__ __forceinline__ bool turned(int e) const { return INTER && e >= 4 ? turn_b : turn_a; }
};

// A lane's 8 pairs: turns per position in 64 bits, and their axes, two bits each.
struct PairRates {
  double rate[8];
  uint32_t axes;
};

constexpr double kPerTurn = 0.15915494309189533577;   // 1 / (2 pi)

// (Every load is made, of pair 0 where a lane turns nothing, so that none waits
// for another: under conditions these 16 took 10 us of a small call.)
template <int D, bool INTER>
__device__ __forceinline__ PairRates pair_rates(const RopeArgs& r, const HeadRuns<D, INTER>& runs) {
  PairRates p = {};
  if (r.rotary_dim == 0) return p;
  float f[8];
  int ax[8] = {};
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = r.inv_freq[runs.turned(e) ? runs.pair(e) : 0];
  if (r.axis) {
#pragma unroll
    for (int e = 0; e < 8; ++e) ax[e] = r.axis[runs.turned(e) ? runs.pair(e) : 0];
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    p.rate[e] = runs.turned(e) ? static_cast<double>(f[e]) * kPerTurn : 0.0;
    p.axes |= static_cast<uint32_t>(ax[e] < 0 ? 0 : ax[e] >= r.num_axes ? r.num_axes - 1 : ax[e]) << (2 * e);
  }
  return p;
}

// The token's positions on every axis.  (Four scalars: an array that is indexed
// at run time goes to LDS, whose address then takes the workgroup's size from
// the dispatch packet in host memory, which cost 8 us of a small call.)
struct Places {
  int32_t x0, x1, x2, x3;

  __device__ __forceinline__ Places(const RopeArgs& r, int64_t token) {
    const int32_t* p = r.positions + token;
    x0 = p[0];
    x1 = p[r.num_axes > 1 ? r.n_tokens : 0];
    x2 = p[r.num_axes > 2 ? 2 * r.n_tokens : 0];
    x3 = p[r.num_axes > 3 ? 3 * r.n_tokens : 0];
  }
  __device__ __forceinline__ explicit Places(int32_t everywhere) : x0(everywhere), x1(everywhere), x2(everywhere), x3(everywhere) {}
  __device__ __forceinline__ int32_t on(uint32_t axis) const {
    const int32_t lo = axis & 1 ? x1 : x0, hi = axis & 1 ? x3 : x2;
    return axis & 2 ? hi : lo;
  }
};

// Pair e's angle at the token, in turns within half a turn.  Three roundings in 64
// bits, of 1 / (2 pi), of the rate and of its product with the position: together
// within 1e-10 turns at position 10^6.
__device__ __forceinline__ double turns(double rate, int32_t position) {
  const double t = static_cast<double>(position) * rate;
  return t - rint(t);
}
__device__ __forceinline__ double turns(const PairRates& p, const Places& at, int e) {
  return turns(p.rate[e], at.on((p.axes >> (2 * e)) & 3));
}

// Sine and cosine of t turns, |t| <= 1/2, to fp32's rounding also next to 0: to the
// nearest quarter turn, then the Taylor series within an eighth in 64 bits (the
// terms left out are below 2e-10 of the result).
__device__ __forceinline__ void sincos_turns32(double t, float& s, float& c) {
  const double q = rint(4.0 * t);
  const double x = (t - 0.25 * q) * 6.283185307179586476925;
  const double z = x * x;
  double a = -1.0 / 39916800.0;                 // 1 / 11!
  a = fma(a, z, 1.0 / 362880.0);
  a = fma(a, z, -1.0 / 5040.0);
  a = fma(a, z, 1.0 / 120.0);
  a = fma(a, z, -1.0 / 6.0);
  a = fma(a * z, x, x);
  double b = -1.0 / 3628800.0;                  // 1 / 10!
  b = fma(b, z, 1.0 / 40320.0);
  b = fma(b, z, -1.0 / 720.0);
  b = fma(b, z, 1.0 / 24.0);
  b = fma(b, z, -0.5);
  b = fma(b, z, 1.0);
  const int n = static_cast<int>(q) & 3;
  const float u = static_cast<float>(n & 1 ? b : a), v = static_cast<float>(n & 1 ? a : b);
  s = n & 2 ? -u : u;
  c = (n + 1) & 2 ? -v : v;
}

// (a, b) rotated by the pairs' sines: the runs of one lane, T float or double.
template <int D, bool INTER, class T>
__device__ __forceinline__ void rotate(const HeadRuns<D, INTER>& runs, T (&a)[8], T (&b)[8], const T (&c)[8],
                                       const T (&s)[8]) {
  if constexpr (INTER) {
    if (runs.turn_a) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const T x = a[2 * i], y = a[2 * i + 1];
        a[2 * i] = x * c[i] - y * s[i];
        a[2 * i + 1] = x * s[i] + y * c[i];
      }
    }
    if (runs.turn_b) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const T x = b[2 * i], y = b[2 * i + 1];
        b[2 * i] = x * c[4 + i] - y * s[4 + i];
        b[2 * i + 1] = x * s[4 + i] + y * c[4 + i];
      }
    }
  } else {
    if (runs.turn_a) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const T x = a[i], y = b[i];
        a[i] = x * c[i] - y * s[i];
        b[i] = x * s[i] + y * c[i];
      }
    }
  }
}

}  // namespace kda
