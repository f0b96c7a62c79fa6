// Runs of consecutive elements between memory and registers: bf16 / fp32
// tensors as floats, and e4m3 rows with their block scales.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "e4m3.h"
#include "kda_device.h"
#include "mfma.h"

namespace kda {

// EPL consecutive io elements (EPL in {1, 2, 4, 8}) at index i of a bf16 or
// fp32 tensor, as floats, with the widest aligned loads.  ONCE: bf16 that no
// one reads again soon (a non-temporal load).
template <bool BF16, int EPL, bool ONCE = false>
__device__ __forceinline__ void load_n(const void* p, size_t i, float (&x)[EPL]) {
  if constexpr (BF16) {
    const uint16_t* q = static_cast<const uint16_t*>(p) + i;
    uint32_t w[(EPL + 1) / 2];
    if constexpr (EPL == 8) {
      typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
      const u32x4* from = reinterpret_cast<const u32x4*>(q);
      const u32x4 v = ONCE ? __builtin_nontemporal_load(from) : *from;
      w[0] = v[0]; w[1] = v[1]; w[2] = v[2]; w[3] = v[3];
    } else if constexpr (EPL == 4) {
      const uint2 v = *reinterpret_cast<const uint2*>(q);
      w[0] = v.x; w[1] = v.y;
    } else if constexpr (EPL == 2) {
      w[0] = *reinterpret_cast<const uint32_t*>(q);
    } else {
      w[0] = *q;
    }
#pragma unroll
    for (int e = 0; e < EPL; ++e) x[e] = __uint_as_float((e & 1) ? (w[e / 2] & 0xffff0000u) : (w[e / 2] << 16));
  } else {
    const float* q = static_cast<const float*>(p) + i;
#pragma unroll
    for (int e = 0; e < EPL; e += (EPL >= 4 ? 4 : EPL)) {
      if constexpr (EPL >= 4) {
        const float4 v = *reinterpret_cast<const float4*>(q + e);
        x[e] = v.x; x[e + 1] = v.y; x[e + 2] = v.z; x[e + 3] = v.w;
      } else if constexpr (EPL == 2) {
        const float2 v = *reinterpret_cast<const float2*>(q);
        x[0] = v.x; x[1] = v.y;
      } else {
        x[0] = *q;
      }
    }
  }
}

template <bool BF16, int EPL>
__device__ __forceinline__ void store_n(void* p, size_t i, const float (&x)[EPL]) {
  if constexpr (BF16) {
    uint16_t* q = static_cast<uint16_t*>(p) + i;
    if constexpr (EPL == 1) {
      *q = static_cast<uint16_t>(pack_bf16x2(x[0], 0.f));
    } else {
      uint32_t w[EPL / 2];
#pragma unroll
      for (int e = 0; e < EPL / 2; ++e) w[e] = pack_bf16x2(x[2 * e], x[2 * e + 1]);
      if constexpr (EPL == 8) *reinterpret_cast<uint4*>(q) = make_uint4(w[0], w[1], w[2], w[3]);
      else if constexpr (EPL == 4) *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
      else *reinterpret_cast<uint32_t*>(q) = w[0];
    }
  } else {
    float* q = static_cast<float*>(p) + i;
    if constexpr (EPL >= 4) {
#pragma unroll
      for (int e = 0; e < EPL; e += 4) *reinterpret_cast<float4*>(q + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
    } else if constexpr (EPL == 2) {
      *reinterpret_cast<float2*>(q) = make_float2(x[0], x[1]);
    } else {
      *q = x[0];
    }
  }
}

// Largest value over aligned groups of 16 lanes, in every lane of the group,
// as unsigned integers.  On the bits of |x| this is the largest magnitude
// with NaN above infinity above every finite value, so a NaN is never lost.
__device__ __forceinline__ uint32_t lane_group_umax16(uint32_t x) {
  auto step = [&](auto ctrl) {
    const uint32_t y = static_cast<uint32_t>(
        __builtin_amdgcn_update_dpp(0, static_cast<int>(x), decltype(ctrl)::value, 0xF, 0xF, true));
    x = y > x ? y : x;
  };
  step(std::integral_constant<int, 0xB1>{});
  step(std::integral_constant<int, 0x4E>{});
  step(std::integral_constant<int, 0x141>{});
  step(std::integral_constant<int, 0x140>{});
  return x;
}

// Sum over aligned groups of W lanes (2, 4, 8 or 16), in every lane of the group.
template <int W>
__device__ __forceinline__ float dpp_group_sum(float x) {
  static_assert(W == 2 || W == 4 || W == 8 || W == 16, "inside one DPP row");
  x += dpp_mov<0xB1>(x);
  if constexpr (W >= 4) x += dpp_mov<0x4E>(x);
  if constexpr (W >= 8) x += dpp_mov<0x141>(x);
  if constexpr (W == 16) x += dpp_mov<0x140>(x);
  return x;
}

// x = 2^k m with m in [0.5, 1): returns 2^k and leaves m in x.  Infinity and NaN
// stay in x, with 2^0; 0 gives 0 and 0.
__device__ __forceinline__ float split_power(float& x) {
  const float p = x == 0.0f ? 0.0f : __builtin_amdgcn_ldexpf(1.0f, __builtin_amdgcn_frexp_expf(x));
  x = __builtin_amdgcn_frexp_mantf(x);
  return p;
}

// The scale of the 128-channel block whose values m * t[e] sit 8 to a lane
// over an aligned group of 16 lanes (every lane active; lanes past the row's
// end hold zeros), and those 8 values as e4m3, rounded to nearest even:
// s = max(amax |m t|, 1e-30) / 448, q = t * (448 / amax |t|).  m (one value in
// every lane of the group), the row's 1 / rms up to a power of two, goes into
// the scale alone: two roundings less per value than (m t) / s.  The norm takes
// the power into t, which so stays in fp32's range where m t does; heads of 128
// pass 1 / rms itself.  A NaN in the block makes its scale NaN.
__device__ __forceinline__ uint2 quantise_block8(const float (&t)[8], float m, float* scale) {
  uint32_t a = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = __float_as_uint(t[e]) & 0x7fffffffu;
    a = b > a ? b : a;
  }
  const float amax = __uint_as_float(lane_group_umax16(a));
  const bool tiny = amax * m <= kAmaxFloor;
  *scale = (tiny ? kAmaxFloor : amax * m) * (1.0f / kE4M3Max);
  // Where amax is below 1 the values are multiplied by 2^-30 of that factor and
  // the conversion multiplies by 2^30, so that the factor is a normal number for
  // every amax (a small eps lifts values near the type's smallest) and a zero
  // times it stays a zero.
  const float raise = amax < 1.0f ? 0x1p-30f : 1.0f;
  const float c = tiny ? fminf(m * (kE4M3Max * 0x1p-30f / kAmaxFloor), 3.4028235e38f) : kE4M3Max * raise / amax;
  typedef short s16x2 __attribute__((ext_vector_type(2)));
  s16x2 lo = {}, hi = {};
  lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, t[0] * c, t[1] * c, raise, false);
  lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, t[2] * c, t[3] * c, raise, true);
  hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(hi, t[4] * c, t[5] * c, raise, false);
  hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(hi, t[6] * c, t[7] * c, raise, true);
  return make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
}

}  // namespace kda
