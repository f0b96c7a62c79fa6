// Appending to and reading from the paged cache of 4-bit keys and values.
//
// A block of 32 channels is held as e2m1 values times 2^e, e the least with
// max|x| <= 6 * 2^e; with max|x| = 1.m * 2^p that is p - 2 where 1.m <= 1.5 and
// p - 1 above, read off the maximum's bits.  The card converts both ways with
// the power applied (v_cvt_scalef32_pk_fp4_f32 to nearest even, and back
// exactly, a scale byte of 255 as NaN; both were compared over their ranges).
//
// Keys are normed and rotated in 64 bits (as fast as fp32 here) and rounded to
// fp32 "to odd": the last bit is set where anything was cut.  No boundary
// between two codes, and no power of two or 1.5 times one, is then crossed or
// reached by that rounding, so every key is held as the nearest value.
//
// 65536 tokens of 2 heads of 256, 64 channels of them rotated: 51 us back to back (174
// MB, 3.4 TB/s: a token begins with five dependent loads, and 64-bit values leave
// registers for two waves a SIMD), 30 to read (6.1 TB/s).
#include <algorithm>

#include "kda_device.h"
#include "kda_internal.h"
#include "kv_cache.h"
#include "rope.h"
#include "vec_io.h"

namespace kda {

namespace {

constexpr int kThreads = 256;

// Sine and cosine of t turns, |t| <= 1/2: to the nearest quarter turn, then the
// Taylor series within an eighth (the terms left out are below 1e-16).
__device__ __forceinline__ void sincos_turns(double t, double& s, double& c) {
  const double q = rint(4.0 * t);
  const double x = (t - 0.25 * q) * 6.283185307179586476925;
  const double z = x * x;
  double a = 1.0 / 355687428096000.0;           // 1 / 17!
  a = fma(a, z, -1.0 / 1307674368000.0);        // 15!
  a = fma(a, z, 1.0 / 6227020800.0);            // 13!
  a = fma(a, z, -1.0 / 39916800.0);             // 11!
  a = fma(a, z, 1.0 / 362880.0);
  a = fma(a, z, -1.0 / 5040.0);
  a = fma(a, z, 1.0 / 120.0);
  a = fma(a, z, -1.0 / 6.0);
  a = fma(a * z, x, x);
  double b = 1.0 / 20922789888000.0;            // 1 / 16!
  b = fma(b, z, -1.0 / 87178291200.0);          // 14!
  b = fma(b, z, 1.0 / 479001600.0);             // 12!
  b = fma(b, z, -1.0 / 3628800.0);              // 10!
  b = fma(b, z, 1.0 / 40320.0);
  b = fma(b, z, -1.0 / 720.0);
  b = fma(b, z, 1.0 / 24.0);
  b = fma(b, z, -0.5);
  b = fma(b, z, 1.0);
  const int n = static_cast<int>(q) & 3;
  const double u = n & 1 ? b : a, v = n & 1 ? a : b;
  s = n & 2 ? -u : u;
  c = (n + 1) & 2 ? -v : v;
}

// Sum over aligned groups of W lanes of doubles, in every lane.
template <int W>
__device__ __forceinline__ double group_sum64(double x) {
  auto step = [&](auto ctrl) {
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(x));
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), decltype(ctrl)::value, 0xF, 0xF, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), decltype(ctrl)::value, 0xF, 0xF, true);
    x += __longlong_as_double(static_cast<long long>(static_cast<uint64_t>(hi) << 32 | lo));
  };
  step(std::integral_constant<int, 0xB1>{});
  step(std::integral_constant<int, 0x4E>{});
  if constexpr (W >= 8) step(std::integral_constant<int, 0x141>{});
  if constexpr (W >= 16) step(std::integral_constant<int, 0x140>{});
  return x;
}

// 1 / sqrt(x) from the hardware's with two Newton steps; 0 at infinity.
__device__ __forceinline__ double rsqrt64(double x) {
  double r = __builtin_amdgcn_rsq(x);
  r = fma(fma(-x * r, r, 1.0), 0.5 * r, r);
  r = fma(fma(-x * r, r, 1.0), 0.5 * r, r);
  return x == __longlong_as_double(0x7ff0000000000000ll) ? 0.0 : r;
}

// y rounded to fp32, to odd: cut (the nearest value, or the one below its
// magnitude), the last bit set where y is not that; subnormal values likewise.
__device__ __forceinline__ float round_odd(double y) {
  const float f = static_cast<float>(y);
  const double near = f;
  return __uint_as_float((__float_as_uint(f) - (fabs(near) > fabs(y))) | (near != y));
}

__device__ __forceinline__ uint32_t max_bits(const float (&x)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = __float_as_uint(x[e]) & 0x7fffffffu;
    m = b > m ? b : m;
  }
  return m;
}

// Largest over aligned groups of 4 lanes, in each of them.
__device__ __forceinline__ uint32_t quad_umax(uint32_t x) {
  uint32_t y = __builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0xB1, 0xF, 0xF, true);
  x = y > x ? y : x;
  y = __builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x4E, 0xF, 0xF, true);
  return y > x ? y : x;
}

// The scale byte of a block whose largest magnitude has these bits.
__device__ __forceinline__ int block_scale_byte(uint32_t amax) {
  const int p = static_cast<int>(amax >> 23);
  if (p >= 254) return kScaleNaN;
  const int e = p - 2 + ((amax & 0x7fffffu) > 0x400000u);
  return e < 1 ? 1 : e;
}

// 8 values as codes, the first in the lowest half byte.
__device__ __forceinline__ uint32_t encode8(const float (&x)[8], int scale_byte) {
  if (scale_byte == kScaleNaN) return 0;
  const float s = __uint_as_float(static_cast<uint32_t>(scale_byte) << 23);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], s, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], s, 3);
  return w;
}

__device__ __forceinline__ void decode8(uint32_t w, int scale_byte, float (&x)[8]) {
  const float s = __uint_as_float(static_cast<uint32_t>(scale_byte) << 23);
  auto put = [&](auto v, int e) {
    x[e] = v[0];
    x[e + 1] = v[1];
  };
  put(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0), 0);
  put(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1), 2);
  put(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2), 4);
  put(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3), 6);
}

}  // namespace

// 8 elements as they are in memory, so that their loads can be under way early.
template <bool BF16>
struct Raw8 {
  uint4 w[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* p, size_t i) {
    const uint4* from = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + i * (BF16 ? 2 : 4));
#pragma unroll
    for (int x = 0; x < (BF16 ? 1 : 2); ++x) w[x] = from[x];
  }
  __device__ __forceinline__ void widen(float (&x)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (BF16) {
        const uint32_t pair = e < 2 ? w[0].x : e < 4 ? w[0].y : e < 6 ? w[0].z : w[0].w;
        x[e] = __uint_as_float(e & 1 ? pair & 0xffff0000u : pair << 16);
      } else {
        const uint4& v = w[e >> 2 & (BF16 ? 0 : 1)];
        x[e] = __uint_as_float((e & 3) == 0 ? v.x : (e & 3) == 1 ? v.y : (e & 3) == 2 ? v.z : v.w);
      }
    }
  }
};

// Group g of D / 16 lanes takes token g / runs and the run g % runs of its heads.
// A head's rows are on their way while the head before them is worked on, the
// first one's while the token's place is looked up.
template <int D, bool BF16, bool INTER>
__global__ __launch_bounds__(kThreads) void append_kv_kernel(RopeArgs r, CacheArgs c, const void* __restrict__ k,
                                                             int64_t k_stride, const void* __restrict__ v,
                                                             int64_t v_stride, const float* __restrict__ w, float eps,
                                                             int run_len) {
  constexpr int L = D / 16;
  // largest magnitudes of the runs of 8 channels, a group's in the channels' order
  __shared__ alignas(16) uint32_t most[kThreads / L][2 * L];
  const int lane = threadIdx.x % L;
  // turns a position and axes of the pairs; sines and cosines of the groups'
  // tokens, each formed by one lane
  __shared__ double rate[D / 2];
  __shared__ uint32_t axis[D / 2];
  __shared__ double2 circle[kThreads / L][D / 2];
  const HeadRuns<D, INTER> runs(lane, r.rotary_dim);
  const int pairs = r.rotary_dim >> 1;
  if (static_cast<int>(threadIdx.x) < pairs) {
    const int ax = r.axis ? r.axis[threadIdx.x] : 0;
    rate[threadIdx.x] = static_cast<double>(r.inv_freq[threadIdx.x]) * kPerTurn;
    axis[threadIdx.x] = ax < 0 ? 0 : ax >= r.num_axes ? r.num_axes - 1 : ax;
  }
  __syncthreads();
  double2* const around = circle[threadIdx.x / L];
  uint32_t* const mine = most[threadIdx.x / L];
  const int va = 8 * lane, vb = D / 2 + 8 * lane;   // the runs of the values
  const int n_runs = (c.heads + run_len - 1) / run_len;
  const int64_t groups = c.n_tokens * n_runs;
  for (int64_t g = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / L; g < groups;
       g += static_cast<int64_t>(gridDim.x) * kThreads / L) {
    const int64_t token = g / n_runs;
    const int h0 = static_cast<int>(g - token * n_runs) * run_len;
    const int h1 = h0 + run_len < c.heads ? h0 + run_len : c.heads;
    Raw8<BF16> raw[4];
    auto fetch = [&](int h) {
      const size_t ki = static_cast<size_t>(token) * k_stride + static_cast<size_t>(h) * D;
      const size_t vi = static_cast<size_t>(token) * v_stride + static_cast<size_t>(h) * D;
      raw[0].load(k, ki + runs.a);
      raw[1].load(k, ki + runs.b);
      raw[2].load(v, vi + va);
      raw[3].load(v, vi + vb);
    };
    fetch(h0);
    const RowAt at = row_at(c, token);
    if (at.seq < 0) continue;
    const int page = page_of(c, at.seq, at.pos);
    if (page < 0) continue;
    const int off = static_cast<int>(at.pos & ((1 << c.page_shift) - 1));
    if (r.rotary_dim) {
      const Places places = r.positions ? Places(r, token) : Places(static_cast<int32_t>(at.pos));
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll 1
      for (int i = lane; i < pairs; i += L) {
        double2 cs;
        sincos_turns(turns(rate[i], places.on(axis[i])), cs.y, cs.x);
        around[i] = cs;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    float wa[8], wb[8];
    if (w) {
      load_n<false, 8>(w, runs.a, wa);
      load_n<false, 8>(w, runs.b, wb);
    }
    for (int h = h0; h < h1; ++h) {
      float ka[8], kb[8], xa[8], xb[8];
      raw[0].widen(ka);
      raw[1].widen(kb);
      raw[2].widen(xa);
      raw[3].widen(xb);
      fetch(h + 1 < h1 ? h + 1 : h);
      double ya[8], yb[8];
      if (w) {
        double ss = 0.0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ya[e] = ka[e];
          yb[e] = kb[e];
          ss = fma(ya[e], ya[e], fma(yb[e], yb[e], ss));
        }
        const double inv = rsqrt64(group_sum64<L>(ss) * (1.0 / D) + static_cast<double>(eps));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ya[e] *= inv * static_cast<double>(wa[e]);
          yb[e] *= inv * static_cast<double>(wb[e]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ya[e] = ka[e];
          yb[e] = kb[e];
        }
      }
      if (runs.turn_a || runs.turn_b) {
        double cs[8], sn[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const double2 x = around[runs.turned(e) ? runs.pair(e) : 0];
          cs[e] = x.x;
          sn[e] = x.y;
        }
        rotate<D, INTER>(runs, ya, yb, cs, sn);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ka[e] = round_odd(ya[e]);
        kb[e] = round_odd(yb[e]);
      }
      // the runs' maxima meet in LDS, within the group and so within a wave
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      mine[runs.a >> 3] = max_bits(ka);
      mine[runs.b >> 3] = max_bits(kb);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      const uint4 ma = *reinterpret_cast<const uint4*>(mine + (runs.a >> 5) * 4);
      const uint4 mb = *reinterpret_cast<const uint4*>(mine + (runs.b >> 5) * 4);
      const int ea = block_scale_byte(std::max(std::max(ma.x, ma.y), std::max(ma.z, ma.w)));
      const int eb = block_scale_byte(std::max(std::max(mb.x, mb.y), std::max(mb.z, mb.w)));
      const size_t values = values_at<D>(c, page, h) + static_cast<size_t>(off) * (D / 2);
      const size_t scales = scales_at<D>(c, page, h) + off;
      *reinterpret_cast<uint32_t*>(c.k + values + (runs.a >> 1)) = encode8(ka, ea);
      *reinterpret_cast<uint32_t*>(c.k + values + (runs.b >> 1)) = encode8(kb, eb);
      if ((runs.a & 31) == 0) c.k_scale[scales + (static_cast<size_t>(runs.a >> 5) << c.page_shift)] = ea;
      if ((runs.b & 31) == 0) c.k_scale[scales + (static_cast<size_t>(runs.b >> 5) << c.page_shift)] = eb;
      const int fa = block_scale_byte(quad_umax(max_bits(xa))), fb = block_scale_byte(quad_umax(max_bits(xb)));
      *reinterpret_cast<uint32_t*>(c.v + values + (va >> 1)) = encode8(xa, fa);
      *reinterpret_cast<uint32_t*>(c.v + values + (vb >> 1)) = encode8(xb, fb);
      if ((lane & 3) == 0) {
        c.v_scale[scales + (static_cast<size_t>(va >> 5) << c.page_shift)] = fa;
        c.v_scale[scales + (static_cast<size_t>(vb >> 5) << c.page_shift)] = fb;
      }
    }
  }
}

// Group g of D / 16 lanes takes row g / heads, head g % heads.
template <int D, bool BF16>
__global__ __launch_bounds__(kThreads) void read_kv_kernel(CacheArgs c, void* __restrict__ k_out,
                                                           void* __restrict__ v_out) {
  constexpr int L = D / 16;
  const int lane = threadIdx.x % L;
  const int64_t groups = c.n_tokens * c.heads;
  for (int64_t g = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / L; g < groups;
       g += static_cast<int64_t>(gridDim.x) * kThreads / L) {
    const int64_t token = g / c.heads;
    const int h = static_cast<int>(g - token * c.heads);
    const RowAt at = row_at(c, token);
    if (at.seq < 0) continue;
    const int page = page_of(c, at.seq, at.pos);
    const int off = static_cast<int>(at.pos & ((1 << c.page_shift) - 1));
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      void* out = which ? v_out : k_out;
      if (!out) continue;
      float x[2][8] = {};
      if (page >= 0) {
        const uint8_t* values = (which ? c.v : c.k) + values_at<D>(c, page, h) + static_cast<size_t>(off) * (D / 2);
        const uint8_t* scales = (which ? c.v_scale : c.k_scale) + scales_at<D>(c, page, h) + off;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int at8 = i * (D / 2) + 8 * lane;
          decode8(*reinterpret_cast<const uint32_t*>(values + (at8 >> 1)),
                  scales[static_cast<size_t>(at8 >> 5) << c.page_shift], x[i]);
        }
      }
      store_n<BF16, 8>(out, static_cast<size_t>(g) * D + 8 * lane, x[0]);
      store_n<BF16, 8>(out, static_cast<size_t>(g) * D + D / 2 + 8 * lane, x[1]);
    }
  }
}

namespace {

template <class F>
hipError_t with_head(int D, bool bf16, F&& f) {
  auto by_type = [&](auto d) {
    if (bf16) f(d, std::true_type{});
    else f(d, std::false_type{});
    return hipGetLastError();
  };
  switch (D) {
    case 64: return by_type(std::integral_constant<int, 64>{});
    case 128: return by_type(std::integral_constant<int, 128>{});
    case 256: return by_type(std::integral_constant<int, 256>{});
    default: return hipErrorInvalidValue;
  }
}

dim3 grid_of(int D, int64_t groups) {
  return dim3(static_cast<unsigned>(std::min<int64_t>((groups * (D / 16) + kThreads - 1) / kThreads, 256 * 16)));
}

}  // namespace

hipError_t launch_append_kv(int D, const RopeArgs& r, const CacheArgs& c, const void* k, int64_t k_stride,
                            const void* v, int64_t v_stride, const float* w, float eps, bool in_bf16, hipStream_t st) {
  // heads of a group: as many as leave 2048 waves, what the card holds of them at once (the sines are formed once).  us
  // with 1, 2, 4, 8: 65536 tokens, 2 heads of 256: 71, 51; 16384: 20.5, 15.7; 4096: 9.5, 9.5; 16384 tokens, 8 heads of 128:
  // 40, 30, 25, 21; 4096: 11.7, 9.5, 9.6, 14.4; 32768, 8 of 64: 50, 35, 28, 24
  const int64_t waves = c.n_tokens * c.heads * (D / 16) / 64;
  const int run = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(c.heads, waves / 2048)));
  const dim3 grid = grid_of(D, c.n_tokens * ((c.heads + run - 1) / run));
  return with_head(D, in_bf16, [&](auto d, auto ib) {
    if (r.interleaved)
      append_kv_kernel<decltype(d)::value, decltype(ib)::value, true>
          <<<grid, kThreads, 0, st>>>(r, c, k, k_stride, v, v_stride, w, eps, run);
    else
      append_kv_kernel<decltype(d)::value, decltype(ib)::value, false>
          <<<grid, kThreads, 0, st>>>(r, c, k, k_stride, v, v_stride, w, eps, run);
  });
}

hipError_t launch_read_kv(int D, const CacheArgs& c, void* k_out, void* v_out, bool out_bf16, hipStream_t st) {
  return with_head(D, out_bf16, [&](auto d, auto ob) {
    read_kv_kernel<decltype(d)::value, decltype(ob)::value>
        <<<grid_of(D, c.n_tokens * c.heads), kThreads, 0, st>>>(c, k_out, v_out);
  });
}

}  // namespace kda
