// Norm of the query and key heads and their rotation by position,
//   y = rotate(x / sqrt(mean x^2 + eps) * w),
// and its backward pass: with g the upstream gradient rotated back, n = x /
// sqrt(mean x^2 + eps) and u = g * w,
//   dx = (u - n * mean(u n)) / sqrt(mean x^2 + eps),  dw = sum g * n.
//
// HBM-bound: each head is read once and kept in the registers of D / 16 lanes
// (rope.h).  Such a group of lanes takes a token and a run of its heads, whose
// sines it forms once, from an angle reduced in 64 bits: for bf16 outputs (in the
// backward, bf16 gradients) with v_sin_f32 and v_cos_f32, which take turns in fp32
// and are at most 1.2e-7 and the angle's rounding off, absolutely; for fp32 ones to
// fp32's own rounding, by a series in 64 bits.  32768 tokens of
// 40 heads of 128 in bf16: 125 us (5.4 TB/s); backward, of 18 heads of 256: 242 (5.0);
// 16384 of 40 of 128 in fp32: 129 (5.2) and 140 (with the hardware's sines 128, 136).
#include <algorithm>

#include "kda_device.h"
#include "kda_internal.h"
#include "rope.h"
#include "vec_io.h"

namespace kda {

namespace {

constexpr int kThreads = 256;

template <int D, bool INTER, bool BF16>
__device__ __forceinline__ void sines(const RopeArgs& r, const PairRates& p, int64_t token, float (&c)[8],
                                      float (&s)[8]) {
  const Places at(r, token);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const double t = turns(p, at, e);
    if constexpr (BF16) {
      c[e] = __builtin_amdgcn_cosf(static_cast<float>(t));
      s[e] = __builtin_amdgcn_sinf(static_cast<float>(t));
    } else {
      sincos_turns32(t, s[e], c[e]);
    }
  }
}

}  // namespace

// Group g of lanes takes token g / runs and the run g % runs of its heads: the
// runs of q's heads, then those of k's, kRun of them, whose loads are in flight
// together.
template <int D, bool IN_BF16, bool OUT_BF16, bool INTER, int kRun>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_kernel(RopeArgs r, QkArgs x, float eps) {
  constexpr int L = D / 16;
  const int lane = threadIdx.x % L;
  const HeadRuns<D, INTER> runs(lane, r.rotary_dim);
  const PairRates rates = pair_rates<D, INTER>(r, runs);
  const int q_runs = (x.heads[0] + kRun - 1) / kRun;
  const int n_runs = q_runs + (x.heads[1] + kRun - 1) / kRun;
  const int64_t groups = r.n_tokens * n_runs;
  for (int64_t g = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / L; g < groups;
       g += static_cast<int64_t>(gridDim.x) * kThreads / L) {
    const int64_t token = g / n_runs;
    const int run = static_cast<int>(g - token * n_runs);
    const int which = run >= q_runs;
    const int h0 = (which ? run - q_runs : run) * kRun;
    const int heads = which ? x.heads[1] : x.heads[0];
    const int h1 = h0 + kRun < heads ? h0 + kRun : heads;
    const void* from = which ? x.in[1] : x.in[0];
    void* to = which ? x.out[1] : x.out[0];
    const float* w = which ? x.w[1] : x.w[0];
    const size_t in0 = static_cast<size_t>(token) * (which ? x.stride[1] : x.stride[0]);
    const size_t out0 = static_cast<size_t>(token) * heads * D;
    float c[8], s[8], wa[8], wb[8];
    if (r.rotary_dim) sines<D, INTER, OUT_BF16>(r, rates, token, c, s);
    if (w) {
      load_n<false, 8>(w, runs.a, wa);
      load_n<false, 8>(w, runs.b, wb);
    }
    float a[kRun][8], b[kRun][8];
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const size_t at = in0 + static_cast<size_t>(h0 + i < h1 ? h0 + i : h1 - 1) * D;
      load_n<IN_BF16, 8>(from, at + runs.a, a[i]);
      load_n<IN_BF16, 8>(from, at + runs.b, b[i]);
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      if (h0 + i >= h1) break;
      if (w) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(a[i][e], a[i][e], fmaf(b[i][e], b[i][e], ss));
        const float inv = rsqrt_precise(dpp_group_sum<L>(ss) * (1.0f / D) + eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          a[i][e] *= inv * wa[e];
          b[i][e] *= inv * wb[e];
        }
      }
      rotate<D, INTER>(runs, a[i], b[i], c, s);
      const size_t at = out0 + static_cast<size_t>(h0 + i) * D;
      store_n<OUT_BF16, 8>(to, at + runs.a, a[i]);
      store_n<OUT_BF16, 8>(to, at + runs.b, b[i]);
    }
  }
}

// Groups take a token's head at a time, first all of q's and then all of k's; a
// lane keeps its channels, so both weights' gradients gather in its registers.  A
// workgroup joins its lanes in LDS and leaves one row of `part`, [2][D].  Groups and
// the order of every sum depend on the sizes alone.  (Runs of four heads whose sines
// are formed once, with two heads' loads in flight, took 140 to 142 us where this
// takes 124 to 138: 16384 tokens, 16 + 2 heads of 256 or 32 + 8 of 128.)
template <int D, bool IN_BF16, bool OUT_BF16, bool INTER>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_bwd_kernel(RopeArgs r, QkArgs x, float eps,
                                                                    float* __restrict__ part) {
  constexpr int L = D / 16;
  __shared__ float red[4][kThreads][8];   // q's and k's weight, the two runs of each
  const int lane = threadIdx.x % L;
  const HeadRuns<D, INTER> runs(lane, r.rotary_dim);
  const PairRates rates = pair_rates<D, INTER>(r, runs);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float da[8] = {}, db[8] = {}, wa[8], wb[8];
    const float* w = x.w[which];
    if (w) {
      load_n<false, 8>(w, runs.a, wa);
      load_n<false, 8>(w, runs.b, wb);
    }
    const int heads = x.heads[which];
    const int64_t groups = r.n_tokens * heads;
    for (int64_t g = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / L; g < groups;
         g += static_cast<int64_t>(gridDim.x) * kThreads / L) {
      const int64_t token = g / heads;
      const size_t in = static_cast<size_t>(token) * x.stride[which] + static_cast<size_t>(g - token * heads) * D;
      const size_t out = static_cast<size_t>(g) * D;
      float a[8], b[8], ga[8], gb[8];
      load_n<IN_BF16, 8, true>(x.in[which], in + runs.a, a);
      load_n<IN_BF16, 8, true>(x.in[which], in + runs.b, b);
      load_n<OUT_BF16, 8, true>(x.dy[which], out + runs.a, ga);
      load_n<OUT_BF16, 8, true>(x.dy[which], out + runs.b, gb);
      if (r.rotary_dim) {
        float c[8], s[8];
        sines<D, INTER, OUT_BF16>(r, rates, token, c, s);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = -s[e];   // back
        rotate<D, INTER>(runs, ga, gb, c, s);
      }
      if (w) {
        float ss = 0.f, sg = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ss = fmaf(a[e], a[e], fmaf(b[e], b[e], ss));
          sg = fmaf(ga[e] * wa[e], a[e], fmaf(gb[e] * wb[e], b[e], sg));
        }
        ss = dpp_group_sum<L>(ss);
        sg = dpp_group_sum<L>(sg);
        const float inv = rsqrt_precise(ss * (1.0f / D) + eps);
        // n * mean(u n) = x * k; 0 where the squares pass fp32's range, as n is
        const float k = inv == 0.f ? 0.f : sg * (1.0f / D) * inv * inv;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          da[e] = fmaf(ga[e], a[e] * inv, da[e]);
          db[e] = fmaf(gb[e], b[e] * inv, db[e]);
          ga[e] = inv * fmaf(-a[e], k, ga[e] * wa[e]);
          gb[e] = inv * fmaf(-b[e], k, gb[e] * wb[e]);
        }
      }
      store_n<false, 8>(x.out[which], out + runs.a, ga);
      store_n<false, 8>(x.out[which], out + runs.b, gb);
    }
    store_n<false, 8>(&red[2 * which][threadIdx.x][0], 0, da);
    store_n<false, 8>(&red[2 * which + 1][threadIdx.x][0], 0, db);
  }
  // the lanes of a channel joined: lane l of every group
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    const int set = i / (8 * L), l = i / 8 % L, e = i % 8;
    const HeadRuns<D, INTER> to(l, r.rotary_dim);
    float t[4] = {};
#pragma unroll
    for (int k = 0; k < kThreads / L; k += 4)
#pragma unroll
      for (int x = 0; x < 4; ++x) t[x] += red[set][(k + x) * L + l][e];
    part[(static_cast<size_t>(blockIdx.x) * 2 + set / 2) * D + (set & 1 ? to.b : to.a) + e] = (t[0] + t[1]) + (t[2] + t[3]);
  }
}

namespace {

template <class F>
hipError_t with_shape(int D, bool in_bf16, bool out_bf16, bool inter, F&& f) {
  using std::false_type;
  using std::true_type;
  auto by_pairs = [&](auto d, auto ib, auto ob) {
    if (inter) f(d, ib, ob, true_type{});
    else f(d, ib, ob, false_type{});
    return hipGetLastError();
  };
  auto by_type = [&](auto d) {
    if (in_bf16 && out_bf16) return by_pairs(d, true_type{}, true_type{});
    if (in_bf16) return by_pairs(d, true_type{}, false_type{});
    if (out_bf16) return by_pairs(d, false_type{}, true_type{});
    return by_pairs(d, false_type{}, false_type{});
  };
  switch (D) {
    case 64: return by_type(std::integral_constant<int, 64>{});
    case 128: return by_type(std::integral_constant<int, 128>{});
    case 256: return by_type(std::integral_constant<int, 256>{});
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

// Four heads a group from 4096 waves of one head on (the sines are formed once,
// and four heads' loads are in flight): 2000 tokens, 40 heads of 128: 11.1 us, with
// one 15.0; 16384 tokens: 64, 75.  Below, latency counts: one token, 16 + 2 heads of
// 256: 7.2, with one 6.3.
hipError_t launch_qk_norm_rope(int D, const RopeArgs& r, const QkArgs& x, float eps, bool in_bf16, bool out_bf16,
                               hipStream_t st) {
  const int64_t lanes = r.n_tokens * (x.heads[0] + x.heads[1]) * (D / 16);
  const int run = lanes / 64 >= 4096 ? 4 : 1;
  const int64_t groups = r.n_tokens * ((x.heads[0] + run - 1) / run + (x.heads[1] + run - 1) / run);
  const int64_t blocks = (groups * (D / 16) + kThreads - 1) / kThreads;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(blocks, 256 * 16)));
  return with_shape(D, in_bf16, out_bf16, r.interleaved, [&](auto d, auto ib, auto ob, auto inter) {
    constexpr int kD = decltype(d)::value;
    constexpr bool kIn = decltype(ib)::value, kOut = decltype(ob)::value, kInter = decltype(inter)::value;
    if (run == 1) qk_norm_rope_kernel<kD, kIn, kOut, kInter, 1><<<grid, kThreads, 0, st>>>(r, x, eps);
    else qk_norm_rope_kernel<kD, kIn, kOut, kInter, 4><<<grid, kThreads, 0, st>>>(r, x, eps);
  });
}

// Workgroups of the backward, each with a row of partial sums: three a CU at most.
int qk_norm_rope_bwd_parts(int D, int64_t n, int heads) {
  const int64_t blocks = (n * heads * (D / 16) + kThreads - 1) / kThreads;
  return static_cast<int>(std::min<int64_t>(blocks, 768));
}

hipError_t launch_qk_norm_rope_bwd(int D, const RopeArgs& r, const QkArgs& x, float eps, float* d_weight, float* part,
                                   bool in_bf16, bool out_bf16, hipStream_t st) {
  const int parts = qk_norm_rope_bwd_parts(D, r.n_tokens, x.heads[0] + x.heads[1]);
  if (parts > 0) {
    const hipError_t e = with_shape(D, in_bf16, out_bf16, r.interleaved, [&](auto d, auto ib, auto ob, auto inter) {
      qk_norm_rope_bwd_kernel<decltype(d)::value, decltype(ib)::value, decltype(ob)::value, decltype(inter)::value>
          <<<dim3(parts), kThreads, 0, st>>>(r, x, eps, part);
    });
    if (e != hipSuccess) return e;
  }
  return launch_column_sums(parts, 2 * D, part, d_weight, st);
}

}  // namespace kda
