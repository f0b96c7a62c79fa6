// The KDA layer's output epilogue: o_norm, an RMS norm over each (token,
// head) row of dv outputs with one weight per channel, times the sigmoid of
// the output gate (AliceAI page, section 三: KDA's o_norm and sigmoid gate;
// section 二: output_gate among the per-token control inputs):
//   y[j] = o[j] / sqrt(mean_j' o[j']^2 + eps) * w[j] * sigmoid(gate[j])
//
// HBM-bound (read o and gate, write y).  A row belongs to 16 consecutive
// lanes (one DPP row), dv / 16 elements each, so a bf16 row of 128 is one
// 16-byte load per lane and operand, and the row's sum of squares is four
// DPP steps with no LDS.  A wave covers four rows; workgroups stride over
// the rows.
#include "kda_device.h"
#include "kda_internal.h"
#include "vec_io.h"

namespace kda {

namespace {

constexpr int kEpiThreads = 256;

}  // namespace

template <int DV, bool O_BF16, bool G_BF16>
__global__ __launch_bounds__(kEpiThreads) void output_gate_kernel(int64_t rows, const void* o, const void* gate,
                                                                  const float* __restrict__ w, float eps, void* y) {
  constexpr int EPL = DV / 16;
  const int l16 = threadIdx.x & 15;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * kEpiThreads + threadIdx.x) >> 4;
  const int64_t step = (static_cast<int64_t>(gridDim.x) * kEpiThreads) >> 4;
  float wv[EPL];
#pragma unroll
  for (int e = 0; e < EPL; ++e) wv[e] = w[l16 * EPL + e];
  // every lane of a 16-lane group takes the same rows, so a group is either
  // wholly active or wholly idle and its DPP sums stay inside it
  for (int64_t r = first; r < rows; r += step) {
    const size_t base = static_cast<size_t>(r) * DV + static_cast<size_t>(l16) * EPL;
    float ov[EPL], gv[EPL];
    load_n<O_BF16, EPL>(o, base, ov);
    load_n<G_BF16, EPL>(gate, base, gv);
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < EPL; ++e) ss = fmaf(ov[e], ov[e], ss);
    ss = lane_group_sum<16>(ss);
    const float inv = 1.0f / sqrtf(ss * (1.0f / DV) + eps);
    float yv[EPL];
#pragma unroll
    for (int e = 0; e < EPL; ++e) yv[e] = ov[e] * inv * wv[e] * sigmoidf_(gv[e]);
    store_n<O_BF16, EPL>(y, base, yv);
  }
}

template <int DV>
static hipError_t launch_output_gate_d(int64_t rows, const void* o, const void* gate, const float* w, float eps,
                                       void* y, bool o_bf16, bool g_bf16, hipStream_t st) {
  const int64_t groups_per_block = kEpiThreads / 16;
  const int64_t blocks = (rows + groups_per_block - 1) / groups_per_block;
  const dim3 grid(static_cast<unsigned>(blocks < (1 << 20) ? blocks : (1 << 20)));
  if (o_bf16 && g_bf16) output_gate_kernel<DV, true, true><<<grid, kEpiThreads, 0, st>>>(rows, o, gate, w, eps, y);
  else if (o_bf16) output_gate_kernel<DV, true, false><<<grid, kEpiThreads, 0, st>>>(rows, o, gate, w, eps, y);
  else if (g_bf16) output_gate_kernel<DV, false, true><<<grid, kEpiThreads, 0, st>>>(rows, o, gate, w, eps, y);
  else output_gate_kernel<DV, false, false><<<grid, kEpiThreads, 0, st>>>(rows, o, gate, w, eps, y);
  return hipGetLastError();
}

hipError_t launch_output_gate(int D, int64_t rows, const void* o, const void* gate, const float* w, float eps,
                              void* y, bool o_bf16, bool g_bf16, hipStream_t st) {
  if (rows <= 0) return hipSuccess;
  switch (D) {
    case 16: return launch_output_gate_d<16>(rows, o, gate, w, eps, y, o_bf16, g_bf16, st);
    case 32: return launch_output_gate_d<32>(rows, o, gate, w, eps, y, o_bf16, g_bf16, st);
    case 64: return launch_output_gate_d<64>(rows, o, gate, w, eps, y, o_bf16, g_bf16, st);
    case 128: return launch_output_gate_d<128>(rows, o, gate, w, eps, y, o_bf16, g_bf16, st);
    default: return hipErrorInvalidValue;
  }
}

// The epilogue with its output in e4m3, the operand of the out projection: a
// token's heads side by side are one row of H * dv channels, in blocks of 128
// (whole heads: dv divides 128) with one scale each.  16 lanes hold a block,
// 8 channels a lane, so dv / 8 lanes sum a head's squares and all 16 the
// block's largest value, all in DPP steps.  HBM-bound: 131072 x 32 x 128 in
// bf16 takes 437 to 445 us, 6.1 TB/s; 256 tokens 3.4 us, the launch and one
// trip to memory.  The sigmoid takes the fast exponential, as the plain epilogue
// does: what that is off by at far gates (65 half steps of fp32 at 85) reaches
// the fp32 scale where all gates of a block are far out, and no e4m3 value by
// more than 2e-4 of its step (the precise one takes 6 us more).
template <int DV, bool O_BF16, bool G_BF16>
__global__ __launch_bounds__(kEpiThreads) void output_gate_fp8_kernel(int64_t units, int row, const void* o,
                                                                      const void* gate, const float* __restrict__ w,
                                                                      float eps, uint8_t* __restrict__ y,
                                                                      float* __restrict__ scale) {
  const int l16 = threadIdx.x & 15;
  const int nblk = (row + kScaleBlock - 1) / kScaleBlock;
  const int64_t step = (static_cast<int64_t>(gridDim.x) * kEpiThreads) >> 4;
  float wv[8];
  load_n<false, 8>(w, (l16 * 8) % DV, wv);
  // uniform over the wave, so every lane takes part in its group's DPP steps
  for (int64_t u0 = (static_cast<int64_t>(blockIdx.x) * kEpiThreads + (threadIdx.x & ~63)) >> 4; u0 < units; u0 += step) {
    const int64_t u = u0 + ((threadIdx.x & 63) >> 4);
    // with whole blocks only, unit u of the tensor starts at element 128 u
    int64_t token = 0;
    int blk = 0, left = kScaleBlock;
    size_t base = static_cast<size_t>(u) * kScaleBlock;
    if (row % kScaleBlock) {
      token = u / nblk;
      blk = static_cast<int>(u - token * nblk);
      left = row - blk * kScaleBlock;
      base = static_cast<size_t>(token) * row + static_cast<size_t>(blk) * kScaleBlock;
    }
    const bool mine = u < units && l16 * 8 < left;
    float ov[8] = {}, gv[8] = {};
    if (mine) {
      load_n<O_BF16, 8>(o, base + l16 * 8, ov);
      load_n<G_BF16, 8>(gate, base + l16 * 8, gv);
    }
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(ov[e], ov[e], ss);
    ss = dpp_group_sum<DV / 8>(ss);
    float inv = rsqrt_precise(ss * (1.0f / DV) + eps);
    // heads narrower than a block have norms of their own inside it, and lanes
    // past the row's end none (with eps = 0 it would be infinite).  They are
    // applied in front of the weight, so that o * weight stays in fp32's range;
    // heads as wide as a block would need the norm's split of 1 / rms for that
    // (131072 x 32 x 128: 454 us, without it 442)
    const float each = DV == kScaleBlock ? 1.0f : (mine ? inv : 0.0f);
    float t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = ov[e] * each * wv[e] * sigmoidf_(gv[e]);
    float s;
    const uint2 q = quantise_block8(t, DV == kScaleBlock ? inv : 1.0f, &s);
    if (mine) {
      *reinterpret_cast<uint2*>(y + base + l16 * 8) = q;
      if (l16 == 0) scale[u] = s;
    }
  }
}

// The epilogue's backward pass, with n = o / sqrt(mean o^2 + eps) per head,
// s = sigmoid(gate) and g = dy * w * s:
//   d_o = (g - n * mean(g * n)) / sqrt(mean o^2 + eps)
//   dgate = dy * w * n * s (1 - s),  dw = sum over tokens and heads of dy * n * s
// One pass over the rows, 8 channels a lane.  A lane keeps its channels for
// the whole launch, so dw gathers in registers; a workgroup joins its lanes
// in LDS and leaves one row of `part`.  The order of every sum is fixed.
// The exponential is the precise one, for the fp32 gradient of far gates (2 us
// more).  HBM-bound: 32768 x 32 x 128 in bf16 takes 300 us with the join, 5.4
// TB/s.
template <int DV, bool O_BF16, bool G_BF16>
__global__ __launch_bounds__(kEpiThreads) void output_gate_bwd_kernel(int64_t chunks, const void* __restrict__ o,
                                                                      const void* __restrict__ gate,
                                                                      const float* __restrict__ w, float eps,
                                                                      const void* __restrict__ dy,
                                                                      void* __restrict__ d_o,
                                                                      float* __restrict__ dgate,
                                                                      float* __restrict__ part) {
  constexpr int kLanes = DV / 8;   // lanes of a head's row
  __shared__ float red[kEpiThreads][8];
  float wv[8], dw[8] = {};
  load_n<false, 8>(w, (threadIdx.x % kLanes) * 8, wv);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kEpiThreads;
  for (int64_t c0 = static_cast<int64_t>(blockIdx.x) * kEpiThreads + (threadIdx.x & ~63); c0 < chunks; c0 += step) {
    const int64_t c = c0 + (threadIdx.x & 63);
    const bool mine = c < chunks;   // all or none of a head's lanes
    const size_t base = static_cast<size_t>(c) * 8;
    float ov[8] = {}, gv[8] = {}, dv[8] = {};
    if (mine) {
      load_n<O_BF16, 8>(o, base, ov);
      load_n<G_BF16, 8>(gate, base, gv);
      load_n<O_BF16, 8>(dy, base, dv);
    }
    float ss = 0.f, sg = 0.f, sig[8], off[8];   // off = 1 - sigmoid, exact also where the sigmoid is near 1
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = exp_precise_any(-gv[e]);
      sig[e] = rcp_fast(1.0f + x);
      off[e] = fminf(x, 1e38f) * sig[e];   // (an infinite x has sigmoid 0)
      ss = fmaf(ov[e], ov[e], ss);
      sg = fmaf(dv[e] * wv[e] * sig[e], ov[e], sg);
    }
    ss = dpp_group_sum<kLanes>(ss);
    sg = dpp_group_sum<kLanes>(sg);
    const float inv = 1.0f / sqrtf(ss * (1.0f / DV) + eps);
    // n * mean(g n) = o * k; 0 where the squares pass fp32's range, as n is
    const float k = inv == 0.f ? 0.f : sg * (1.0f / DV) * inv * inv;
    float a[8], b[8];
    if (mine) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = ov[e] * inv, ds = dv[e] * sig[e];
        dw[e] = fmaf(ds, n, dw[e]);
        a[e] = inv * fmaf(-ov[e], k, ds * wv[e]);
        b[e] = ds * wv[e] * n * off[e];
      }
      store_n<O_BF16, 8>(d_o, base, a);
      store_n<false, 8>(dgate, base, b);
    }
  }
  store_n<false, 8>(&red[threadIdx.x][0], 0, dw);
  __syncthreads();
  if (threadIdx.x < DV) {
    float s = 0.f;
    for (int t = threadIdx.x / 8; t < kEpiThreads; t += kLanes) s += red[t][threadIdx.x & 7];
    part[static_cast<size_t>(blockIdx.x) * DV + threadIdx.x] = s;
  }
}

// Calls f with the head size and the two types as constants.
template <class F>
static hipError_t with_gate_types(int D, bool o_bf16, bool g_bf16, F&& f) {
  auto by_type = [&](auto d) {
    if (o_bf16 && g_bf16) f(d, std::true_type{}, std::true_type{});
    else if (o_bf16) f(d, std::true_type{}, std::false_type{});
    else if (g_bf16) f(d, std::false_type{}, std::true_type{});
    else f(d, std::false_type{}, std::false_type{});
    return hipGetLastError();
  };
  switch (D) {
    case 16: return by_type(std::integral_constant<int, 16>{});
    case 32: return by_type(std::integral_constant<int, 32>{});
    case 64: return by_type(std::integral_constant<int, 64>{});
    case 128: return by_type(std::integral_constant<int, 128>{});
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_output_gate_fp8(int D, int64_t n_tokens, int row, const void* o, const void* gate, const float* w,
                                  float eps, uint8_t* y, float* scale, bool o_bf16, bool g_bf16, hipStream_t st) {
  const int64_t units = n_tokens * ((row + kScaleBlock - 1) / kScaleBlock);
  const int64_t blocks = (units + kEpiThreads / 16 - 1) / (kEpiThreads / 16);
  const dim3 grid(static_cast<unsigned>(blocks < (1 << 20) ? blocks : (1 << 20)));
  return with_gate_types(D, o_bf16, g_bf16, [&](auto d, auto ob, auto gb) {
    output_gate_fp8_kernel<decltype(d)::value, decltype(ob)::value, decltype(gb)::value>
        <<<grid, kEpiThreads, 0, st>>>(units, row, o, gate, w, eps, y, scale);
  });
}

// Workgroups of the backward, each with a row of partial sums: three a CU.
// 32768 x 32 x 128 in bf16: 308 us with 768, 325 with 512, 320 with 1024, 371
// with 2048 (more rows at a time, in five streams of memory).
int output_gate_bwd_parts(int D, int64_t rows) {
  const int64_t blocks = (rows * (D / 8) + kEpiThreads - 1) / kEpiThreads;
  return static_cast<int>(blocks < 768 ? blocks : 768);
}

hipError_t launch_output_gate_bwd(int D, int64_t rows, const void* o, const void* gate, const float* w, float eps,
                                  const void* dy, void* d_o, float* dgate, float* dw, float* part, bool o_bf16,
                                  bool g_bf16, hipStream_t st) {
  const int parts = output_gate_bwd_parts(D, rows);
  if (parts > 0) {
    const hipError_t e = with_gate_types(D, o_bf16, g_bf16, [&](auto d, auto ob, auto gb) {
      output_gate_bwd_kernel<decltype(d)::value, decltype(ob)::value, decltype(gb)::value>
          <<<dim3(parts), kEpiThreads, 0, st>>>(rows * (D / 8), o, gate, w, eps, dy, d_o, dgate, part);
    });
    if (e != hipSuccess) return e;
  }
  return launch_column_sums(parts, D, part, dw, st);
}

}  // namespace kda
