// The norm in front of a KDA layer, with the residual's addition:
//   h = x + residual (rounded to the io type, as it is stored)
//   y = h / sqrt(mean_j h[j]^2 + eps) * w[j]
// in bf16 / fp32, or as e4m3 values with one fp32 scale per 128 channels (the
// operand of the block-scaled product); and its backward pass, with n = h /
// sqrt(mean h^2 + eps) and g = dy * w:
//   dx = (g - n * mean(g * n)) / sqrt(mean h^2 + eps) + d_h
//   dw = sum over tokens of dy * n
//
// HBM-bound: each row is read once and kept in registers between the row's
// sums and its outputs (but for the backward's rows of more than 16384 channels,
// below).  A row belongs to L lanes (16, 32 or whole waves), 8
// channels a lane and step (16-byte loads in bf16), NV steps; 16 lanes hold
// one scale block, so its largest value is four DPP steps.
// 131072 x 4096 in bf16 with a residual and e4m3 out: 655 us, 5.8 TB/s (a large
// copy reaches 4.8).  A single row of 4096 takes 3.0 us, the launch and one trip
// to memory.
#include <algorithm>

#include "kda_device.h"
#include "kda_internal.h"
#include "vec_io.h"

namespace kda {

namespace {

enum class Out { kBf16, kFp32, kFp8 };

// Sums of A values over the L lanes of a row, in each of them.  `parity`
// alternates between the two halves of `red`, so one barrier per call is
// enough: a wave that writes a half again has passed the barrier of the call
// in between, which every wave reaches after reading that half.
template <int L, int A>
__device__ __forceinline__ void row_sums(float (&s)[A], float (*red)[16][A], int wave, int parity) {
#pragma unroll
  for (int a = 0; a < A; ++a) {
    s[a] = lane_group_sum<16>(s[a]);
    if constexpr (L > 16) s[a] += __shfl_xor(s[a], 16);
    if constexpr (L > 32) s[a] += __shfl_xor(s[a], 32);
  }
  if constexpr (L > 64) {
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int a = 0; a < A; ++a) red[parity][wave][a] = s[a];
    __syncthreads();
#pragma unroll
    for (int a = 0; a < A; ++a) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < L / 64; ++w) t += red[parity][w][a];
      s[a] = t;
    }
  }
}

// Threads of a workgroup: a row at a time, or 256 with several rows.
constexpr int threads_of(int lanes) { return lanes < 256 ? 256 : lanes; }

}  // namespace

template <bool BF16, Out OUT, int L, int NV>
__global__ __launch_bounds__(threads_of(L)) void add_rmsnorm_kernel(
    int64_t n_rows, int hidden, const void* x, const void* res, const float* __restrict__ w, float eps, void* h,
    void* y, float* __restrict__ scale) {
  constexpr int kRows = threads_of(L) / L;   // rows at a time
  __shared__ float red[2][16][1];
  const int lane = threadIdx.x % L;
  const int nvec = hidden >> 3;
  const int nblk = (hidden + kScaleBlock - 1) / kScaleBlock;
  const float rcp = 1.0f / static_cast<float>(hidden);
  float wv[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = i * L + lane;
#pragma unroll
    for (int e = 0; e < 8; ++e) wv[i][e] = 0.f;
    if (v < nvec) load_n<false, 8>(w, static_cast<size_t>(v) * 8, wv[i]);
  }
  int parity = 0;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / L; r < n_rows;
       r += static_cast<int64_t>(gridDim.x) * kRows, parity ^= 1) {
    const size_t base = static_cast<size_t>(r) * hidden;
    float hv[NV][8];
    float ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = i * L + lane;
#pragma unroll
      for (int e = 0; e < 8; ++e) hv[i][e] = 0.f;
      if (v < nvec) {
        load_n<BF16, 8>(x, base + static_cast<size_t>(v) * 8, hv[i]);
        if (res) {
          float rv[8];
          load_n<BF16, 8>(res, base + static_cast<size_t>(v) * 8, rv);
#pragma unroll
          for (int e = 0; e < 8; ++e) hv[i][e] += rv[e];
          if constexpr (BF16) {   // the norm is of the stored sum
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const uint32_t p = pack_bf16x2(hv[i][e], hv[i][e + 1]);
              hv[i][e] = __uint_as_float(p << 16);
              hv[i][e + 1] = __uint_as_float(p & 0xffff0000u);
            }
          }
        }
        if (h) store_n<BF16, 8>(h, base + static_cast<size_t>(v) * 8, hv[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss[0] = fmaf(hv[i][e], hv[i][e], ss[0]);
      }
    }
    row_sums<L, 1>(ss, red, threadIdx.x >> 6, parity);
    const float inv = 1.0f / sqrtf(ss[0] * rcp + eps);
    float m = inv;
    const float up = OUT == Out::kFp8 ? split_power(m) : 1.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = i * L + lane;
      float t[8];
      if constexpr (OUT == Out::kFp8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = hv[i][e] * up * wv[i][e];
        float s;
        const uint2 q = quantise_block8(t, m, &s);   // whole groups of 16 lanes: zeros past the row's end
        if (v < nvec) {
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(y) + base + static_cast<size_t>(v) * 8) = q;
          if ((lane & 15) == 0) scale[static_cast<size_t>(r) * nblk + (v >> 4)] = s;
        }
      } else if (v < nvec) {
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = hv[i][e] * inv * wv[i][e];
        store_n<OUT == Out::kBf16, 8>(y, base + static_cast<size_t>(v) * 8, t);
      }
    }
  }
}

// dx of a row and the lanes' sums of dy * n over the workgroup's rows, one
// row of `part` per workgroup.  Rows go to the workgroups by a rule on the
// sizes alone and the sums are joined in a fixed order, so dw is the same in
// every run.  32768 x 4096 in bf16 with d_h: 280 us with the join, 5.7 TB/s.
// Above 16384 channels the 128 values a lane of h, dy, w and dw do not fit the
// 128 registers that 1024 lanes leave it: 131 to 133 are spilled, and the pass
// runs at half the rate (TB/s at 16384 / 16392 / 32768 channels: bf16 5.3 / 2.5 / 2.8,
// fp32 5.0 / 3.1 / 3.1; the forward 5.6 / 5.3 / 5.4 and 5.0 / 5.3 / 5.3).
template <bool H_BF16, bool DY_BF16, int L, int NV>
__global__ __launch_bounds__(threads_of(L)) void add_rmsnorm_bwd_kernel(
    int64_t n_rows, int hidden, const void* __restrict__ h, const float* __restrict__ w, float eps,
    const void* __restrict__ dy, const float* dh, float* dx, float* __restrict__ part) {
  constexpr int kRows = threads_of(L) / L;
  __shared__ float red[2][16][2];
  __shared__ float join[kRows > 1 ? kRows * NV * L * 8 : 1];
  const int lane = threadIdx.x % L;
  const int nvec = hidden >> 3;
  const float rcp = 1.0f / static_cast<float>(hidden);
  float wv[NV][8], dw[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = i * L + lane;
#pragma unroll
    for (int e = 0; e < 8; ++e) wv[i][e] = dw[i][e] = 0.f;
    if (v < nvec) load_n<false, 8>(w, static_cast<size_t>(v) * 8, wv[i]);
  }
  int parity = 0;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / L; r < n_rows;
       r += static_cast<int64_t>(gridDim.x) * kRows, parity ^= 1) {
    const size_t base = static_cast<size_t>(r) * hidden;
    float hv[NV][8], gv[NV][8];
    float s[2] = {0.f, 0.f};   // sum h^2, sum g h
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = i * L + lane;
#pragma unroll
      for (int e = 0; e < 8; ++e) hv[i][e] = gv[i][e] = 0.f;
      if (v < nvec) {
        load_n<H_BF16, 8, true>(h, base + static_cast<size_t>(v) * 8, hv[i]);
        load_n<DY_BF16, 8, true>(dy, base + static_cast<size_t>(v) * 8, gv[i]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s[0] = fmaf(hv[i][e], hv[i][e], s[0]);
        s[1] = fmaf(gv[i][e] * wv[i][e], hv[i][e], s[1]);
      }
    }
    row_sums<L, 2>(s, red, threadIdx.x >> 6, parity);
    const float inv = 1.0f / sqrtf(s[0] * rcp + eps);
    // n * mean(g n) = h * c; 0 where the squares pass fp32's range, as n is, and not an infinite sum times 0
    const float c = inv == 0.f ? 0.f : s[1] * rcp * inv * inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = i * L + lane;
      if (v < nvec) {
        float t[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dw[i][e] = fmaf(gv[i][e], hv[i][e] * inv, dw[i][e]);
          t[e] = inv * fmaf(-hv[i][e], c, gv[i][e] * wv[i][e]);
        }
        if (dh) {
          float d[8];
          load_n<false, 8>(dh, base + static_cast<size_t>(v) * 8, d);
#pragma unroll
          for (int e = 0; e < 8; ++e) t[e] += d[e];
        }
        store_n<false, 8>(dx, base + static_cast<size_t>(v) * 8, t);
      }
    }
  }
  if constexpr (kRows > 1) {   // the rows' lanes joined
    const int row = threadIdx.x / L * NV * L;
#pragma unroll
    for (int i = 0; i < NV; ++i) store_n<false, 8>(join, (row + i * L + lane) * 8, dw[i]);
    __syncthreads();
    for (int c = threadIdx.x; c < hidden; c += 256) {
      float t = 0.f;
#pragma unroll
      for (int k = 0; k < kRows; ++k) t += join[k * NV * L * 8 + c];
      part[static_cast<size_t>(blockIdx.x) * hidden + c] = t;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = i * L + lane;
      if (v < nvec) store_n<false, 8>(part, static_cast<size_t>(blockIdx.x) * hidden + static_cast<size_t>(v) * 8, dw[i]);
    }
  }
}

// out[c] = sum over p of part[p][c]: 64 columns a workgroup, 16 waves over the
// partial rows, each with eight loads in flight and a sum of its own.
__global__ __launch_bounds__(1024) void column_sums_kernel(int parts, int cols, const float* __restrict__ part,
                                                           float* __restrict__ out) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  float s[8] = {};
  if (c < cols) {
    const float* from = part + c;
    int p = wave;
    for (; p + 16 * 7 < parts; p += 16 * 8)
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] += from[static_cast<size_t>(p + 16 * i) * cols];
    for (; p < parts; p += 16) s[0] += from[static_cast<size_t>(p) * cols];
  }
  red[wave][lane] = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
  __syncthreads();
  if (wave == 0 && c < cols) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += red[i][lane];
    out[c] = t;
  }
}

hipError_t launch_column_sums(int parts, int cols, const float* part, float* out, hipStream_t st) {
  column_sums_kernel<<<dim3((cols + 63) / 64), 1024, 0, st>>>(parts, cols, part, out);
  return hipGetLastError();
}

// Calls f with the lanes per row and the steps of 8 channels a lane that hold
// a row of `hidden` channels in registers.  A wave to a row needs no barrier;
// the more lanes a row has beyond that, the more of them the odd sizes leave
// idle, but wide rows on few lanes leave few loads of other rows in flight.
// (400 MB tensors, TB/s, forward with e4m3 out / backward.  bf16: 520 channels
// on 256 lanes 2.8 / 2.2, on 64 4.8 / 5.0; 1032 4.7 / 3.7, 4.9 / 5.2; 2048
// 5.7 / 5.4, 5.4 / 4.7; 4104 on 1024 lanes 4.3 / 4.0, on 256 4.9 / 4.8; 8192
// 5.6 / 5.3, 5.2 / 4.3.  fp32: 520 5.0 / 3.5, 5.3 / 5.3; 1000 5.6 / 5.2, 5.3 /
// 5.2; 5120 5.9 / 5.2, 5.6 / 5.2.)
template <bool BF16, class F>
static hipError_t with_row_shape(int hidden, F&& f) {
  using std::integral_constant;
  if (hidden <= 128) return f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  if (hidden <= 256) return f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  if (hidden <= 512) return f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  if (hidden <= (BF16 ? 1024 : 768)) return f(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  if constexpr (BF16)
    if (hidden <= 1536) return f(integral_constant<int, 64>{}, integral_constant<int, 3>{});
  if (hidden <= 2048) return f(integral_constant<int, 256>{}, integral_constant<int, 1>{});
  if (hidden <= 4096) return f(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  if constexpr (BF16)
    if (hidden <= 6144) return f(integral_constant<int, 256>{}, integral_constant<int, 3>{});
  if (hidden <= 8192) return f(integral_constant<int, 1024>{}, integral_constant<int, 1>{});
  if (hidden <= 16384) return f(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
  return f(integral_constant<int, 1024>{}, integral_constant<int, 4>{});
}

hipError_t launch_add_rmsnorm(int64_t n, int hidden, const void* x, const void* res, const float* w, float eps,
                              void* h, void* y, float* scale, bool io_bf16, bool out_bf16, hipStream_t st) {
  auto by_io = [&](auto bf) {
    return with_row_shape<decltype(bf)::value>(hidden, [&](auto lanes, auto nv) {
      constexpr int L = decltype(lanes)::value, NV = decltype(nv)::value;
      constexpr int kRows = threads_of(L) / L;
      const int64_t blocks = (n + kRows - 1) / kRows;
      const dim3 grid(static_cast<unsigned>(blocks < 65536 ? blocks : 65536));
      auto go = [&](auto out) {
        add_rmsnorm_kernel<decltype(bf)::value, decltype(out)::value, L, NV>
            <<<grid, dim3(threads_of(L)), 0, st>>>(n, hidden, x, res, w, eps, h, y, scale);
      };
      if (scale) go(std::integral_constant<Out, Out::kFp8>{});
      else if (out_bf16) go(std::integral_constant<Out, Out::kBf16>{});
      else go(std::integral_constant<Out, Out::kFp32>{});
      return hipGetLastError();
    });
  };
  return io_bf16 ? by_io(std::true_type{}) : by_io(std::false_type{});
}

// Workgroups of the backward, each with a row of partial sums to write and to
// join: at most three a CU, and with a row at a time a whole number a CU.  One
// until three rows would share it (us, 700 x 2056 fp32: 11.9 with 256, 12.6
// with 512, 13.9 with 700), two up to 3000 rows (1200 x 4096 bf16: 20.9, 18.9,
// 19.8 with 768), then three (8000 x 4096 bf16: 115, 81, 77; 32768 x 4096: 296
// with 1024, 292 with 768).  Several rows at a time take what they fill (1600 x
// 640 bf16: 9.5 with 256, 8.8 with 400).
template <int kRows>
static int bwd_groups(int64_t n) {
  const int64_t groups = (n + kRows - 1) / kRows;
  if (kRows > 1 || groups <= 256) return static_cast<int>(std::min<int64_t>(groups, 768));
  return groups <= 768 ? 256 : groups <= 3000 ? 512 : 768;
}

int add_rmsnorm_bwd_parts(int64_t n) { return static_cast<int>(std::min<int64_t>(n, 768)); }   // the most of them

hipError_t launch_add_rmsnorm_bwd(int64_t n, int hidden, const void* h, const float* w, float eps, const void* dy,
                                  const float* dh, float* dx, float* dw, float* part, bool h_bf16, bool dy_bf16,
                                  hipStream_t st) {
  int parts = 0;
  auto by_h = [&](auto hb) {
    return with_row_shape<decltype(hb)::value>(hidden, [&](auto lanes, auto nv) {
      constexpr int L = decltype(lanes)::value, NV = decltype(nv)::value;
      constexpr int kRows = threads_of(L) / L;
      parts = bwd_groups<kRows>(n);
      if (parts == 0) return hipSuccess;
      auto go = [&](auto db) {
        add_rmsnorm_bwd_kernel<decltype(hb)::value, decltype(db)::value, L, NV>
            <<<dim3(parts), dim3(threads_of(L)), 0, st>>>(n, hidden, h, w, eps, dy, dh, dx, part);
      };
      if (dy_bf16) go(std::true_type{});
      else go(std::false_type{});
      return hipGetLastError();
    });
  };
  const hipError_t e = h_bf16 ? by_h(std::true_type{}) : by_h(std::false_type{});
  return e != hipSuccess ? e : launch_column_sums(parts, hidden, part, dw, st);
}

}  // namespace kda
