// The layer's projections in 8 bits: y = a w^T with e4m3 operands, one fp32
// scale per token and 128 channels (a) and per 128 x 128 block (w):
//   y[m][n] = sum_b sa[m][b] sw[n / 128][b] sum_{k in block b} a[m][k] w[n][k]
// The inner sum of a scale block is one v_mfma_f32_16x16x128 step (K = 128);
// its four fp32 results a lane are scaled and added on the vector ALU.  The
// weight's rows are the step's M side and the tokens its N side, so a lane's
// four results are four consecutive outputs of one token and share one scale
// sa[m][b] * sw.
//
// Operand layout of the step: lane l holds row (or column) l % 16, channels
// 32 * (l / 16) .. + 31; both sides use the same order of channels, so any
// other assignment of channels to lanes gives the same product.  Result: lane
// l holds D[4 * (l / 16) + i][l % 16], i < 4.
#include "kda_device.h"
#include "kda_internal.h"
#include "vec_io.h"

namespace kda {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// Eight e4m3 values as bf16 (exact).
__device__ __forceinline__ bf16x8 widen(int lo, int hi) {
  const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// The product of one scale block, 16 x 128 times 128 x 16.
//
// For bf16 outputs one e4m3 step.  The matrix cores align the products of an
// e4m3 step to the largest one and drop what lies below 2^-13 of it (measured;
// the K = 32 form does the same): 1.3e-5 of the result's norm, 1 / 100 of what
// the output's own rounding costs.  For fp32 outputs the operands are widened
// to bf16, which holds every e4m3 value, and multiplied in four bf16 steps,
// whose sums keep fp32's bits (1e-8 measured), at half the rate.
template <bool FAST>
__device__ __forceinline__ f32x4 mfma_block(const i32x8& a, const i32x8& b) {
  if constexpr (FAST) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero4(), 0, 0, 0, 0, 0, 0);
  } else {
    f32x4 c = zero4();
#pragma unroll
    for (int i = 0; i < 8; i += 2) c = mfma(widen(a[i], a[i + 1]), widen(b[i], b[i + 1]), c);
    return c;
  }
}

// 32 channels of a row from channel k on, zeros past its end (rows are whole
// runs of 16).
__device__ __forceinline__ i32x8 load_frag(const uint8_t* row, int k, int K) {
  const uint4 z = make_uint4(0, 0, 0, 0);
  const uint4 lo = k < K ? *reinterpret_cast<const uint4*>(row + k) : z;
  const uint4 hi = k + 16 < K ? *reinterpret_cast<const uint4*>(row + k + 16) : z;
  return i32x8{static_cast<int>(lo.x), static_cast<int>(lo.y), static_cast<int>(lo.z), static_cast<int>(lo.w),
               static_cast<int>(hi.x), static_cast<int>(hi.y), static_cast<int>(hi.z), static_cast<int>(hi.w)};
}

// Four consecutive outputs n .. n + 3 of one token, those below N.
template <bool BF16>
__device__ __forceinline__ void store_out(void* y, size_t row, int n, int N, const f32x4& v) {
  if ((N & 3) == 0) {
    if (n < N) {
      const float t[4] = {v[0], v[1], v[2], v[3]};
      store_n<BF16, 4>(y, row + n, t);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) st<BF16>(y, row + n + i, v[i]);
  }
}

}  // namespace

// 16 outputs x 16 T tokens a workgroup; its waves share the scale blocks and
// join their sums in LDS in a fixed order.
template <int T, int WAVES, bool OUT_BF16>
__global__ __launch_bounds__(64 * WAVES) void fp8_matmul_rows_kernel(
    int64_t M, int N, int K, const uint8_t* __restrict__ a, const float* __restrict__ sa,
    const uint8_t* __restrict__ w, const float* __restrict__ sw, void* __restrict__ y) {
  __shared__ float4 red[WAVES][T][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, kq = (lane >> 4) * 32;
  const int KB = (K + kScaleBlock - 1) / kScaleBlock;
  const int n0 = blockIdx.y * 16;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * (16 * T);
  const uint8_t* wrow = w + static_cast<size_t>(min(n0 + l16, N - 1)) * K;
  const float* swrow = sw + static_cast<size_t>(n0 / kScaleBlock) * KB;
  int64_t tok[T];
  f32x4 acc[T];
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const int64_t m = m0 + 16 * t + l16;
    tok[t] = m < M ? m : M - 1;
    acc[t] = zero4();
  }
  for (int b = wave; b < KB; b += WAVES) {
    const int k = b * kScaleBlock + kq;
    const i32x8 wf = load_frag(wrow, k, K);
    const float s = swrow[b];
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const i32x8 af = load_frag(a + static_cast<size_t>(tok[t]) * K, k, K);
      const float sc = s * sa[static_cast<size_t>(tok[t]) * KB + b];
      const f32x4 p = mfma_block<OUT_BF16>(wf, af);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][i] = fmaf(p[i], sc, acc[t][i]);
    }
  }
#pragma unroll
  for (int t = 0; t < T; ++t) red[wave][t][lane] = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
  __syncthreads();
  for (int t = wave; t < T; t += WAVES) {
    f32x4 v = zero4();
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
      const float4 r = red[i][t][lane];
      v[0] += r.x; v[1] += r.y; v[2] += r.z; v[3] += r.w;
    }
    const int64_t m = m0 + 16 * t + l16;
    if (m < M) store_out<OUT_BF16>(y, static_cast<size_t>(m) * N, n0 + 4 * (lane >> 4), N, v);
  }
}

// The kernel for many tokens: a TN x TT tile of outputs x tokens per
// workgroup, WN x WT waves.  Each scale block (128 channels) of the tile's
// rows goes to LDS straight from memory, 16 bytes a lane, one block ahead of
// the products in the other of two buffers, so one barrier per block is
// enough.  A row's eight 16-byte pieces are stored in the order piece ^ (row
// % 8), which spreads the 16 rows that a product's operand read touches over
// all banks; the loads read the same 128-byte lines either way.
//
// The loads are written in assembly (they have no register output): the
// compiler's own form of them makes every later LDS read wait for all of
// them.  Their order against the LDS reads is the barrier below.
__device__ __forceinline__ void load_lds16(uint32_t lds, uint32_t voff, const uint8_t* base) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(voff), "s"(base) : "memory", "m0");
}

// Every load of this wave has landed and its LDS reads are done; then every
// wave's.
__device__ __forceinline__ void wait_all_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

template <int TN, int TT, int WN, int WT, bool OUT_BF16>
__global__ __launch_bounds__(64 * WN * WT) void fp8_matmul_tile_kernel(
    int64_t M, int N, int K, int n_tiles, int64_t tiles, const uint8_t* __restrict__ a, const float* __restrict__ sa,
    const uint8_t* __restrict__ w, const float* __restrict__ sw, void* __restrict__ y) {
  constexpr int kWaves = WN * WT;
  constexpr int NT = TN / WN / 16, TTW = TT / WT / 16;    // 16 x 16 results of a wave
  constexpr int kRows = TN + TT;
  constexpr int kLoads = kRows / 8 / kWaves;              // 8 rows of 128 bytes a load
  constexpr int kBuf = kRows * kScaleBlock;
  static_assert(kRows % (8 * kWaves) == 0 && TN / WN <= kScaleBlock && kScaleBlock % (TN / WN) == 0, "tile shape");
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const uint32_t smem0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)smem));

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, grp = lane >> 4;
  const int wn = wave / WT, wt = wave % WT;
  const int KB = (K + kScaleBlock - 1) / kScaleBlock;

  // workgroups go to the 8 XCDs in turn: each XCD takes a run of neighbouring tiles
  int64_t id = blockIdx.x;
  {
    const int64_t per = tiles / 8;
    if (id < per * 8) id = (id & 7) * per + (id >> 3);
  }
  const int tn = static_cast<int>(id % n_tiles);
  const int64_t tt = id / n_tiles;
  const int n0 = tn * TN;
  const int64_t m0 = tt * TT;

  const uint8_t* wbase = w + static_cast<size_t>(n0) * K;
  const uint8_t* abase = a + static_cast<size_t>(m0) * K;
  const int nlast = min(TN, N - n0) - 1;
  const int mlast = static_cast<int>(M - m0 < TT ? M - m0 : TT) - 1;

  // this lane's piece of each load: row 8 i + lane / 8, piece (lane % 8) ^ (row % 8)
  const int piece = ((lane & 7) ^ (lane >> 3)) * 16;
  uint32_t voff[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int row = (i * kWaves + wave) * 8 + (lane >> 3);   // a load is within one operand: TN is a multiple of 8
    voff[i] = (row < TN ? min(row, nlast) : min(row - TN, mlast)) * static_cast<uint32_t>(K) + piece;
  }
  auto issue = [&](int kb, int buf) {
    const bool past = kb * kScaleBlock + piece >= K;   // beyond a short last block: any byte of the row, masked later
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int r0 = (i * kWaves + wave) * 8;
      const uint8_t* base = (r0 < TN ? wbase : abase) + kb * kScaleBlock;
      load_lds16(smem0 + buf * kBuf + r0 * kScaleBlock, past ? voff[i] - piece : voff[i], base);
    }
  };

  // operand reads: rows l16 of a 16-row group, pieces grp and grp + 4 of the block
  const int rd0 = l16 * kScaleBlock + ((grp ^ (l16 & 7)) * 16);
  const int rd1 = l16 * kScaleBlock + (((grp + 4) ^ (l16 & 7)) * 16);
  auto frag = [&](const uint8_t* rows) {
    const uint4 lo = *reinterpret_cast<const uint4*>(rows + rd0);
    const uint4 hi = *reinterpret_cast<const uint4*>(rows + rd1);
    return i32x8{static_cast<int>(lo.x), static_cast<int>(lo.y), static_cast<int>(lo.z), static_cast<int>(lo.w),
                 static_cast<int>(hi.x), static_cast<int>(hi.y), static_cast<int>(hi.z), static_cast<int>(hi.w)};
  };
  // pieces past K of the last block hold other channels: zeros on both sides
  auto masked = [&](i32x8 f, int kb) {
    const bool k0 = kb * kScaleBlock + grp * 16 < K, k1 = kb * kScaleBlock + (grp + 4) * 16 < K;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = k0 ? f[i] : 0;
      f[i + 4] = k1 ? f[i + 4] : 0;
    }
    return f;
  };

  const float* sap[TTW];
  float sa_next[TTW];
#pragma unroll
  for (int t = 0; t < TTW; ++t) {
    const int m = min(wt * (TT / WT) + 16 * t + l16, mlast);
    sap[t] = sa + static_cast<size_t>(m0 + m) * KB;
    sa_next[t] = sap[t][0];
  }
  const int nw = n0 + wn * (TN / WN);   // the wave's outputs lie in one scale block
  const float* swp = sw + static_cast<size_t>(min(nw, N - 1) / kScaleBlock) * KB;

  f32x4 acc[NT][TTW];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int t = 0; t < TTW; ++t) acc[j][t] = zero4();

  auto step = [&](int kb, auto last_short) {
    wait_all_barrier();
    float s[TTW];
    const float sb = swp[kb];
#pragma unroll
    for (int t = 0; t < TTW; ++t) {
      s[t] = sa_next[t] * sb;
      asm volatile("" : "+v"(s[t]));   // used up before the loads below are counted
    }
    if (kb + 1 < KB) {
      issue(kb + 1, (kb + 1) & 1);
#pragma unroll
      for (int t = 0; t < TTW; ++t) sa_next[t] = sap[t][kb + 1];
    }
    const uint8_t* buf = smem + (kb & 1) * kBuf;
    const uint8_t* wr = buf + wn * (TN / WN) * kScaleBlock;
    const uint8_t* ar = buf + (TN + wt * (TT / WT)) * kScaleBlock;
    i32x8 af[TTW];
#pragma unroll
    for (int t = 0; t < TTW; ++t) {
      af[t] = frag(ar + t * 16 * kScaleBlock);
      if constexpr (decltype(last_short)::value) af[t] = masked(af[t], kb);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      i32x8 wf = frag(wr + j * 16 * kScaleBlock);
      if constexpr (decltype(last_short)::value) wf = masked(wf, kb);
#pragma unroll
      for (int t = 0; t < TTW; ++t) {
        const f32x4 p = mfma_block<OUT_BF16>(wf, af[t]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][t][i] = fmaf(p[i], s[t], acc[j][t][i]);
      }
    }
  };
  issue(0, 0);
  const int whole = K / kScaleBlock;
  for (int kb = 0; kb < whole; ++kb) step(kb, std::false_type{});
  if (whole < KB) step(whole, std::true_type{});

#pragma unroll
  for (int t = 0; t < TTW; ++t) {
    const int m = wt * (TT / WT) + 16 * t + l16;
    if (m > mlast) continue;
#pragma unroll
    for (int j = 0; j < NT; ++j)
      store_out<OUT_BF16>(y, static_cast<size_t>(m0 + m) * N, nw + 16 * j + 4 * grp, N, acc[j][t]);
  }
}

template <int TN, int TT, int WN, int WT, bool OUT_BF16>
static hipError_t launch_tiles(int64_t M, int N, int K, const uint8_t* a, const float* sa, const uint8_t* w,
                               const float* sw, void* y, hipStream_t st) {
  const auto kernel = fp8_matmul_tile_kernel<TN, TT, WN, WT, OUT_BF16>;
  constexpr int kLds = 2 * (TN + TT) * kScaleBlock;
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  if (e != hipSuccess) return e;
  const int n_tiles = (N + TN - 1) / TN;
  const int64_t tiles = n_tiles * ((M + TT - 1) / TT);
  kernel<<<dim3(static_cast<unsigned>(tiles)), 64 * WN * WT, kLds, st>>>(M, N, K, n_tiles, tiles, a, sa, w, sw, y);
  return hipGetLastError();
}

template <bool OUT_BF16>
static hipError_t launch_fp8_matmul_to(int64_t M, int N, int K, const uint8_t* a, const float* sa, const uint8_t* w,
                                       const float* sw, void* y, hipStream_t st) {
  if (M > 64) return launch_tiles<256, 256, 2, 4, OUT_BF16>(M, N, K, a, sa, w, sw, y, st);
  const dim3 grid(static_cast<unsigned>((M + 63) / 64), (N + 15) / 16);
  fp8_matmul_rows_kernel<4, 8, OUT_BF16><<<grid, 512, 0, st>>>(M, N, K, a, sa, w, sw, y);
  return hipGetLastError();
}

hipError_t launch_fp8_matmul(int64_t M, int N, int K, const uint8_t* a, const float* sa, const uint8_t* w,
                             const float* sw, void* y, bool out_bf16, hipStream_t st) {
  return out_bf16 ? launch_fp8_matmul_to<true>(M, N, K, a, sa, w, sw, y, st)
                  : launch_fp8_matmul_to<false>(M, N, K, a, sa, w, sw, y, st);
}

}  // namespace kda
