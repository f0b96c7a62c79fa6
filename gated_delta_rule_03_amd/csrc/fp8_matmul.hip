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
#include <algorithm>

#include "fp8_matmul_choice.h"
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
// For bf16 outputs one e4m3 step.  Its products are summed in eights of
// neighbouring channels (8 i .. 8 i + 7), in units of 2^-13 of the power of two
// of the largest (by the operands' exponents, -6 for subnormal ones; products
// of 0 do not count), each cut to whole units; the sums of the eights keep
// fp32's bits, rounded down (measured value by value).  An eight loses less
// than 7 units, so a row at most 7 * 2^-13 < 2^-10 of the sum of |a w| (2^-7 in
// an eight whose largest product has a subnormal operand), against the 2^-8
// that half a step of bf16 is; on Gaussian operands 1.3e-5 of the
// result's norm, with two channels in 128 a hundred times larger 4.2e-5, 1 / 130
// and 1 / 40 of what the rounding to bf16 costs.  For fp32 outputs the operands
// are widened to bf16, which holds every e4m3 value, and multiplied in four
// bf16 steps, whose sums keep fp32's bits (also between large products that
// cancel; 1e-8 measured), at half the rate.
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

// Eight consecutive outputs n .. n + 7 of one token, those below N.
template <bool BF16>
__device__ __forceinline__ void store_out8(void* y, size_t row, int n, int N, const f32x4& u, const f32x4& v) {
  if ((N & 7) == 0) {
    if (n < N) {
      const float t[8] = {u[0], u[1], u[2], u[3], v[0], v[1], v[2], v[3]};
      store_n<BF16, 8>(y, row + n, t);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (n + i < N) st<BF16>(y, row + n + i, u[i]);
      if (n + 4 + i < N) st<BF16>(y, row + n + 4 + i, v[i]);
    }
  }
}

}  // namespace

// The kernel for few tokens: 16 J outputs x 16 T tokens a workgroup, the
// operands straight from memory to registers.  Its waves share the scale
// blocks, each with U blocks' loads in flight, and join their sums in LDS in
// a fixed order.  It is bound by the weight's bytes and, as the call is short,
// by the launch and one trip to memory: 1 x 4096 x 4096 takes 5.2 us, 3.2
// TB/s, where a large copy's rate would take 3.5.
template <int J, int T, int WAVES, int U, bool OUT_BF16>
__global__ __launch_bounds__(64 * WAVES) void fp8_matmul_rows_kernel(
    int64_t M, int N, int K, const uint8_t* __restrict__ a, const float* __restrict__ sa,
    const uint8_t* __restrict__ w, const float* __restrict__ sw, void* __restrict__ y) {
  __shared__ float4 red[WAVES][J * T][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, kq = (lane >> 4) * 32;
  const int KB = (K + kScaleBlock - 1) / kScaleBlock;
  const int n0 = blockIdx.x * (16 * J);
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * (16 * T);
  const uint8_t* wrow[J];
#pragma unroll
  for (int j = 0; j < J; ++j) wrow[j] = w + static_cast<size_t>(min(n0 + 16 * j + l16, N - 1)) * K;
  const float* swrow = sw + static_cast<size_t>(n0 / kScaleBlock) * KB;
  const uint8_t* arow[T];
  const float* sarow[T];
  f32x4 acc[J][T];
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const int64_t m = m0 + 16 * t + l16 < M ? m0 + 16 * t + l16 : M - 1;
    arow[t] = a + static_cast<size_t>(m) * K;
    sarow[t] = sa + static_cast<size_t>(m) * KB;
#pragma unroll
    for (int j = 0; j < J; ++j) acc[j][t] = zero4();
  }
  // 32 channels from k on; behind the row's end any bytes of it, masked below
  auto load = [&](const uint8_t* row, int k) {
    const uint4 lo = *reinterpret_cast<const uint4*>(row + (k < K ? k : 0));
    const uint4 hi = *reinterpret_cast<const uint4*>(row + (k + 16 < K ? k + 16 : 0));
    return i32x8{static_cast<int>(lo.x), static_cast<int>(lo.y), static_cast<int>(lo.z), static_cast<int>(lo.w),
                 static_cast<int>(hi.x), static_cast<int>(hi.y), static_cast<int>(hi.z), static_cast<int>(hi.w)};
  };
  auto masked = [&](i32x8 f, int k) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = k < K ? f[i] : 0;
      f[i + 4] = k + 16 < K ? f[i + 4] : 0;
    }
    return f;
  };
  for (int b0 = wave; b0 < KB; b0 += WAVES * U) {
    i32x8 wf[U][J], af[U][T];
    float sc[U][T];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = b0 + u * WAVES, k = b * kScaleBlock + kq;
      if (b >= KB) break;
#pragma unroll
      for (int j = 0; j < J; ++j) wf[u][j] = load(wrow[j], k);
      const float s = swrow[b];
#pragma unroll
      for (int t = 0; t < T; ++t) {
        af[u][t] = load(arow[t], k);
        sc[u][t] = s * sarow[t][b];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = b0 + u * WAVES, k = b * kScaleBlock + kq;
      if (b >= KB) break;
      if ((b + 1) * kScaleBlock > K) {
#pragma unroll
        for (int j = 0; j < J; ++j) wf[u][j] = masked(wf[u][j], k);
#pragma unroll
        for (int t = 0; t < T; ++t) af[u][t] = masked(af[u][t], k);
      }
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int t = 0; t < T; ++t) {
          const f32x4 p = mfma_block<OUT_BF16>(wf[u][j], af[u][t]);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[j][t][i] = fmaf(p[i], sc[u][t], acc[j][t][i]);
        }
    }
  }
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int t = 0; t < T; ++t)
      red[wave][j * T + t][lane] = make_float4(acc[j][t][0], acc[j][t][1], acc[j][t][2], acc[j][t][3]);
  __syncthreads();
  for (int i = wave; i < J * T; i += WAVES) {
    const int j = i / T, t = i % T;
    f32x4 sum = zero4();
#pragma unroll
    for (int v = 0; v < WAVES; ++v) {
      const float4 r = red[v][i][lane];
      sum[0] += r.x; sum[1] += r.y; sum[2] += r.z; sum[3] += r.w;
    }
    const int64_t m = m0 + 16 * t + l16;
    if (m < M) store_out<OUT_BF16>(y, static_cast<size_t>(m) * N, n0 + 16 * j + 4 * (lane >> 4), N, sum);
  }
}

// The kernel for many tokens: TN x TT tiles of outputs x tokens, one after
// the other in each workgroup (one per CU), WN x WT waves.  Each scale block
// (128 channels) of the tile's rows goes to LDS straight from memory, 16 bytes
// a lane, one block ahead of the products in the other of two buffers, also
// from a tile's last block to the next one's first; one barrier per block
// hands over the buffers.  With SPLIT > 1, each of as many groups of WN x WT
// waves takes an equal part of K, and their sums are joined at the tile's end.
//
// The 256 x 256 tile (8 waves, one workgroup a CU) runs 32768 x 4096 x 4096 in
// 455 to 490 us, 2.24 to 2.4 PFLOP/s, and 128 x 128 tiles in 610; the library's
// product without block scales takes 389 to 427.  Both are bound by the clock
// that the card's power leaves on such operands (on zeros they take 362 and
// 256), and this one by the four scaled additions a lane of each product.
//
// A row's eight 16-byte pieces are stored in the order piece ^ key, with a key
// of 0 .. 7 from the row's index, which spreads the 16 rows that a product's
// operand read touches over all banks; the loads read the same 128-byte lines
// either way.
//
// The loads are written in assembly (they have no register output): the
// compiler's own form of them makes every later LDS read wait for all of
// them.  Their order against the LDS reads is the barrier below.  m0 is named
// as written, so that no value of the compiler's own is carried across in it
// (its warning about that says only that it never allocates m0).  A load that
// reads m0 needs one wait state behind a scalar write of it (s_nop 0), and five
// behind a vector instruction that wrote its scalar address, which the compiler
// does not count in front of assembly (s_nop 4).  The first form is COUNT loads
// where k < end, to LDS `step` bytes apart; its branch is inside the assembly
// so that the products around it stay one block of code, whose registers the
// compiler can place (with a branch of its own it spills).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int COUNT, int STEP>
__device__ __forceinline__ void load_lds16_if(int k, int end, uint32_t lds, const uint32_t* voff, const uint8_t* base) {
  static_assert(COUNT == 1 || COUNT == 2 || COUNT == 4, "");
  k = __builtin_amdgcn_readfirstlane(k);
  end = __builtin_amdgcn_readfirstlane(end);
  lds = __builtin_amdgcn_readfirstlane(lds);
#define KDA_LDS_FIRST \
  "s_cmp_ge_i32 %0, %1\n\ts_cbranch_scc1 .Lskip%=\n\ts_mov_b32 m0, %2\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %5, %3\n"
#define KDA_LDS_NEXT(v) "\ts_add_u32 m0, m0, %4\n\ts_nop 0\n\tglobal_load_lds_dwordx4 " v ", %3\n"
  if constexpr (COUNT == 4)
    asm volatile(KDA_LDS_FIRST KDA_LDS_NEXT("%6") KDA_LDS_NEXT("%7") KDA_LDS_NEXT("%8") ".Lskip%=:" ::"s"(k), "s"(end),
                 "s"(lds), "s"(base), "n"(STEP), "v"(voff[0]), "v"(voff[1]), "v"(voff[2]), "v"(voff[3])
                 : "memory", "scc", "m0");
  else if constexpr (COUNT == 2)
    asm volatile(KDA_LDS_FIRST KDA_LDS_NEXT("%6") ".Lskip%=:" ::"s"(k), "s"(end), "s"(lds), "s"(base), "n"(STEP),
                 "v"(voff[0]), "v"(voff[1])
                 : "memory", "scc", "m0");
  else
    asm volatile(KDA_LDS_FIRST ".Lskip%=:" ::"s"(k), "s"(end), "s"(lds), "s"(base), "n"(STEP), "v"(voff[0])
                 : "memory", "scc", "m0");
#undef KDA_LDS_FIRST
#undef KDA_LDS_NEXT
}
__device__ __forceinline__ void load_lds4(uint32_t lds, uint32_t voff, const void* base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dword %1, %2" ::"s"(lds), "v"(voff), "s"(base)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// Every load of this wave has landed and its LDS reads are done; then every
// wave's.
__device__ __forceinline__ void wait_all_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// This wave's LDS accesses are done; then every wave's.
__device__ __forceinline__ void wait_lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// The order of the tiles: workgroups go to the 8 XCDs in turn, so each XCD
// takes a run of neighbouring tiles, and within it groups of kGroup token
// tiles wide, so that the tiles running at a time share rows in its L2
// (8192 x 8192 x 8192, us: 530 row by row, 485 two wide, 470 six, 489 sixteen;
// 32768 x 16416 x 2048: 1205, 1102, 1089, 1171).
constexpr int kGroup = 6;
struct TileOrder {
  int n_tiles, t_tiles, turn;   // turn: workgroups, a multiple of 8 where they are fewer than the tiles
  // The first tile of an XCD's run: an equal part of them, and one more for the first few.
  __device__ int first(int xcd) const {
    const int tiles = n_tiles * t_tiles;
    return xcd * (tiles >> 3) + min(xcd, tiles & 7);
  }
  __device__ int count(int wg) const {
    const int left = first((wg & 7) + 1) - first(wg & 7) - (wg >> 3);
    return left <= 0 ? 0 : (left + each() - 1) / each();
  }
  __device__ int each() const { return (turn + 7) >> 3; }   // workgroups of an XCD
  __device__ int2 at(int wg, int i) const {   // (output tile, token tile)
    const int id = first(wg & 7) + (wg >> 3) + i * each();
    const int g = id / (kGroup * n_tiles), r = id - g * (kGroup * n_tiles);
    const int wide = min(kGroup, t_tiles - g * kGroup);
    return make_int2(r / wide, g * kGroup + r % wide);
  }
};

template <int TN, int TT, int WN, int WT, int SPLIT, bool OUT_BF16>
__global__ __launch_bounds__(64 * WN * WT * SPLIT, tile_waves(TN, TT, WN * WT)) void fp8_matmul_tile_kernel(
    int64_t M, int N, int K, TileOrder order, const uint8_t* __restrict__ a, const float* __restrict__ sa,
    const uint8_t* __restrict__ w, const float* __restrict__ sw, void* __restrict__ y) {
  constexpr int kWaves = WN * WT;
  constexpr int NT = TN / WN / 16, TTW = TT / WT / 16;    // 16 x 16 results of a wave
  constexpr int kRows = TN + TT;
  constexpr int kLoads = kRows / 8 / kWaves;              // 8 rows of 128 bytes a load
  constexpr int kWLoads = TN / 8 / kWaves;                // those of the weight
  // Loads are issued kBatch at every kEvery products.  Spread out where the
  // matrix cores are full (8 waves; 8192^3: 470 us, 505 in two batches), in two
  // batches where the wave's own instructions count (4 waves, 250 x 16416 x
  // 4096: 39, spread out 44).
  constexpr int kBatch = kWaves == 8 ? 1 : kWLoads, kEvery = kWaves == 8 ? 2 : 1;
  constexpr int kBuf = kRows * kScaleBlock;
  constexpr int kScaleLoads = (TT * kSteps / 64 + kWaves - 1) / kWaves;
  constexpr int kScaleBuf = TT * kSteps * 4;
  static_assert(TN % (8 * kWaves) == 0 && TT % (8 * kWaves) == 0 && kWaves % 2 == 0, "whole loads");
  static_assert(TN / WN <= kScaleBlock && kScaleBlock % (TN / WN) == 0 && (TN + kScaleBlock - 1) / kScaleBlock <= 64 / kSteps, "scales");
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem_all[];
  const int lane = threadIdx.x & 63;
  const int wave_id = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = wave_id / kWaves, wave = wave_id % kWaves;   // part of K
  const int l16 = lane & 15, grp = lane >> 4;
  const int wn = wave / WT, wt = wave % WT;
  // The scale blocks of a row, of this part, and its whole ones (with SPLIT > 1 all are).
  const int row_blocks = (K + kScaleBlock - 1) / kScaleBlock, KB = row_blocks / SPLIT;
  const int whole = SPLIT > 1 ? KB : K / kScaleBlock;

  uint8_t* const smem = smem_all + part * tile_lds(TN, TT);
  const uint32_t smem0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)smem));

  // The tile whose blocks are being loaded.
  const uint8_t* wbase;
  const uint8_t* abase;
  const float* sabase;
  const float* swbase;
  int mlast, wrows;
  uint32_t voff[kLoads];
  // This lane's piece of each load, of row 8 q + lane / 8: the weight's rows
  // have key (row % 4) + 4 (row / 8 % 2), the tokens' row % 8.
  const int piece_w = ((lane & 7) ^ (((lane >> 3) & 3) + 4 * (wave & 1))) * 16;
  const int piece_a = ((lane & 7) ^ (lane >> 3)) * 16;
  auto set_tile = [&](int2 t) {
    const int n0 = t.x * TN;
    const int64_t m0 = static_cast<int64_t>(t.y) * TT;
    wbase = w + static_cast<size_t>(n0) * K + part * KB * kScaleBlock;
    abase = a + static_cast<size_t>(m0) * K + part * KB * kScaleBlock;
    sabase = sa + static_cast<size_t>(m0) * row_blocks + part * KB;
    const int wrow0 = n0 / kScaleBlock;
    swbase = sw + static_cast<size_t>(wrow0) * row_blocks + part * KB;
    wrows = (N - 1) / kScaleBlock - wrow0;
    const int nlast = min(TN, N - n0) - 1;
    mlast = static_cast<int>(M - m0 < TT ? M - m0 : TT) - 1;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {   // rows past the tile's last are that row again
      const int row = (i * kWaves + wave) * 8 + (lane >> 3);
      voff[i] = i < kWLoads ? min(row, nlast) * static_cast<uint32_t>(K) + piece_w
                            : min(row - TN, mlast) * static_cast<uint32_t>(K) + piece_a;
    }
  };
  // kBatch loads of block kb, if there is one, to a buffer.
  auto issue = [&](int kb, int end, int buf, int i) {
    load_lds16_if<kBatch, kWaves * 8 * kScaleBlock>(kb, end, smem0 + buf + (i * kWaves + wave) * 8 * kScaleBlock,
                                                    voff + i, (i < kWLoads ? wbase : abase) + kb * kScaleBlock);
  };
  // Before a short last block is loaded: pieces beyond it are any others of the row, masked later.
  auto set_short = [&] {
    const int left = K - (KB - 1) * kScaleBlock;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int piece = i < kWLoads ? piece_w : piece_a;
      voff[i] -= piece >= left ? piece : 0;
    }
  };
  // The scales go to LDS for kSteps = 8 blocks at a time: a token's scales are
  // one run of memory, so a load of 8 tokens touches 8 lines where a load per
  // block would touch one for each token.  Each load's 64 values lie
  // [block][token], the blocks of every other load turned by one, so that the
  // 16 tokens of a read are in different banks.
  auto issue_scales = [&](int chunk, int half) {
    const int turned = min(chunk * kSteps + ((lane / 8 - (wave & 1)) & 7), KB - 1);
#pragma unroll
    for (int i = 0; i < kScaleLoads; ++i) {
      const int r0 = (i * kWaves + wave) * (64 / kSteps);
      if (TT * kSteps % (64 * kWaves) == 0 || r0 < TT)
        load_lds4(smem0 + 2 * kBuf + half * kScaleBuf + r0 * (kSteps * 4),
                  (min(r0 + lane % 8, mlast) * row_blocks + turned) * 4u, sabase);
    }
    if (wave == 0)   // [row of blocks][block]
      load_lds4(smem0 + 2 * kBuf + 2 * kScaleBuf + half * 256,
                (min(lane / kSteps, wrows) * row_blocks + min(chunk * kSteps + lane % kSteps, KB - 1)) * 4u, swbase);
  };

  // Operand reads: 16 rows, pieces grp and grp + 4 of the block.  Two groups
  // of the weight's rows take turns of four in 32 rows, so that a lane's
  // results of both are eight neighbouring outputs.
  const int off0 = (grp ^ (l16 & 7)) * 16, off1 = ((grp + 4) ^ (l16 & 7)) * 16;
  auto frag = [&](const uint8_t* row) {
    const uint4 lo = *reinterpret_cast<const uint4*>(row + off0);
    const uint4 hi = *reinterpret_cast<const uint4*>(row + off1);
    return i32x8{static_cast<int>(lo.x), static_cast<int>(lo.y), static_cast<int>(lo.z), static_cast<int>(lo.w),
                 static_cast<int>(hi.x), static_cast<int>(hi.y), static_cast<int>(hi.z), static_cast<int>(hi.w)};
  };
  const int nw = wn * (TN / WN);   // the wave's outputs lie in one scale block
  const uint8_t* wr = smem + (nw + 8 * (l16 >> 2) + (l16 & 3)) * kScaleBlock;
  const uint8_t* ar = smem + (TN + wt * (TT / WT) + l16) * kScaleBlock;
  auto frag_w = [&](int buf, int j) { return frag(wr + buf + (32 * (j >> 1) + 4 * (j & 1)) * kScaleBlock); };
  auto frag_a = [&](int buf, int t) { return frag(ar + buf + 16 * t * kScaleBlock); };
  const float* sal = reinterpret_cast<const float*>(smem + 2 * kBuf) + wt * (TT / WT) * kSteps + (l16 >> 3) * 64 + (l16 & 7);
  const float* swl = reinterpret_cast<const float*>(smem + 2 * kBuf + 2 * kScaleBuf) + nw / kScaleBlock * kSteps;
  // pieces past K of the last block hold other channels: zeros on both sides
  auto masked = [&](i32x8 f) {
    const int left = K - (KB - 1) * kScaleBlock;
    const bool k0 = grp * 16 < left, k1 = (grp + 4) * 16 < left;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = k0 ? f[i] : 0;
      f[i + 4] = k1 ? f[i + 4] : 0;
    }
    return f;
  };

  // One turn of the loop: the products of the last row group of block kb - 1,
  // then those of all but the last of block kb.  Each group's rows are read a
  // group ahead, and block kb's first operands during that leftover group, in
  // the registers that it has done with, so the matrix cores do not wait for
  // LDS at the start of a block.  At the top every wave has read all rows of
  // block kb - 1, whose buffer the loads of the next block take, and the loads
  // of block kb have landed.  (A tile's first turn has a leftover of zeros.)
  //
  // A product's scaled addition follows kLag products later, so neither waits
  // for the other; the last ones of a turn fall into the next one.  The fences
  // keep this order: left alone, the compiler puts each addition right behind
  // its product.  One product is enough where two waves of the workgroup share
  // a SIMD (32768 x 4096 x 4096, us: 489, with three 497) and where a product
  // is four steps (fp32 outputs).
  constexpr int kLag = TTW < 4 || kWaves == 8 || !OUT_BF16 ? 1 : 3, kUnits = NT * TTW;
  static_assert(NT % 2 == 0 && kUnits % (kLag + 1) == 0 && kLag <= TTW, "register slots repeat from turn to turn");
  i32x8 wf[2], af[TTW];
  f32x4 acc[NT][TTW], p[kLag + 1];
  float s[TTW], s_old[TTW];
  auto add = [&](int q, const float (&by)[TTW]) {   // product q of a block
#pragma unroll
    for (int e = 0; e < 4; ++e)
      acc[q / TTW][q % TTW][e] = fmaf(p[q % (kLag + 1)][e], by[q % TTW], acc[q / TTW][q % TTW][e]);
  };
  int buf = 0, half = 0;   // the block's buffer (byte offset) and its scales'
  // next, end: the block to load meanwhile, of the tile set by set_tile, if next < end
  auto turn = [&](int kb, int next, int end, auto is_short) {
    constexpr bool kShort = decltype(is_short)::value;
    wait_all_barrier();
    if (next < end) {
      if (next % kSteps == 0) issue_scales(next / kSteps, half ^ 1);
      if (next == whole) set_short();
    }
    const int at = half * (TT * kSteps) + ((kb + (l16 >> 3)) & 7) * 8;
    wf[0] = frag_w(buf, 0);
    const float sb = swl[half * 64 + kb % kSteps];
#pragma unroll
    for (int t = 0; t < TTW; ++t) s_old[t] = s[t];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int i = (u + kUnits - TTW) % kUnits, j = i / TTW, t = i % TTW;
      if (u >= TTW && t == 0) {
        if constexpr (kShort) wf[j & 1] = masked(wf[j & 1]);
        wf[(j + 1) & 1] = frag_w(buf, j + 1);
      }
      if (kShort && u >= TTW && u < 2 * TTW) af[t] = masked(af[t]);
      if (u % kEvery == 0 && u / kEvery * kBatch < kLoads) issue(next, end, kBuf - buf, u / kEvery * kBatch);
      __builtin_amdgcn_sched_barrier(0);
      p[i % (kLag + 1)] = mfma_block<OUT_BF16>(wf[j & 1], af[t]);
      __builtin_amdgcn_sched_barrier(0);
      if (u < TTW) {
        af[t] = frag_a(buf, t);
        s[t] = sal[at + 16 * t * kSteps] * sb;
      }
      const int q = (i + kUnits - kLag) % kUnits;
      if (u < TTW + kLag) add(q, s_old);
      else add(q, s);
    }
    buf = kBuf - buf;
    if (next % kSteps == 0) half ^= 1;
  };

  const int count = order.count(blockIdx.x);
  if (count <= 0) return;
  int2 tile = order.at(blockIdx.x, 0);
  set_tile(tile);
  if (whole == 0) set_short();
#pragma unroll
  for (int i = 0; i < kLoads; i += kBatch) issue(0, 1, 0, i);
  issue_scales(0, 0);
  for (int it = 0; it < count; ++it) {
    const int2 here = tile;
    wf[1] = i32x8{};
#pragma unroll
    for (int t = 0; t < TTW; ++t) {
      af[t] = i32x8{};
      s[t] = 0.f;
    }
#pragma unroll
    for (int i = 0; i <= kLag; ++i) p[i] = zero4();
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int t = 0; t < TTW; ++t) acc[j][t] = zero4();

    const int more = it + 1 < count;   // another tile: its first block is loaded during this one's last
    for (int kb = 0; kb < whole; ++kb) {
      const bool last = kb + 1 == KB;
      if (last && more) set_tile(tile = order.at(blockIdx.x, it + 1));
      turn(kb, last ? 0 : kb + 1, last ? more : KB, std::false_type{});
    }
    if (whole < KB) {
      if (more) set_tile(tile = order.at(blockIdx.x, it + 1));
      turn(whole, 0, more, std::true_type{});
      wf[1] = masked(wf[1]);
    }
#pragma unroll
    for (int i = kUnits - TTW; i < kUnits; ++i) {
      p[i % (kLag + 1)] = mfma_block<OUT_BF16>(wf[1], af[i % TTW]);
      add(i - kLag, s);
    }
#pragma unroll
    for (int i = kUnits - kLag; i < kUnits; ++i) add(i, s);

    if constexpr (SPLIT > 1) {
      // The parts' sums are joined, in their order, in the buffers of the
      // block just done (the others may be filling with the next tile's first).
      constexpr int kChunk = kUnits * 4 * 64 * 4;   // a wave's sums
      static_assert(kBuf % kChunk == 0 && (SPLIT - 1) * kWaves * kChunk <= SPLIT * kBuf, "room for all parts but one");
      auto chunk = [&](int c) {
        return reinterpret_cast<float*>(smem_all + c / (kBuf / kChunk) * tile_lds(TN, TT) + (kBuf - buf) +
                                        c % (kBuf / kChunk) * kChunk) + lane;
      };
      wait_lds_barrier();
      if (part) {
        float* to = chunk((part - 1) * kWaves + wave);
#pragma unroll
        for (int i = 0; i < kUnits; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) to[(i * 4 + e) * 64] = acc[i / TTW][i % TTW][e];
      }
      wait_lds_barrier();
      if (part) continue;
#pragma unroll
      for (int k = 0; k < SPLIT - 1; ++k) {
        const float* from = chunk(k * kWaves + wave);
#pragma unroll
        for (int i = 0; i < kUnits; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i / TTW][i % TTW][e] += from[(i * 4 + e) * 64];
      }
    }
    const int n0 = here.x * TN + nw + 8 * grp;
#pragma unroll
    for (int t = 0; t < TTW; ++t) {
      const int64_t m = static_cast<int64_t>(here.y) * TT + wt * (TT / WT) + 16 * t + l16;
      if (m < M) {
#pragma unroll
        for (int j = 0; j < NT; j += 2)
          store_out8<OUT_BF16>(y, static_cast<size_t>(m) * N, n0 + 16 * j, N, acc[j][t], acc[j + 1][t]);
      }
    }
  }
}

template <int TN, int TT, int WN, int WT, int SPLIT, bool OUT_BF16>
static hipError_t launch_tiles(int64_t M, int N, int K, const uint8_t* a, const float* sa, const uint8_t* w,
                               const float* sw, void* y, int ncu, hipStream_t st) {
  const auto kernel = fp8_matmul_tile_kernel<TN, TT, WN, WT, SPLIT, OUT_BF16>;
  constexpr int kLds = SPLIT * tile_lds(TN, TT);
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  if (e != hipSuccess) return e;
  TileOrder order;
  order.n_tiles = (N + TN - 1) / TN;
  order.t_tiles = static_cast<int>((M + TT - 1) / TT);
  const int64_t tiles = static_cast<int64_t>(order.n_tiles) * order.t_tiles;
  if (tiles > INT32_MAX / 2) return hipErrorInvalidValue;
  const int slots = std::max(8, ncu * tile_groups(TN, TT, WN * WT) / SPLIT / 8 * 8);
  order.turn = static_cast<int>(tiles < slots ? tiles : slots);
  kernel<<<dim3(order.turn), 64 * WN * WT * SPLIT, kLds, st>>>(M, N, K, order, a, sa, w, sw, y);
  return hipGetLastError();
}

template <int J, int T, int WAVES, int U, bool OUT_BF16>
static hipError_t launch_rows(int64_t M, int N, int K, const uint8_t* a, const float* sa, const uint8_t* w,
                              const float* sw, void* y, hipStream_t st) {
  const dim3 grid((N + 16 * J - 1) / (16 * J), static_cast<unsigned>((M + 16 * T - 1) / (16 * T)));
  fp8_matmul_rows_kernel<J, T, WAVES, U, OUT_BF16><<<grid, 64 * WAVES, 0, st>>>(M, N, K, a, sa, w, sw, y);
  return hipGetLastError();
}

template <bool OUT_BF16>
static hipError_t launch_fp8_matmul_to(int64_t M, int N, int K, const uint8_t* a, const float* sa, const uint8_t* w,
                                       const float* sw, void* y, hipStream_t st) {
  int ncu = 0;
  const hipError_t e = device_cus(&ncu);
  if (e != hipSuccess) return e;
  const Choice best = choose_fp8_matmul(OUT_BF16, M, N, K, ncu);
  if constexpr (OUT_BF16) {
    if (best.outs == 256) return launch_tiles<256, 256, 2, 4, 1, OUT_BF16>(M, N, K, a, sa, w, sw, y, ncu, st);
  }
  if (best.split == 0) {
    if (best.outs == 64) return launch_rows<4, 2, 8, 1, OUT_BF16>(M, N, K, a, sa, w, sw, y, st);
    if (best.toks == 32) return launch_rows<2, 2, 16, 1, OUT_BF16>(M, N, K, a, sa, w, sw, y, st);
    if (best.outs == 32) return launch_rows<2, 1, 16, 1, OUT_BF16>(M, N, K, a, sa, w, sw, y, st);
    // (Without a second block for the waves the shorter code is 0.3 us faster.)
    if (K <= 16 * kScaleBlock) return launch_rows<1, 1, 16, 1, OUT_BF16>(M, N, K, a, sa, w, sw, y, st);
    return launch_rows<1, 1, 16, 2, OUT_BF16>(M, N, K, a, sa, w, sw, y, st);
  }
  if (best.outs == 128) {
    if (best.split == 2) return launch_tiles<128, 128, 2, 2, 2, OUT_BF16>(M, N, K, a, sa, w, sw, y, ncu, st);
    return launch_tiles<128, 128, 2, 2, 1, OUT_BF16>(M, N, K, a, sa, w, sw, y, ncu, st);
  }
  if (best.split == 4) return launch_tiles<64, 64, 2, 2, 4, OUT_BF16>(M, N, K, a, sa, w, sw, y, ncu, st);
  if (best.split == 2) return launch_tiles<64, 64, 2, 2, 2, OUT_BF16>(M, N, K, a, sa, w, sw, y, ncu, st);
  return launch_tiles<64, 64, 2, 2, 1, OUT_BF16>(M, N, K, a, sa, w, sw, y, ncu, st);
}

hipError_t launch_fp8_matmul(int64_t M, int N, int K, const uint8_t* a, const float* sa, const uint8_t* w,
                             const float* sw, void* y, bool out_bf16, hipStream_t st) {
  return out_bf16 ? launch_fp8_matmul_to<true>(M, N, K, a, sa, w, sw, y, st)
                  : launch_fp8_matmul_to<false>(M, N, K, a, sa, w, sw, y, st);
}

}  // namespace kda
