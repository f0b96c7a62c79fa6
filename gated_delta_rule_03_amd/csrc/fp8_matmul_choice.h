// Which kernel the block-scaled product takes for its sizes (host code that
// needs no HIP headers, so that a test can ask it).
#pragma once

#include <algorithm>
#include <cstdint>

#include "e4m3.h"

namespace kda {

constexpr int kSteps = 8;   // scale blocks whose scales are loaded together, 8 tokens a load

// LDS of a tile: two buffers of operand rows, of token scales and of weight scales.
constexpr int tile_lds(int TN, int TT) { return 2 * ((TN + TT) * kScaleBlock + TT * kSteps * 4 + 256); }

// Waves of a SIMD (by their registers) and workgroups of a CU (also by LDS)
// that run at a time.
constexpr int tile_waves(int TN, int TT, int waves) { return TN * TT / waves <= 1024 ? 4 : 2; }
constexpr int tile_groups(int TN, int TT, int waves) {
  return std::min(160 * 1024 / tile_lds(TN, TT), 4 * tile_waves(TN, TT, waves) / waves);
}

// The kernel by the sizes: the one whose measured time is least.
//
// A launch of `groups` workgroups, ncu * per of which run at a time, takes
//   base + loads * each + (scale blocks of a row) * (full * whole loads + the last load's)
// where the last load costs `one` with at most a workgroup a CU, up to `full`
// with `per`.  The figures (ns) are a fit to 583 sizes of 17 to 8000 tokens,
// 256 to 16416 outputs and 512 to 8192 channels: the kernel that they pick
// takes 1.1% longer than the fastest of them on average (1.0% with fp32
// outputs).  A rows kernel of 16 outputs x 32 tokens is not among them, which
// is up to 22% faster for 17 to 32 tokens (17 x 4096 x 8192: 12.4 us, here 15.7;
// 17 x 4096 x 4096: 7.65, here 8.6).
//
// What they say: the rows kernel is the fastest while its workgroups are few
// (32 tokens, 4096 x 4096, bf16: 8.6 us, tiles 11.9; fp32, 200 tokens, 1024 x
// 4096: 11.6, tiles 17.2) and loses to the tiles' reuse beyond (128 tokens,
// 4096 x 4096, bf16: 14.9, tiles 12.5).  The parts of K pay where the tiles
// are few (256 tokens, 4096 outputs: 13.0 in four parts, 14.2 in two, 19.7
// whole; 1024 tokens in 128 x 128 tiles: 24.1 in two, 27.9 whole) and cost
// where they are many (2048 tokens: 43, 39).  fp32 outputs have no 256 x 256
// tile: with its operands widened in registers 128 x 256 took as long as 128 x
// 128 (1077, 1118 us for 32768 tokens).
struct Choice {
  int outs, toks, split;   // the workgroup's results; split 0: the rows kernel
  int base, each, full, one;
};
constexpr Choice kChoicesBf16[] = {
    {16, 16, 0, 3570, 0, 100, 0},      {32, 16, 0, 3820, 0, 151, 0},      {32, 32, 0, 3260, 370, 221, 0},
    {64, 32, 0, 3650, 0, 313, 0},      {64, 64, 4, 2900, 1650, 242, 0},   {64, 64, 2, 3550, 380, 446, 272},
    {64, 64, 1, 3520, 430, 841, 336},  {128, 128, 2, 2990, 2020, 542, 0}, {128, 128, 1, 2880, 1690, 971, 613},
    {256, 256, 1, 3160, 5080, 1418, 0}};
constexpr Choice kChoicesFp32[] = {
    {16, 16, 0, 3480, 90, 105, 0},      {32, 16, 0, 3760, 0, 159, 0},      {32, 32, 0, 2980, 640, 234, 0},
    {64, 32, 0, 3310, 290, 350, 0},     {64, 64, 4, 4850, 1870, 359, 0},   {64, 64, 2, 4880, 1070, 726, 373},
    {64, 64, 1, 4230, 1470, 1540, 465}, {128, 128, 2, 4030, 4790, 964, 0}, {128, 128, 1, 4120, 5580, 1951, 987}};

// Workgroups of a choice that a CU runs at a time.
inline int64_t choice_per_cu(const Choice& c) {
  return c.split ? tile_groups(c.outs, c.toks, c.outs == 256 ? 8 : 4) / c.split : 1;
}

inline int64_t choice_cost(const Choice& c, int64_t M, int N, int blocks, int ncu) {
  const int64_t per = choice_per_cu(c), slots = ncu * per;
  const int64_t groups = (N + c.outs - 1) / c.outs * ((M + c.toks - 1) / c.toks);
  const int64_t left = groups % slots;
  int64_t loads = groups / slots, time = loads * c.full;
  if (left) {
    const int64_t deep = (left + ncu - 1) / ncu;   // workgroups on the fullest CU
    time += deep == per ? c.full : c.one + (c.full - c.one) * (deep - 1) / (per - 1);
    ++loads;
  }
  return c.base + loads * c.each + blocks * time;
}

inline Choice choose_fp8_matmul(bool out_bf16, int64_t M, int N, int K, int ncu) {
  const int blocks = (K + kScaleBlock - 1) / kScaleBlock;
  const Choice& rows_16x16 = out_bf16 ? kChoicesBf16[0] : kChoicesFp32[0];
  const Choice& rows_32x16 = out_bf16 ? kChoicesBf16[1] : kChoicesFp32[1];
  // One load of the smallest groups is the least of every figure.  With up to
  // 16 tokens the rows kernels share no tokens, and what counts beyond is the
  // stream of the weight: many short loads for a few tokens and a long K (1 x
  // 16416 x 4096: 14.1 us, with 32 outputs a workgroup 17.0; x 2048 9.1, 8.8),
  // fewer reads of the tokens for more of them (16 x 16416 x 4096: 24.3, 21.3).
  const bool one_load = (M + 15) / 16 * ((N + 15) / 16) <= ncu;
  if (one_load || (M < 8 && blocks >= 32)) return rows_16x16;
  if (M <= 16) return rows_32x16;
  int64_t least = INT64_MAX;
  Choice best{};
  const auto weigh = [&](const Choice& c) {
    if (c.split == 0 && M > 4096) return;   // (the grid's second axis)
    // equal parts of K, of four blocks or more
    if (c.split > 1 && (K % (kScaleBlock * c.split) || blocks < 4 * c.split)) return;
    const int64_t cost = choice_cost(c, M, N, blocks, ncu);
    if (cost < least) {
      least = cost;
      best = c;
    }
  };
  if (out_bf16)
    for (const Choice& c : kChoicesBf16) weigh(c);
  else
    for (const Choice& c : kChoicesFp32) weigh(c);
  return best;
}

}  // namespace kda
