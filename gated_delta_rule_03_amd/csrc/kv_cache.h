// A paged cache of 4-bit keys and values: where a call's rows are in it.
// Every index that comes from the device (sequence offsets, lengths, page
// numbers) is checked against its range before it is used.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_internal.h"

namespace kda {

constexpr int kMxBlock = 32;    // channels that share an e8m0 scale
constexpr int kScaleNaN = 255;  // the byte of a block with a NaN or an infinity

// The sequence of a call's row and the position it stands for; seq -1: no sequence's.
struct RowAt {
  int seq;
  int64_t pos;
};

__device__ __forceinline__ RowAt row_at(const CacheArgs& c, int64_t row) {
  if (!c.cu) return row < c.N ? RowAt{static_cast<int>(row), static_cast<int64_t>(c.lengths[row]) - 1} : RowAt{-1, 0};
  if (row >= c.cu[c.N]) return {-1, 0};
  int lo = 0, hi = c.N;   // cu[lo] <= row (taken as given for 0), cu[hi] > row
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (c.cu[mid] <= row) lo = mid;
    else hi = mid;
  }
  return {lo, static_cast<int64_t>(c.lengths[lo]) - (static_cast<int64_t>(c.cu[lo + 1]) - row)};
}

// The page of a position, or -1 where none is held.
__device__ __forceinline__ int page_of(const CacheArgs& c, int seq, int64_t pos) {
  if (pos < 0) return -1;
  const int64_t i = pos >> c.page_shift;
  if (i >= c.max_pages) return -1;
  const int page = c.table[static_cast<size_t>(seq) * c.max_pages + i];
  return static_cast<uint32_t>(page) < static_cast<uint32_t>(c.num_pages) ? page : -1;
}

// Byte offsets of a head's rows in a page: values, and the scales of its first block.
template <int D>
__device__ __forceinline__ size_t values_at(const CacheArgs& c, int page, int head) {
  return (static_cast<size_t>(page) * c.heads + head) * (D / 2) << c.page_shift;
}
template <int D>
__device__ __forceinline__ size_t scales_at(const CacheArgs& c, int page, int head) {
  return (static_cast<size_t>(page) * c.heads + head) * (D / kMxBlock) << c.page_shift;
}

}  // namespace kda
