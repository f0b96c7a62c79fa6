// What the kernels of attention over the paged 4-bit cache share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_device.h"
#include "kda_internal.h"
#include "kv_cache.h"
#include "mfma.h"
#include "vec_io.h"

namespace kda {

constexpr int kStep = 32;                   // positions of a wave's step: inside one page
constexpr int kChunkRows = 256;             // rows of a unit of the chunk kernel
constexpr float kRaise = 8.0f;              // log2 by which a score may pass the running maximum
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xff800000u); }

struct Sequence {
  int first;          // its first row of q
  int tokens;         // new tokens
  int length;         // positions held: of its length, those that the table has room for
  int base;           // positions of its length in front of the new tokens; below 0: that many tokens see nothing

  // Positions that new token j sees.  (The limit comes from the length as given: beyond the table a token sees what is held.)
  __device__ __forceinline__ uint32_t seen(int j) const {
    const int x = base + j + 1;   // at most the length as given, since j is below the number of tokens
    return static_cast<uint32_t>(x < 0 ? 0 : x < length ? x : length);
  }
};

// A value that is the same in every lane, as the compiler cannot see.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
  const uint32_t lo = uniform(static_cast<int>(x)), hi = uniform(static_cast<int>(x >> 32));
  return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}

__device__ __forceinline__ Sequence sequence(const CacheArgs& c, int n) {
  Sequence s;
  s.first = c.cu ? c.cu[n] : n;
  const int64_t end = c.cu ? c.cu[n + 1] : n + 1;
  const int64_t last = end < c.n_tokens ? end : c.n_tokens;
  s.tokens = s.first < 0 || last <= s.first ? 0 : static_cast<int>(last - s.first);
  const int64_t most = static_cast<int64_t>(c.max_pages) << c.page_shift;
  const int len = c.lengths[n];
  s.length = len < 0 ? 0 : len < most ? len : static_cast<int>(most);
  s.base = static_cast<int>((len < 0 ? 0 : len) - (end - s.first));
  return s;
}

// before[n] = sum over m < n of count(m), n = 0 .. N, at most the type's largest;
// sums: THREADS values of shared memory.  Ends with a barrier.
template <int THREADS, class T, class F>
__device__ __forceinline__ void lay_out(int N, T* before, int64_t* sums, F&& count) {
  // each thread a run of neighbouring sequences, then the threads' sums
  const int per = (N + THREADS - 1) / THREADS;
  const int n0 = threadIdx.x * per, n1 = n0 + per < N ? n0 + per : N;
  int64_t mine = 0;
  for (int n = n0; n < n1; ++n) mine += count(n);
  sums[threadIdx.x] = mine;
  __syncthreads();
  constexpr int kEach = THREADS / 64;
  if (threadIdx.x < 64) {
    int64_t front[kEach], t = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      front[i] = t;
      t += sums[threadIdx.x * kEach + i];
    }
    int64_t run = t;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const int64_t up = __shfl_up(run, m);
      if (threadIdx.x >= m) run += up;
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) sums[threadIdx.x * kEach + i] = run - t + front[i];
  }
  __syncthreads();
  constexpr int64_t kMost = static_cast<int64_t>(~static_cast<uint64_t>(0) >> (65 - 8 * sizeof(T)));
  int64_t at = sums[threadIdx.x];
  for (int n = n0; n < n1; ++n) {
    at += count(n);
    before[n + 1] = static_cast<T>(at < kMost ? at : kMost);
  }
  if (threadIdx.x == 0) before[0] = 0;
  __syncthreads();
}

// What the joining kernel has to know of a unit whose positions were shared out.
struct alignas(32) Split {
  int first, row0, rows;   // the sequence's first token; the unit's first row in it and how many are there
  int head;
  int pieces;              // 0: nothing to join
};

// A step's first bytes in the cache; the same in every lane.
struct StepAt {
  int64_t values, scales;
  bool held;
};

// The page of a position, -1 where none is held; the same in every lane.  Through
// the scalar cache: a vector load here would wait for all those in flight.
__device__ __forceinline__ int page_through_scalar(const CacheArgs& c, int seq, uint32_t pos, bool inside) {
  typedef const __attribute__((address_space(4))) int32_t* Scalar;
  const int i = static_cast<int>(pos >> c.page_shift);
  int page = -1;
  if (inside && i < c.max_pages) page = ((Scalar)(c.table + static_cast<int64_t>(seq) * c.max_pages))[i];
  return static_cast<uint32_t>(page) < static_cast<uint32_t>(c.num_pages) ? page : -1;
}

// Where a head's steps are: page_bytes apart from page to page.
template <int D>
__device__ __forceinline__ StepAt step_at(const CacheArgs& c, int seq, int64_t page_bytes, int64_t head_bytes,
                                          uint32_t pos, bool inside) {
  const int page = page_through_scalar(c, seq, pos, inside);
  const int64_t first = (page < 0 ? 0 : page) * page_bytes + head_bytes;
  const int off = static_cast<int>(pos & ((1u << c.page_shift) - 1));
  return {first + static_cast<int64_t>(off) * (D / 2), (first >> 4) + off, page >= 0};
}

__device__ __forceinline__ float scale_of(uint32_t bytes, int i) {
  return __uint_as_float(((bytes >> (8 * i)) & 0xffu) << 23);
}

template <int B>
__device__ __forceinline__ uint32_t widen(uint32_t w, float s) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, B));
}

// 8 codes as the bf16 values they stand for, in their order.
__device__ __forceinline__ bf16x8 widen8(uint32_t w, float s) {
  return __builtin_bit_cast(bf16x8, make_uint4(widen<0>(w, s), widen<1>(w, s), widen<2>(w, s), widen<3>(w, s)));
}

typedef float f32x16 __attribute__((ext_vector_type(16)));

// The log of a row's sum of exponentials, from its running maximum (in base 2) and its weights' sum.
__device__ __forceinline__ float row_lse(float m, float l) {
  return l == 0.0f ? neg_inf() : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// The chunk kernel (attention_chunk.hip), bf16 queries and outputs: workspace, launch (scale
// in base 2) and the joining of its units' parts, `stride` pieces apart.
int64_t most_chunk_units(const CacheArgs& c, int group);   // that a call can have
size_t attention_chunk_ws(int D, int64_t units);
hipError_t launch_attention_chunk(int D, const CacheArgs& c, const void* q, int group, float scale,
                                  int64_t max_rows, void* o, float* lse, void* ws, hipStream_t st);
hipError_t launch_join_parts(int D, const CacheArgs& c, int group, void* o, float* lse, const Split* joins,
                             float* pieces, int units, int stride, hipStream_t st);

}  // namespace kda
