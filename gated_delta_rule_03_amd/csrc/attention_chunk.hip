// Attention over the paged 4-bit cache for chunks of many new tokens, bf16
// queries and outputs.  The matrix cores' and vector units' time counts here, so
// values are widened once for a whole workgroup:
//
// A workgroup has 8 waves of 32 rows (rows are a sequence's new tokens times the
// query heads of one key head) and walks the positions in blocks.  Everything
// comes through LDS: keys and values go there from memory as they are, without
// registers, three and four blocks ahead (all workgroups of an XCD touch a block
// for the first time together, so a block's bytes come from far away); while a
// block is worked on, some of the lanes widen the next one's values to bf16 and
// leave them in the order in which the matrix cores' operands read them; one
// barrier a block.  Keys stay in their 4 bits there, and each wave widens what it
// multiplies (four conversions a step; shared in bf16 they would not fit the LDS at
// 256 channels).  16-byte pieces of neighbouring keys lie permuted, so that eight lanes'
// reads have no bank conflict.
//   S^T = K Q^T, O^T += V^T P^T   (32 positions x 32 rows, 32x32x16 steps)
// A weight is two bf16 values (attention.hip), the smaller one multiplied first.
// Lane l has row l % 32 of S^T at positions 8 b + 4 (l / 32) + i, and P^T's
// operand takes them in that order, so weights stay in their lane.  Channel
// 8 / NC of tile c's row r is r * NC + c (NC = D / 32 tiles): what a lane widens,
// 8 neighbouring channels of 8 positions, then goes to 8 neighbouring rows' or
// tiles' places.  Two waves a SIMD (four at 64 channels, two workgroups), so that
// one's softmax runs under the other's products.  Two chunks of 2048 tokens of 16384
// positions, 16 query heads on 2 key heads of 256: 1270 us, 0.81 PFLOP/s of the
// formula's products (half as many again are made for the second halves of the
// weights; matrix cores 51% busy, vector units 40); 32 on 8 of 128: 1398, 0.73; of
// 64: 860, 0.60.
//
// A workgroup takes one (sequence, key head, row tile), the last tiles (which
// see the most) first, or one of up to `splits` equal parts of its positions
// where the tiles do not fill the CUs; the parts meet in the join kernel.
#include <algorithm>

#include "attention.h"

namespace kda {

namespace {

constexpr int kChunkWaves = kChunkRows / 32;

__device__ __forceinline__ f32x16 mfma32(const bf16x8& a, const bf16x8& b, const f32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Loads from memory to LDS without registers: 16 bytes (4) a lane, lane l's to
// lds + 16 l (4 l).  The wait is in lds_barrier.  (The compiler's own form waits
// for such a load in front of every LDS read.)  A load reads m0 five wait states
// behind its scalar write at the earliest here.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_lds16(uint32_t lds, const uint8_t* base, uint32_t lane_offset) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(uniform(static_cast<int>(lds))), "v"(lane_offset),
               "s"(uniform(static_cast<int64_t>(reinterpret_cast<uintptr_t>(base))))
               : "memory", "m0");
}
__device__ __forceinline__ void load_lds4(uint32_t lds, const uint8_t* lane_address) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dword %1, off" ::"s"(uniform(static_cast<int>(lds))), "v"(lane_address)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// The wave's LDS accesses done and at most `in_flight` of its loads left (0, 2 ..
// 6 of them: the last ones issued), then the workgroup's barrier.  Loads that the
// compiler adds only make the wait a longer one.
__device__ __forceinline__ void lds_barrier(int in_flight) {
  if (in_flight == 6) asm volatile("s_waitcnt vmcnt(6)" ::: "memory");
  else if (in_flight == 4) asm volatile("s_waitcnt vmcnt(4)" ::: "memory");
  else if (in_flight == 2) asm volatile("s_waitcnt vmcnt(2)" ::: "memory");
  else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const uint8_t*)p));
}

// Pages of a block's steps; -1: not held.
struct Pages {
  int x0, x1, x2, x3;
  // (the values pass through readfirstlane, so that choosing among them is no
  // load at an address computed at run time, which would keep them in memory)
  __device__ __forceinline__ int of(int step) const {
    const int a = uniform(x0), b = uniform(x1), c = uniform(x2), d = uniform(x3);
    return step < 2 ? (step == 0 ? a : b) : (step == 2 ? c : d);
  }
  __device__ __forceinline__ bool any_missing(int steps) const {
    return uniform(steps == 2 ? x0 | x1 : x0 | x1 | x2 | x3) < 0;
  }
};

// What a kernel of D channels keeps in LDS.
template <int D>
struct ChunkShape {
  static constexpr int kPos = D == 256 ? 64 : 128;       // positions of a block
  static constexpr int kSteps = kPos / kStep;
  static constexpr int kLeast = 3;                       // blocks of a part: its rows' sums are written and read again
  static constexpr int kAhead = 4;                       // blocks' raw bytes in LDS
  static constexpr int kAtOnce = D == 256 ? 1 : 2;       // steps whose scores a wave forms together
  static constexpr int kRowBytes = D / 2;
  static constexpr int kRaw = kPos * kRowBytes;          // bytes of a block's keys, of its values
  static constexpr int kScales = D / 32 * kPos;
  static constexpr int kWide = kPos * D * 2;
  static constexpr int kChunks = kRaw / 1024;            // loads of a wave each
  static constexpr int kStepChunks = kStep * kRowBytes / 1024;
  static constexpr int kScaleLoads = kScales / 256;
  static constexpr int kTaskLanes = D / 2;               // lanes that widen a step
  static constexpr int kTaskWaves = kSteps * kTaskLanes / 64;
  uint8_t wide[2][kWide];
  uint8_t k[kAhead][kRaw], v[kAhead][kRaw], ks[kAhead][kScales], vs[kAhead][kScales];
  int bad[2][kChunkWaves];
  // where 16-byte piece x of a key is, within its row
  static __device__ __forceinline__ int piece(int row, int x) {
    const int turn = D == 256 ? row & 7 : D == 128 ? (row >> 1) & 3 : (row >> 2) & 1;
    return x ^ turn;
  }
};

}  // namespace

// (64 channels: registers for four waves a SIMD, so that two workgroups fit a CU: 2 x 2048 tokens of 16384 positions, 32
// heads on 8: 1031 -> 909 us.)
template <int D>
__global__ __launch_bounds__(kChunkWaves * 64, D == 64 ? 4 : 2) void attention_chunk_kernel(CacheArgs c, const void* __restrict__ q, int group,
                                                                    float scale, int splits, int units,
                                                                    void* __restrict__ o, float* __restrict__ lse,
                                                                    Split* __restrict__ joins,
                                                                    float* __restrict__ pieces) {
  using S = ChunkShape<D>;
  constexpr int W = kChunkWaves;
  constexpr int kRows = kChunkRows;
  constexpr int NC = D / 32;              // channel tiles
  constexpr int kBlocks = D / 64;         // blocks of 32 channels of a lane's half of a head
  static_assert(S::kChunks <= W && 2 * S::kScaleLoads <= W && S::kTaskWaves <= W, "a load, a word a wave");
  __shared__ alignas(1024) S sm;
  extern __shared__ int32_t before[];     // [N + 1]: tiles in front of each sequence
  const int lane = threadIdx.x & 63, wave = uniform(static_cast<int>(threadIdx.x >> 6)), row32 = lane & 31, h = lane >> 5;
  const int Hq = c.heads * group;
  const uint32_t flip = scale < 0.0f ? 0x80008000u : 0u;
  scale = fminf(fmaxf(fabsf(scale), 1.17549435e-38f), 3.4028235e38f);

  lay_out<W * 64>(c.N, before, reinterpret_cast<int64_t*>(sm.wide), [&](int n) {
    return (static_cast<int64_t>(sequence(c, n).tokens) * group + kRows - 1) / kRows;
  });
  if (splits > 1 && threadIdx.x == 0)   // (those that there are: by their first part)
    for (int64_t i = static_cast<int64_t>(before[c.N]) * c.heads + blockIdx.x; i < units; i += gridDim.x) joins[i].pieces = 0;
  // the workgroup's unit and part.  Workgroups go to the XCDs in turn, and a
  // sequence's units are numbered head by head, the last tiles (which see the most)
  // of all heads first: an XCD has few heads, whose keys and values its workgroups
  // share in its cache, as much to do as the others, and its short units at the end
  // (one chunk of 8192 tokens, 2 key heads of 256: 690 us, 8 of 128: 790.  In a form
  // with cheaper products 505, with an eighth of the line of heads and tiles to each
  // XCD 817; 588, with the tiles of one head after the other over all XCDs 790.)
  const int64_t there = static_cast<int64_t>(before[c.N]) * c.heads;
  const int n_units = uniform(static_cast<int>(there < units ? there : units));
  const int place = blockIdx.x;
  if (place >= n_units * splits) return;
  const int part = uniform(place / n_units), id = uniform(place - part * n_units);
  int n = 0;
  for (int hi = c.N; hi - n > 1;) {   // the last with its tiles' first unit <= id
    const int mid = (n + hi) >> 1;
    if (static_cast<int64_t>(before[mid]) * c.heads <= id) n = mid;
    else hi = mid;
  }
  n = uniform(n);
  const Sequence s = sequence(c, n);
  const int rows = s.tokens * group;
  const int tiles = (rows + kRows - 1) / kRows;
  const int local = uniform(static_cast<int>(id - static_cast<int64_t>(before[n]) * c.heads));
  const int turn = uniform(local / c.heads), head = local - turn * c.heads, tile = tiles - 1 - turn;
  __syncthreads();   // (sm.wide held lay_out's sums)

  auto seen = [&](int row) { return s.seen(row / group); };   // positions that a row sees
  auto seen_by = [&](int row) { return static_cast<uint32_t>(uniform(static_cast<int>(seen(row)))); };   // of a scalar
  const int wave_row = tile * kRows + wave * 32;
  const int row = wave_row + row32;
  const int r = row < rows ? row : rows - 1;
  const uint32_t sees = seen(r);
  // positions that every row of the wave sees, that any does, and the same of the workgroup
  const uint32_t least = seen_by(wave_row < rows ? wave_row : rows - 1);
  const uint32_t most = wave_row < rows ? seen_by((wave_row + 32 < rows ? wave_row + 32 : rows) - 1) : 0;
  const uint32_t least_all = seen_by(tile * kRows);
  const uint32_t most_all = seen_by(((tile + 1) * kRows < rows ? (tile + 1) * kRows : rows) - 1);

  // queries: step i takes channels h * D / 2 + 8 i ..
  bf16x8 qv[D / 16];
  {
    const int t = r / group;
    const size_t from = (static_cast<size_t>(s.first + t) * Hq + head * group + (r - t * group)) * D + h * (D / 2);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(q) + from + 8 * i);
      w.x ^= flip;
      w.y ^= flip;
      w.z ^= flip;
      w.w ^= flip;
      qv[i] = __builtin_bit_cast(bf16x8, w);
    }
  }

  const int64_t page_bytes = static_cast<int64_t>(c.heads) * (D / 2) << c.page_shift;
  const int64_t head_bytes = static_cast<int64_t>(head) * (D / 2) << c.page_shift;
  // the part's blocks
  const int blocks = c.num_pages > 0 ? static_cast<int>((static_cast<int64_t>(most_all) + S::kPos - 1) / S::kPos) : 0;
  const int shares = blocks < S::kLeast * splits ? (blocks < 2 * S::kLeast ? 1 : blocks / S::kLeast) : splits;
  if (part >= shares) return;
  const int b0 = uniform(static_cast<int>(static_cast<int64_t>(blocks) * part / shares));
  const int b1 = uniform(static_cast<int>(static_cast<int64_t>(blocks) * (part + 1) / shares));

  auto pages_of = [&](int b) {
    const uint32_t pos = static_cast<uint32_t>(b) * S::kPos;
    Pages p = {-1, -1, -1, -1};
    p.x0 = page_through_scalar(c, n, pos, b < b1);
    p.x1 = page_through_scalar(c, n, pos + kStep, b < b1);
    if constexpr (S::kSteps == 4) {
      p.x2 = page_through_scalar(c, n, pos + 2 * kStep, b < b1);
      p.x3 = page_through_scalar(c, n, pos + 3 * kStep, b < b1);
    }
    return p;
  };
  // the first bytes of a block's step: values, and scales
  const uint32_t in_page = (1u << c.page_shift) - 1;
  auto scales_of = [&](int page, int b, int step) {
    const uint32_t off = (static_cast<uint32_t>(b) * S::kPos + step * kStep) & in_page;
    return (((page < 0 ? 0 : page) * page_bytes + head_bytes) >> 4) + off;
  };
  // The lane's number, anew: what is derived from it is then formed where it is
  // used.  Kept across the steps it would not fit the registers (256 channels),
  // and what is read back from scratch waits for the loads in flight.
  auto lane_anew = [&] {
    int l = lane;
    asm volatile("" : "+v"(l));
    return l;
  };
  // a block's keys (values) and their scales to LDS: 1 KB a wave, and 256 bytes
  auto fetch = [&](const Pages& p, int b, bool keys, int buf) {
    if (b >= b1) return;
    const int l = lane_anew();
    if (wave < S::kChunks) {
      const int step = wave / S::kStepChunks;
      const int page = p.of(step);
      const uint32_t off = (static_cast<uint32_t>(b) * S::kPos + step * kStep) & in_page;
      const int64_t from = (page < 0 ? 0 : page) * page_bytes + head_bytes + static_cast<int64_t>(off) * S::kRowBytes +
                           wave % S::kStepChunks * 1024;
      const int row = l * 16 / S::kRowBytes, piece = l * 16 % S::kRowBytes / 16;
      load_lds16(lds_offset(keys ? sm.k[buf] : sm.v[buf]) + wave * 1024, (keys ? c.k : c.v) + from,
                 keys ? row * S::kRowBytes + S::piece(row, piece) * 16 : l * 16);
    }
    const int w = keys ? wave : wave - W / 2;
    if (w >= 0 && w < S::kScaleLoads) {
      const int at = (w * 64 + l) * 4, block = at / S::kPos, step = at % S::kPos / kStep;
      int64_t from = scales_of(p.x0, b, 0);
#pragma unroll
      for (int i = 1; i < S::kSteps; ++i) from = step == i ? scales_of(p.of(i), b, i) : from;
      load_lds4(lds_offset(keys ? sm.ks[buf] : sm.vs[buf]) + w * 256,
                (keys ? c.k_scale : c.v_scale) + from + (static_cast<uint32_t>(block) << c.page_shift) + at % kStep);
    }
  };

  // values: a lane widens 8 neighbouring channels (a word) of the 8 positions
  // 16 u + 4 h + {0 .. 3, 8 .. 11} of one step
  auto widen_words = [&](const Pages& p, int b, int from_buf, int buf, int task_wave) {
    const int l = lane_anew();
    const int task = task_wave * 64 + l;
    const int step = task / S::kTaskLanes, in = task % S::kTaskLanes;
    const int col = in % (D / 8), tu = in / (D / 8) >> 1, th = in / (D / 8) & 1;
    const int first = step * kStep + 16 * tu + 4 * th;
    const uint8_t* words = sm.v[from_buf] + first * S::kRowBytes + col * 4;
    const uint8_t* scales = sm.vs[from_buf] + (col / 4) * S::kPos + first;
    uint8_t* const to = sm.wide[buf] + step * (kStep * D * 2) + (tu * 64 + th * 32) * 16;
    // (a page that is not held stands for page 0, whose bytes its weights of 0 meet)
    const bool wary = static_cast<uint32_t>(b + 1) * S::kPos > least_all || p.any_missing(S::kSteps);
    bool bad = false;
    // kEach positions at a time: with 256 channels all 8 would not fit the registers beside the sums and the queries
    constexpr int kEach = D == 256 ? 4 : 8;
#pragma unroll
    for (int half = 0; half < 8; half += kEach) {
      uint32_t w[kEach];
      float vs[kEach];
#pragma unroll
      for (int e = 0; e < kEach; ++e)
        w[e] = *reinterpret_cast<const uint32_t*>(words + (((half + e) & 3) + 8 * ((half + e) >> 2)) * S::kRowBytes);
#pragma unroll
      for (int z = 0; z < kEach; z += 4) {
        const uint32_t four = *reinterpret_cast<const uint32_t*>(scales + 2 * (half + z));
#pragma unroll
        for (int e = 0; e < 4; ++e) vs[z + e] = scale_of(four, e);
      }
      if (wary) {   // what not every row sees must not meet a weight of 0 as a NaN or an infinity
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          const bool out = vs[e] >= 0x1p126f;   // bytes 253 and up
          bad |= out;
          vs[e] = out ? 0.0f : vs[e];
        }
      }
#pragma unroll
      for (int y = 0; y < 4; ++y) {   // a byte: channels 2 y, 2 y + 1 of the word
        uint32_t x[kEach], lo[kEach / 2], hi[kEach / 2];
#pragma unroll
        for (int e = 0; e < kEach; ++e)
          x[e] = y == 0 ? widen<0>(w[e], vs[e]) : y == 1 ? widen<1>(w[e], vs[e])
                 : y == 2 ? widen<2>(w[e], vs[e]) : widen<3>(w[e], vs[e]);
#pragma unroll
        for (int e = 0; e < kEach / 2; ++e) {
          lo[e] = __builtin_amdgcn_perm(x[2 * e + 1], x[2 * e], 0x05040100u);
          hi[e] = __builtin_amdgcn_perm(x[2 * e + 1], x[2 * e], 0x07060302u);
        }
        // channel k of the word: tile k % NC, row col * 8 / NC + k / NC
        auto put = [&](int k, const uint32_t(&v)[kEach / 2]) {
          const int rr = col * (8 / NC) + k / NC;
          uint8_t* const at = to + ((k % NC) * 128 + rr) * 16 + half * 2;
          if constexpr (kEach == 8) *reinterpret_cast<uint4*>(at) = make_uint4(v[0], v[1], v[2], v[3]);
          else *reinterpret_cast<uint2*>(at) = make_uint2(v[0], v[1]);
        };
        put(2 * y, lo);
        put(2 * y + 1, hi);
      }
    }
    const bool any = __any(bad);
    if (l == 0) sm.bad[buf][task_wave] = any;
  };

  f32x16 acc[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[i][e] = 0.f;
  float top_of_row = neg_inf(), sum_of_row = 0.f;

  // Block b's bytes are in place (b - b0) % 4; keys are fetched three blocks before
  // they are used, values four (they are widened one before).  The first four
  // turns only fetch and widen: in one loop with the others, since a workgroup's
  // first run through any code waits for it to come from memory.
  if (b0 < b1) {
    Pages now, p1, p2, p3, p4 = pages_of(b0);
    now = p1 = p2 = p3 = {-1, -1, -1, -1};
    // this wave's loads of two turns
    const int in_flight = 2 * (2 * (wave < S::kChunks) + (wave < S::kScaleLoads) +
                               (wave >= W / 2 && wave < W / 2 + S::kScaleLoads));
#pragma unroll 1
    for (int b = b0 - 4; b < b1; ++b) {
      const int buf = (b - b0) & 1, raw = (b - b0) & 3;
      if (b + 3 >= b0) fetch(p3, b + 3, true, (raw + 3) & 3);
      fetch(p4, b + 4, false, raw);
      const Pages p5 = pages_of(b + 5);
      const int task_wave = (wave + 4 * buf) & (W - 1);   // the other half of the waves each time
      if (b + 1 >= b0 && b + 1 < b1 && task_wave < S::kTaskWaves) widen_words(p1, b + 1, (raw + 1) & 3, buf ^ 1, task_wave);
#pragma unroll 1
      for (int step = b < b0 ? S::kSteps : 0; step < S::kSteps; step += S::kAtOnce) {
        const uint32_t at = static_cast<uint32_t>(b) * S::kPos + step * kStep;
        if (at >= most) break;
        f32x16 sc[S::kAtOnce];
        bool held[S::kAtOnce], any_held = false;
#pragma unroll
        for (int z = 0; z < S::kAtOnce; ++z) {
          held[z] = now.of(step + z) >= 0;
          any_held |= held[z];
#pragma unroll
          for (int e = 0; e < 16; ++e) sc[z][e] = 0.f;
        }
        if (!any_held) continue;
        const uint8_t* keys = sm.k[raw] + (step * kStep + row32) * S::kRowBytes;
        const uint8_t* scales = sm.ks[raw] + (h * (D / 64)) * S::kPos + step * kStep + row32;
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
          uint4 kw[S::kAtOnce];
          float ks[S::kAtOnce];
#pragma unroll
          for (int z = 0; z < S::kAtOnce; ++z) {
            kw[z] = *reinterpret_cast<const uint4*>(keys + z * (kStep * S::kRowBytes) + S::piece(row32, h * (D / 64) + i) * 16);
            ks[z] = scale_of(scales[i * S::kPos + z * kStep], 0);
          }
#pragma unroll
          for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int z = 0; z < S::kAtOnce; ++z)
              sc[z] = mfma32(widen8(y == 0 ? kw[z].x : y == 1 ? kw[z].y : y == 2 ? kw[z].z : kw[z].w, ks[z]), qv[4 * i + y], sc[z]);
        }
        if (at + S::kAtOnce * kStep > least || !(held[0] && held[S::kAtOnce - 1])) {
          // (against constants: the positions of 16 elements would be kept in registers throughout)
          const int rel = static_cast<int>(sees - at) - 4 * h;
#pragma unroll
          for (int z = 0; z < S::kAtOnce; ++z) {
            const int mine = held[z] ? rel - z * kStep : 0;
#pragma unroll
            for (int e = 0; e < 16; ++e) sc[z][e] = 8 * (e >> 2) + (e & 3) < mine ? sc[z][e] : neg_inf();
          }
        }
        float top = sc[0][0];
#pragma unroll
        for (int z = 0; z < S::kAtOnce; ++z)
#pragma unroll
          for (int e = 0; e < 16; ++e) top = fmaxf(top, sc[z][e]);
        top *= scale;
        if (__any(top > top_of_row + kRaise)) {
          top = fmaxf(top, __shfl_xor(top, 32));
          const float up = fmaxf(top_of_row, top);
          const float down = up == neg_inf() ? 1.0f : __builtin_amdgcn_exp2f(top_of_row - up);
          top_of_row = up;
          sum_of_row *= down;
#pragma unroll
          for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][e] *= down;
        }
        const float base = top_of_row == neg_inf() ? 0.0f : top_of_row;
#pragma unroll
        for (int z = 0; z < S::kAtOnce; ++z) {
          const uint8_t* from = sm.wide[buf] + (step + z) * (kStep * D * 2) + lane * 16;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t w[4][2];
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float a = __builtin_amdgcn_exp2f(fmaf(sc[z][8 * u + 2 * e], scale, -base));
              const float b = __builtin_amdgcn_exp2f(fmaf(sc[z][8 * u + 2 * e + 1], scale, -base));
              sum += a + b;
              // (what split_pair gives; its dot products took 5 and 6% more of chunks of 64 and 128 channels)
              w[e][0] = pack_bf16x2(a, b);
              w[e][1] = pack_bf16x2(a - __uint_as_float(w[e][0] << 16), b - __uint_as_float(w[e][0] & 0xffff0000u));
            }
            sum_of_row += sum;
            bf16x8 pw[2];
#pragma unroll
            for (int p = 0; p < 2; ++p) pw[p] = __builtin_bit_cast(bf16x8, make_uint4(w[0][p], w[1][p], w[2][p], w[3][p]));
            // (two tiles in turn, since a product waits for the one before it on the same sums: 1270 us of the call above, tile
            // by tile 1335; weights formed for 16 positions at a time, or some would be put aside at 256 channels)
#pragma unroll
            for (int i = 0; i < NC; i += 2) {
              const bf16x8 v0 = load_bf16x8(from + (i * 2 + u) * 1024), v1 = load_bf16x8(from + (i * 2 + 2 + u) * 1024);
              acc[i] = mfma32(v0, pw[1], acc[i]);
              acc[i + 1] = mfma32(v1, pw[1], acc[i + 1]);
              acc[i] = mfma32(v0, pw[0], acc[i]);
              acc[i + 1] = mfma32(v1, pw[0], acc[i + 1]);
            }
          }
        }
        int bad = 0;   // the waves that widened these steps
#pragma unroll
        for (int i = 0; i < (S::kAtOnce * S::kTaskLanes + 63) / 64; ++i) bad |= sm.bad[buf][step * S::kTaskLanes / 64 + i];
        if (uniform(bad)) {   // a row that sees such a value has NaN in its 32 channels
#pragma unroll 1
          for (int z = 0; z < S::kAtOnce; ++z) {
            if (now.of(step + z) < 0) continue;
            const uint8_t* of_step = c.v_scale + scales_of(now.of(step + z), b, step + z);
            uint32_t rows_with = 0;   // elements of the lane whose 32 channels hold one
#pragma unroll 1
            for (int e = 0; e < 16; ++e) {
              const int ch = (8 * (e >> 2) + 4 * h + (e & 3)) * NC;   // of tile 0
              const uint8_t* of = of_step + (static_cast<uint32_t>(ch >> 5) << c.page_shift);
#pragma unroll 1
              for (int x = 0; x < kStep; ++x)
                if (of[x] >= 253 && at + z * kStep + x < sees) rows_with |= 1u << e;
            }
#pragma unroll
            for (int e = 0; e < 16; ++e)
#pragma unroll
              for (int i = 0; i < NC; ++i) acc[i][e] = rows_with >> e & 1 ? __uint_as_float(0x7fc00000u) : acc[i][e];
          }
        }
      }
      // the next block's keys and the values of the one after it are there
      lds_barrier(b + 4 < b1 ? in_flight : 0);
      now = p1;
      p1 = p2;
      p2 = p3;
      p3 = p4;
      p4 = p5;
    }
  }

  sum_of_row += __shfl_xor(sum_of_row, 32);
  if (splits > 1 && part == 0 && threadIdx.x == 0)
    joins[id] = {s.first, tile * kRows, std::min(rows - tile * kRows, kRows), head, shares > 1 ? shares : 0};
  if (row >= rows) return;
  if (shares > 1) {
    float* piece = pieces + (static_cast<int64_t>(id) * splits + part) * (static_cast<int64_t>(kRows) * (D + 2));
    const int at = wave * 32 + row32;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int ch = (8 * (e >> 2) + 4 * h + (e & 3)) * NC;
      float x[NC];
#pragma unroll
      for (int i = 0; i < NC; ++i) x[i] = acc[i][e];
      store_n<false, NC>(piece, static_cast<size_t>(at) * D + ch, x);
    }
    if (h == 0) {
      piece[kRows * D + 2 * at] = top_of_row;
      piece[kRows * D + 2 * at + 1] = sum_of_row;
    }
  } else {
    const int t = row / group;
    const size_t to = static_cast<size_t>(s.first + t) * Hq + head * group + (row - t * group);
    const float inv = sum_of_row == 0.0f ? 0.0f : 1.0f / sum_of_row;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int ch = (8 * (e >> 2) + 4 * h + (e & 3)) * NC;
      float x[NC];
#pragma unroll
      for (int i = 0; i < NC; ++i) x[i] = sum_of_row == 0.0f ? 0.0f : acc[i][e] * inv;
      store_n<true, NC>(o, to * D + ch, x);
    }
    if (lse && h == 0) lse[to] = row_lse(top_of_row, sum_of_row);
  }
}

namespace {

constexpr int kMostParts = 128;

// Places for the sums of parts (256 rows each: 264 KB at 256 channels).  Up to 85
// units, of which one round of workgroups takes three parts each, as many as one
// round (one a CU; at 64 and 128 channels, where a place is smaller, three and two
// rounds); above, where shares that come out even are worth a second and a third
// round, 768: 203 MB, 103 or 52.  (One chunk behind 8192 positions, 2 key heads of
// 256, with 256 and 768 places: 64 units 217 us both, 94 units 401 and 353.)
int64_t most_pieces(int D, int64_t units) {
  if (units > 85) return 768;
  return D == 256 ? 256 : D == 128 ? 512 : 768;
}

// Units to be expected: no sequence has more than max_rows rows.  (The results
// do not rest on it.)
int64_t units_by(const CacheArgs& c, int group, int64_t max_rows) {
  const int64_t tiles = std::max(c.n_tokens * group / kChunkRows, (max_rows + kChunkRows - 1) / kChunkRows * c.N);
  return std::min(tiles * c.heads, most_chunk_units(c, group));
}

// Equal parts of each unit's positions at most, of the blocks that the page table
// has room for: what takes the CUs (a workgroup each; the second that fits at 64
// channels is not counted) the least time, in blocks of 256 rows: a workgroup costs
// two and a half besides its own, the join one and a half, and a part's sums,
// written and read again, a thirtieth on all CUs (with a quarter to a third less of
// each, chunks of 512 to 6000 tokens behind 0 to 32768 positions took the same).
// The kernel takes fewer where the positions are few.
template <int D>
int parts_of(const CacheArgs& c, int64_t units, int64_t most_units) {
  const int64_t room = (static_cast<int64_t>(c.max_pages) << c.page_shift) / ChunkShape<D>::kPos + 1;
  int best = 1;
  double least = 1e30;
  for (int s = 1; s <= kMostParts && (s == 1 || most_units * s <= most_pieces(D, most_units)); ++s) {
    const double cost = static_cast<double>((units * s + 255) / 256) * (static_cast<double>((room + s - 1) / s) + 2.5) +
                        (s > 1 ? 1.5 + 0.033 * static_cast<double>(units * s) : 0.0);
    if (cost < least) {
      least = cost;
      best = s;
    }
  }
  return best;
}

int parts_of(int D, const CacheArgs& c, int64_t units, int64_t most_units) {
  return D == 64 ? parts_of<64>(c, units, most_units) : D == 128 ? parts_of<128>(c, units, most_units) : parts_of<256>(c, units, most_units);
}

}  // namespace

// Every sequence's last tile may be a short one.
int64_t most_chunk_units(const CacheArgs& c, int group) {
  return (c.n_tokens * group + (kChunkRows - 1) * std::min<int64_t>(c.N, c.n_tokens)) / kChunkRows * c.heads;
}

// What any call of at most so many units needs.
size_t attention_chunk_ws(int D, int64_t units) {
  return units * sizeof(Split) + std::min(kMostParts * units, most_pieces(D, units)) * (static_cast<size_t>(kChunkRows) * (D + 2) * 4);
}

hipError_t launch_attention_chunk(int D, const CacheArgs& c, const void* q, int group, float scale,
                                  int64_t max_rows, void* o, float* lse, void* ws, hipStream_t st) {
  const int64_t units = most_chunk_units(c, group);
  const int parts = parts_of(D, c, units_by(c, group, max_rows), units);
  Split* joins = static_cast<Split*>(ws);
  float* pieces = reinterpret_cast<float*>(joins + units);
  const dim3 grid(static_cast<unsigned>(units * parts));
  const size_t shared = (static_cast<size_t>(c.N) + 1) * 4;
  auto go = [&](auto d) {
    constexpr int kD = decltype(d)::value;
    attention_chunk_kernel<kD><<<grid, kChunkWaves * 64, shared, st>>>(c, q, group, scale, parts, static_cast<int>(units), o,
                                                                     lse, joins, pieces);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || parts == 1) return e;
    return launch_join_parts(kD, c, group, o, lse, joins, pieces, static_cast<int>(units), parts, st);
  };
  switch (D) {
    case 64: return go(std::integral_constant<int, 64>{});
    case 128: return go(std::integral_constant<int, 128>{});
    case 256: return go(std::integral_constant<int, 256>{});
    default: return hipErrorInvalidValue;
  }
}

}  // namespace kda
