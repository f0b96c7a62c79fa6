// Attention of each sequence's newest tokens over its paged 4-bit cache.
//
// With G query heads to a key head, the q_n tokens of a sequence give q_n * G
// rows that share one head's keys and values.  Transposed products keep a row
// in one column of lanes all the way:
//   S^T = K Q^T   (32 positions x 16 rows: two 16x16x32 steps per 32 channels)
//   O^T += V^T P^T
// The result layout of S^T (lane l: positions 8 (l / 16) .. + 7, row l % 16) is
// the operand layout of P^T when the 32 positions are taken in the order
// 2 j + t (row j of step t), so the softmax and its weights never leave their
// lane.  Keys and values go from memory to registers and are widened to bf16
// there (exact; half an instruction a value with the scale applied), each lane
// reading whole bytes: of keys d / 4 channels of two neighbouring positions, of
// values d / 16 channels of eight.
//
// The running maximum of a row is raised only when a score passes it by 2^8:
// weights then reach 256, which neither fp32 sums nor bf16 operands mind, and
// the accumulators are rescaled a few times a row instead of at every step.
//
// Precision.  Keys are widened to bf16 (exact) and queries enter as they are: as
// one bf16 value, or the three that an fp32 one is the sum of, so that scores have
// the rounding of fp32 sums alone, whatever the channels' sizes.  (The matrix cores
// would take the keys' 4 bits as they lie, next to queries of 6 or 8 bits.  A query
// is then a sum of such values that share a power of two: what is small beside the
// largest of its 32 channels loses bits that a key may turn into the whole score,
// and 8-bit products are cut 2^13 below a step's largest.)  Weights enter as two
// bf16 values for bf16 outputs (off by 2^-16; one is off by 2^-8, which moves an
// output by as much as its own rounding) and as three for fp32 ones; their sum is of
// the weights before that, so that a token's result is the same to that precision
// whatever else is in the call, and lse has fp32's.
//
// Work: all (sequence, key head, row tile) units are laid end to end in blocks
// of 128 positions, and every workgroup takes an equal share of that line, so
// ragged batches balance without the host knowing a length.  A unit that one
// workgroup finishes is written at once; the pieces of the others (at most two
// a workgroup) go to the workspace and a second kernel joins them in their
// order.  A step of 256 sequences at up to 8192 positions, 16 query heads on 2 key
// heads of 256, takes 130 us and 5 for the join (4.9 TB/s of the cache's bytes); 37
// with 4 drafts each at up to 16384, 32 on 8 of 128: 80 and 5 (4.6 TB/s).
#include <algorithm>

#include "attention.h"

namespace kda {

namespace {

constexpr int kWaves = 4;
constexpr int kBlockPos = kWaves * kStep;   // positions of a block
constexpr int kMostWorkgroups = 512;        // two a CU
constexpr int64_t kMostUnits = 1 << 22;     // of the chunk kernel
// A piece's place in the workspace: its rows' sums, then maxima and weights' sums.
template <int D, int ROWS>
__device__ __forceinline__ float* piece_at(float* pieces, int64_t slot) {
  return pieces + slot * (static_cast<int64_t>(ROWS) * (D + 2));
}

// Waves a SIMD that the registers leave room for.
constexpr int waves_of(int D, int mt) { return D / 16 * mt > 16 ? 1 : 2; }

// bf16 values that a query is held in, exactly: what it comes as, or the three of an fp32 one.
template <bool IN_BF16>
constexpr int kQueryPieces = IN_BF16 ? 1 : 3;

// A wave's step of 32 positions as it lies in memory.  Of a position's key a lane reads d / 4 channels.
template <int D>
struct RawKeys {
  uint32_t w[2][D / 32];            // positions 2 (l % 16) and the next
  uint32_t scale[D > 128 ? 2 : 1];  // their scale bytes, for each 32 channels of the lane
};
template <int D>
struct RawValues {
  uint32_t w[8][D > 128 ? 2 : 1];   // positions 8 (l / 16) ..
  uint2 scale;                      // their scale bytes
};

// Where a lane's bytes of a step are, from the step's first byte.
template <int D>
struct LaneOffsets {
  uint32_t k, ks[D > 128 ? 2 : 1], v, vs;

  __device__ __forceinline__ explicit LaneOffsets(int page_shift) {
    const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
    k = 2 * j * (D / 2) + g * (D / 8);
#pragma unroll
    for (int i = 0; i < (D > 128 ? 2 : 1); ++i) ks[i] = ((g * D / 128 + i) << page_shift) + 2 * j;
    v = 8 * g * (D / 2) + j * (D / 32);
    vs = ((j * D / 512) << page_shift) + 8 * g;
  }
};

template <int D>
__device__ __forceinline__ void load_keys(const CacheArgs& c, const StepAt& at, const LaneOffsets<D>& lane, RawKeys<D>& r) {
  const uint8_t* row = c.k + at.values;
  const uint8_t* scales = c.k_scale + at.scales;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    if constexpr (D == 64) {
      const uint2 w = *reinterpret_cast<const uint2*>(row + lane.k + t * (D / 2));
      r.w[t][0] = w.x;
      r.w[t][1] = w.y;
    } else {
#pragma unroll
      for (int i = 0; i < D / 128; ++i) {
        const uint4 w = *reinterpret_cast<const uint4*>(row + lane.k + t * (D / 2) + 16 * i);
        r.w[t][4 * i] = w.x;
        r.w[t][4 * i + 1] = w.y;
        r.w[t][4 * i + 2] = w.z;
        r.w[t][4 * i + 3] = w.w;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < (D > 128 ? 2 : 1); ++i) r.scale[i] = *reinterpret_cast<const uint16_t*>(scales + lane.ks[i]);
}

template <int D>
__device__ __forceinline__ void load_values(const CacheArgs& c, const StepAt& at, const LaneOffsets<D>& lane,
                                            RawValues<D>& r) {
  const uint8_t* row = c.v + at.values;
  r.scale = *reinterpret_cast<const uint2*>(c.v_scale + at.scales + lane.vs);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint8_t* from = row + lane.v + e * (D / 2);
    if constexpr (D == 64) {
      r.w[e][0] = *reinterpret_cast<const uint16_t*>(from);
    } else if constexpr (D == 128) {
      r.w[e][0] = *reinterpret_cast<const uint32_t*>(from);
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(from);
      r.w[e][0] = w.x;
      r.w[e][1] = w.y;
    }
  }
}

// Rows' accumulators of one wave: MT tiles of 16 rows, this lane's row l % 16 of each.
template <int D, int MT>
struct Rows {
  f32x4 o[MT][D / 16];   // channel (4 (l / 16) + i) * D / 16 + c of o[.][c][i]
  float m[MT], l[MT];    // running maximum (of the row), sum of this lane's weights
};

// Queries of 16 rows as operands: a lane holds the channels of its keys.  The
// smallest of the three pieces of 256 channels waits in LDS (every wave's is the
// same), or two waves a SIMD would not fit the registers.
template <int D, int QP>
constexpr bool kThirdInLds = D == 256 && QP == 3;

template <int D, int QP>
struct Queries {
  SplitN<kThirdInLds<D, QP> ? 2 : QP> v[D / 32];
};

// row: the first element of the row's head; flip: 0x80008000 turns every sign.
template <int D, bool BF16>
__device__ __forceinline__ void load_queries(const void* q, size_t row, uint32_t flip, Queries<D, kQueryPieces<BF16>>& r,
                                             uint4 (*third)[64]) {
  constexpr int QP = kQueryPieces<BF16>;
  const int lane = threadIdx.x & 63, g = lane >> 4;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const size_t at = row + g * (D / 4) + 8 * i;
    SplitN<QP> x;
    if constexpr (BF16) x.v[0] = load_bf16x8(static_cast<const uint16_t*>(q) + at);
    else x = load_split<3>(static_cast<const float*>(q) + at);
#pragma unroll
    for (int p = 0; p < QP; ++p) {
      uint4 w = __builtin_bit_cast(uint4, x.v[p]);
      w.x ^= flip;
      w.y ^= flip;
      w.z ^= flip;
      w.w ^= flip;
      if constexpr (kThirdInLds<D, QP>) {
        if (p == 2) {
          third[i][lane] = w;
          continue;
        }
      }
      r.v[i].v[p] = __builtin_bit_cast(bf16x8, w);
    }
  }
}

// S^T of a step: element (position 8 g + e, row j) in s[.][e & 1][e >> 1].
template <int D, int MT, int QP>
__device__ __forceinline__ void scores(const RawKeys<D>& r, const Queries<D, QP> (&q)[MT], const uint4 (*third)[64],
                                       f32x4 (&s)[MT][2]) {
  constexpr bool kThird = kThirdInLds<D, QP>;
  int lane = threadIdx.x & 63;
  if constexpr (kThird) asm volatile("" : "+v"(lane));   // read anew in every step, not kept across them
#pragma unroll
  for (int m = 0; m < MT; ++m) s[m][0] = s[m][1] = zero4();
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const bf16x8 k = widen8(r.w[t][i], scale_of(D > 128 && i >= 4 ? r.scale[D > 128 ? 1 : 0] : r.scale[0], t));
      if constexpr (kThird) s[0][t] = mfma(k, load_bf16x8(&third[i][lane]), s[0][t]);
#pragma unroll
      for (int p = (kThird ? 2 : QP) - 1; p >= 0; --p)
#pragma unroll
        for (int m = 0; m < MT; ++m) s[m][t] = mfma(k, q[m].v[i].v[p], s[m][t]);
    }
}

// The step's weights, and its values' part of the sums.
// scale > 0 (queries carry its sign); `whole`: every row sees all of the positions.
template <int D, int MT, int PP>
__device__ __forceinline__ void weigh(const RawValues<D>& r, const f32x4 (&s)[MT][2], float scale, bool whole,
                                      uint32_t at, const uint32_t (&sees)[MT], const uint8_t* v_scales, int page_shift,
                                      Rows<D, MT>& acc) {
  const int lane = threadIdx.x & 63, g = lane >> 4;
  uint32_t w[MT][4][PP];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    float x[8];   // position 8 g + e
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = s[m][e & 1][e >> 1];
    if (!whole) {
      const int rel = static_cast<int>(sees[m] - at) - 8 * g;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = e < rel ? x[e] : neg_inf();
    }
    float top = x[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) top = fmaxf(top, x[e]);
    top *= scale;
    if (__any(top > acc.m[m] + kRaise)) {
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const float up = fmaxf(acc.m[m], top);
      const float down = up == neg_inf() ? 1.0f : __builtin_amdgcn_exp2f(acc.m[m] - up);
      acc.m[m] = up;
      acc.l[m] *= down;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) acc.o[m][i] *= down;
    }
    const float base = acc.m[m] == neg_inf() ? 0.0f : acc.m[m];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __builtin_amdgcn_exp2f(fmaf(x[e], scale, -base));
#pragma unroll
    for (int e = 0; e < 4; ++e) split_pair<PP>(x[2 * e], x[2 * e + 1], w[m][e]);
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += x[e];
    acc.l[m] += sum;
  }
  float vs[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) vs[e] = scale_of(e < 4 ? r.scale.x : r.scale.y, e & 3);
  bool bad = false;
  if (!whole) {   // what not every row sees must not meet a weight of 0 as a NaN or an infinity
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const bool out = vs[e] >= 0x1p126f;   // bytes 253 and up
      bad |= out;
      vs[e] = out ? 0.0f : vs[e];
    }
  }
#pragma unroll
  for (int b = 0; b < D / 32; ++b) {   // a byte: two channels
    __builtin_amdgcn_sched_barrier(0);
    uint32_t x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t word = r.w[e][b >> 2];
      x[e] = (b & 3) == 0 ? widen<0>(word, vs[e]) : (b & 3) == 1 ? widen<1>(word, vs[e])
             : (b & 3) == 2 ? widen<2>(word, vs[e]) : widen<3>(word, vs[e]);
    }
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      lo[e] = __builtin_amdgcn_perm(x[2 * e + 1], x[2 * e], 0x05040100u);
      hi[e] = __builtin_amdgcn_perm(x[2 * e + 1], x[2 * e], 0x07060302u);
    }
    const bf16x8 v0 = __builtin_bit_cast(bf16x8, make_uint4(lo[0], lo[1], lo[2], lo[3]));
    const bf16x8 v1 = __builtin_bit_cast(bf16x8, make_uint4(hi[0], hi[1], hi[2], hi[3]));
#pragma unroll
    for (int p = PP - 1; p >= 0; --p)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const bf16x8 pw = __builtin_bit_cast(bf16x8, make_uint4(w[m][0][p], w[m][1][p], w[m][2][p], w[m][3][p]));
        acc.o[m][2 * b] = mfma(v0, pw, acc.o[m][2 * b]);
        acc.o[m][2 * b + 1] = mfma(v1, pw, acc.o[m][2 * b + 1]);
      }
  }
  if (!whole && __any(bad)) {   // a row that sees such a value has NaN in its 32 channels
    uint32_t with = 0;   // bit 4 m + i: the lane's channels i of row tile m
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      const uint8_t* of = v_scales + (static_cast<uint32_t>((4 * g + i) * D / 512) << page_shift);
#pragma unroll 1
      for (int e = 0; e < kStep; ++e) {
        if (of[e] < 253) continue;
#pragma unroll
        for (int m = 0; m < MT; ++m)
          if (at + e < sees[m]) with |= 1u << (4 * m + i);
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int x = 0; x < D / 16; ++x)
          acc.o[m][x][i] = with >> (4 * m + i) & 1 ? __uint_as_float(0x7fc00000u) : acc.o[m][x][i];
  }
}

}  // namespace

template <int D, int MT, bool IN_BF16, bool OUT_BF16>
__global__ __launch_bounds__(kWaves * 64, waves_of(D, MT)) void paged_attention_kernel(
    CacheArgs c, const void* __restrict__ q, int group, float scale, void* __restrict__ o, float* __restrict__ lse,
    Split* __restrict__ splits, float* __restrict__ pieces) {
  constexpr int kRows = 16 * MT, QP = kQueryPieces<IN_BF16>, PP = OUT_BF16 ? 2 : 3;
  constexpr int kPitch = D + 4;
  __shared__ float meet[kWaves][16][kPitch];
  __shared__ float tops[kWaves][kRows][2];
  __shared__ uint4 third[kThirdInLds<D, QP> ? D / 32 : 1][64];
  static_assert(!kThirdInLds<D, QP> || MT == 1, "one tile's");
  // [N + 1].  (At 256 channels a second workgroup fits a CU up to 1855 sequences, with fp32 queries up to 831: single tokens at
  // 1000 positions take 0.123 us each in a call of 1840 and 0.153 in one of 1880, in fp32 0.147 of 800 and 0.182 of 900.)
  extern __shared__ int64_t before[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), j = lane & 15, g = lane >> 4;
  const int Hq = c.heads * group;
  // a negative scale turns the queries' sign; of 0 every score is 0, as of the least (where -infinity stays what it is)
  const uint32_t flip = scale < 0.0f ? 0x80008000u : 0u;
  scale = fminf(fmaxf(fabsf(scale), 1.17549435e-38f), 3.4028235e38f);
  lay_out<kWaves * 64>(c.N, before, reinterpret_cast<int64_t*>(meet), [&](int n) {
    const Sequence s = sequence(c, n);
    const int64_t tiles = (static_cast<int64_t>(s.tokens) * group + kRows - 1) / kRows;
    return tiles * c.heads * ((static_cast<int64_t>(s.length) + kBlockPos - 1) / kBlockPos);
  });
  const int64_t total = before[c.N];
  const int64_t share = (total + gridDim.x - 1) / gridDim.x;
  const int64_t start = share * blockIdx.x;
  const int64_t end = start + share < total ? start + share : total;
  Split split = {0, 0, 0, 0, 0};
  const LaneOffsets<D> lanes(c.page_shift);
  const int64_t page_bytes = static_cast<int64_t>(c.heads) * (D / 2) << c.page_shift;

  // sequences that hold nothing: their rows see nothing
  for (int n = blockIdx.x; n < c.N; n += gridDim.x) {
    const Sequence s = sequence(c, n);
    if (s.length > 0) continue;
    for (int64_t i = threadIdx.x; i < static_cast<int64_t>(s.tokens) * Hq * (D / 8); i += kWaves * 64) {
      const float zero[8] = {};
      store_n<OUT_BF16, 8>(o, static_cast<size_t>(s.first) * Hq * D + i * 8, zero);
    }
    if (lse)
      for (int64_t i = threadIdx.x; i < static_cast<int64_t>(s.tokens) * Hq; i += kWaves * 64)
        lse[static_cast<size_t>(s.first) * Hq + i] = neg_inf();
  }

  for (int64_t cur = start; cur < end;) {
    int n = 0;
    for (int hi = c.N; hi - n > 1;) {   // the last with before[n] <= cur
      const int mid = (n + hi) >> 1;
      if (before[mid] <= cur) n = mid;
      else hi = mid;
    }
    n = uniform(n);
    const Sequence s = sequence(c, n);
    const int blocks = static_cast<int>((static_cast<int64_t>(s.length) + kBlockPos - 1) / kBlockPos);
    const int rows = s.tokens * group;
    const int tiles = (rows + kRows - 1) / kRows;
    const int64_t local = uniform(cur - before[n]);
    const int64_t unit = local / blocks;
    const int b0 = static_cast<int>(local - unit * blocks);
    const int b1 = end - cur < blocks - b0 ? b0 + static_cast<int>(end - cur) : blocks;
    const int head = static_cast<int>(unit / tiles), tile = static_cast<int>(unit - static_cast<int64_t>(head) * tiles);
    // this lane's rows
    Queries<D, QP> qf[MT];
    uint32_t sees[MT];
    auto seen = [&](int row) { return s.seen(row / group); };   // positions that a row sees
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int row = tile * kRows + m * 16 + j;
      const int r = row < rows ? row : rows - 1;
      const int t = r / group;
      load_queries<D, IN_BF16>(q, (static_cast<size_t>(s.first + t) * Hq + head * group + (r - t * group)) * D, flip, qf[m],
                               third);
      sees[m] = seen(r);
    }
    // positions that every row sees, and that any does
    const uint32_t least = seen(tile * kRows), most = seen(((tile + 1) * kRows < rows ? (tile + 1) * kRows : rows) - 1);
    Rows<D, MT> acc;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      acc.m[m] = neg_inf();
      acc.l[m] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) acc.o[m][i] = zero4();
    }
    // A step's values are on their way while its scores are formed, the next
    // step's keys while its values are weighed, the page after that meanwhile.
    const int64_t head_bytes = static_cast<int64_t>(head) * (D / 2) << c.page_shift;
    const uint32_t first_pos = wave * kStep;
    int stop = most > first_pos ? static_cast<int>((most - first_pos + kBlockPos - 1) / kBlockPos) : 0;
    stop = c.num_pages == 0 ? b0 : stop < b1 ? stop : b1;   // blocks in front of it have a step to be seen
    if (b0 < stop) {
      auto place = [&](int b) {
        return step_at<D>(c, n, page_bytes, head_bytes, static_cast<uint32_t>(b) * kBlockPos + first_pos, b < stop);
      };
      StepAt here = place(b0);
      RawKeys<D> keys;
      load_keys<D>(c, here, lanes, keys);
      StepAt next = place(b0 + 1);
      for (int b = b0; b < stop; ++b) {
        const uint32_t at = static_cast<uint32_t>(b) * kBlockPos + first_pos;
        RawValues<D> values;
        load_values<D>(c, here, lanes, values);
        f32x4 s4[MT][2];
        scores<D, MT, QP>(keys, qf, third, s4);
        __builtin_amdgcn_sched_barrier(0);
        load_keys<D>(c, next, lanes, keys);
        const StepAt after = place(b + 2);
        if (here.held)
          weigh<D, MT, PP>(values, s4, scale, at + kStep <= least, at, sees, c.v_scale + here.scales, c.page_shift, acc);
        here = next;
        next = after;
      }
    }
    // The waves' sums joined, 16 rows at a time.  (A row's single values are
    // stored in front of its channels: where such a branch ended together with
    // the one around it, the compiler brought registers back from where it had
    // put them aside for the branch's lanes alone, and rows came out wrong.)
    const bool whole = b0 == 0 && b1 == blocks;
    float* piece = piece_at<D, kRows>(pieces, 2 * static_cast<int64_t>(blockIdx.x) + (b0 == 0));
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      acc.l[m] += __shfl_xor(acc.l[m], 16);
      acc.l[m] += __shfl_xor(acc.l[m], 32);
      if (g == 0) {
        tops[wave][m * 16 + j][0] = acc.m[m];
        tops[wave][m * 16 + j][1] = acc.l[m];
      }
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float up = tops[0][m * 16 + j][0];
#pragma unroll
      for (int x = 1; x < kWaves; ++x) up = fmaxf(up, tops[x][m * 16 + j][0]);
      const float f = acc.m[m] == neg_inf() ? 0.0f : __builtin_amdgcn_exp2f(acc.m[m] - up);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int x = 0; x < D / 16; x += 4)
          *reinterpret_cast<float4*>(&meet[wave][j][(4 * g + i) * (D / 16) + x]) =
              make_float4(acc.o[m][x][i] * f, acc.o[m][x + 1][i] * f, acc.o[m][x + 2][i] * f, acc.o[m][x + 3][i] * f);
      __syncthreads();
      for (int i = threadIdx.x; i < 16 * (D / 8); i += kWaves * 64) {
        const int rr = i / (D / 8), ch = (i - rr * (D / 8)) * 8;
        const int row = tile * kRows + m * 16 + rr;
        if (row >= rows) continue;
        float up2 = tops[0][m * 16 + rr][0], l = 0.f, x[8] = {};
#pragma unroll
        for (int y = 1; y < kWaves; ++y) up2 = fmaxf(up2, tops[y][m * 16 + rr][0]);
#pragma unroll
        for (int y = 0; y < kWaves; ++y) {
          const float my = tops[y][m * 16 + rr][0];
          // (nothing seen: 0; NaN scores alone leave no maximum either, and a sum of NaN)
          l = fmaf(my == neg_inf() ? 0.0f : __builtin_amdgcn_exp2f(my - up2), tops[y][m * 16 + rr][1], l);
          float part[8];
          load_n<false, 8>(&meet[y][rr][0], ch, part);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] += part[e];
        }
        if (whole) {
          const int t = row / group;
          const size_t to = static_cast<size_t>(s.first + t) * Hq + head * group + (row - t * group);
          const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = l == 0.0f ? 0.0f : x[e] * inv;
          if (lse && ch == 0) lse[to] = row_lse(up2, l);
          store_n<OUT_BF16, 8>(o, to * D + ch, x);
        } else {
          if (ch == 0) {
            piece[kRows * D + 2 * (m * 16 + rr)] = up2;
            piece[kRows * D + 2 * (m * 16 + rr) + 1] = l;
          }
          store_n<false, 8>(piece, static_cast<size_t>(m * 16 + rr) * D + ch, x);
        }
      }
      __syncthreads();
    }
    if (!whole && b0 == 0)
      split = {s.first, tile * kRows, std::min(rows - tile * kRows, kRows), head,
               1 + static_cast<int>((blocks - b1 + share - 1) / share)};
    cur += b1 - b0;
  }
  if (threadIdx.x == 0) splits[blockIdx.x] = split;
}

// Joins the pieces of units: PARTS: of the chunk kernel's, of `stride` places each;
// otherwise of those that began in one of the `units` workgroups of the kernel
// above.  A wave takes a row, eight pieces of it in flight, or kWide waves do where
// there are more than eight; the workgroups take the units of few pieces by their
// own number, and find those of many by a count over all.  us with 4, 8, 16 waves:
// one row tile of 16384 positions, 2 key heads of 256: 9.3, 6.4, 5.9; 256 sequences
// at 8192 (few pieces): 4.8, 4.8, 5.6; parts of 4 x 512 rows at 8192: 16.4, 23.3, -.
template <int D, int ROWS, bool OUT_BF16, bool PARTS>
__global__ __launch_bounds__(1024) void join_pieces_kernel(int heads, int group, void* __restrict__ o,
                                                           float* __restrict__ lse, const Split* __restrict__ splits,
                                                           const float* __restrict__ pieces, int units, int stride) {
  constexpr int E = D / 64, kTogether = 8;   // channels of a lane; pieces whose loads are in flight
  constexpr int kWide = PARTS ? 4 : 8;         // waves of a row of many pieces
  __shared__ float meet[16][64][E], tops[16][2];
  __shared__ int counts[16], list[PARTS ? 1 : kMostWorkgroups];
  const int wave = uniform(static_cast<int>(threadIdx.x >> 6)), lane = threadIdx.x & 63;

  // row rr of a unit, of which this wave takes pieces first, first + step ..
  auto join = [&](int unit, int rr, int first, int step) {
    const bool shared = step > 1;
    const Split* split = splits + unit;
    const int n_pieces = split->pieces, row = split->row0 + rr;
    const bool mine = rr < split->rows;
    auto at = [&](int i) {   // (in a workgroup's two, a unit that begins there is the second)
      return pieces + (PARTS ? static_cast<int64_t>(unit) * stride + i : 2 * static_cast<int64_t>(unit + i) + (i == 0)) *
                          (static_cast<int64_t>(ROWS) * (D + 2));
    };
    float up = neg_inf(), l = 0.f, x[E] = {};
    for (int i = first; mine && i < n_pieces; i += step * kTogether) {
      float m[kTogether], w[kTogether] = {}, y[kTogether][E] = {};
#pragma unroll
      for (int k = 0; k < kTogether; ++k) {
        m[k] = neg_inf();
        if (i + step * k >= n_pieces) continue;
        const float* p = at(i + step * k);
        m[k] = p[ROWS * D + 2 * rr];
        w[k] = p[ROWS * D + 2 * rr + 1];
        load_n<false, E>(p, static_cast<size_t>(rr) * D + lane * E, y[k]);
      }
      float top = up;
#pragma unroll
      for (int k = 0; k < kTogether; ++k) top = fmaxf(top, m[k]);
      const float down = up == neg_inf() ? 0.0f : __builtin_amdgcn_exp2f(up - top);
      up = top;
      l *= down;
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] *= down;
#pragma unroll
      for (int k = 0; k < kTogether; ++k) {
        // (a piece in which the row saw nothing holds zeros; a NaN maximum stays NaN)
        const float f = m[k] == neg_inf() ? 0.0f : __builtin_amdgcn_exp2f(m[k] - up);
        l = fmaf(f, w[k], l);
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = fmaf(f, y[k][e], x[e]);
      }
    }
    float top = up;
    if (shared) {
      store_n<false, E>(&meet[wave][lane][0], 0, x);
      if (lane == 0) {
        tops[wave][0] = up;
        tops[wave][1] = l;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kWide; ++k) top = fmaxf(top, tops[(wave & ~(kWide - 1)) + k][0]);
      l = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = 0.f;
#pragma unroll
      for (int k = 0; k < kWide; ++k) {
        const float m = tops[(wave & ~(kWide - 1)) + k][0], f = m == neg_inf() ? 0.0f : __builtin_amdgcn_exp2f(m - top);
        l = fmaf(f, tops[(wave & ~(kWide - 1)) + k][1], l);
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = fmaf(f, meet[(wave & ~(kWide - 1)) + k][lane][e], x[e]);
      }
      __syncthreads();
    }
    if (mine && first == 0) {
      const int t = row / group;
      const size_t to = static_cast<size_t>(split->first + t) * heads * group + split->head * group + (row - t * group);
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = l == 0.0f ? 0.0f : x[e] / l;
      if (lse && lane == 0) lse[to] = row_lse(top, l);
      store_n<OUT_BF16, E>(o, to * D + lane * E, x);
    }
  };

  constexpr int kFew = ROWS / 16, kMany = ROWS * kWide / 16;   // a unit's jobs
  if constexpr (PARTS) {
    const bool many = stride > kTogether;
    const int jobs = many ? kMany : kFew;
    for (int job = blockIdx.x; job < units * jobs; job += gridDim.x) {
      const int unit = job / jobs, own = job - unit * jobs;
      if (splits[unit].pieces == 0) continue;
      if (many) join(unit, own * (16 / kWide) + wave / kWide, wave % kWide, kWide);
      else join(unit, own * 16 + wave, 0, 1);
    }
  } else {
    static_assert(kMostWorkgroups <= 1024, "a thread each");
    const bool many = static_cast<int>(threadIdx.x) < units && splits[threadIdx.x].pieces > kTogether;
    for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
      const int n = splits[unit].pieces;
      if (n == 0 || n > kTogether) continue;
      for (int own = 0; own < kFew; ++own) join(unit, own * 16 + wave, 0, 1);
    }
    const uint64_t with = __ballot(many);
    if (lane == 0) counts[wave] = __popcll(with);
    __syncthreads();
    int to = __popcll(with & ((1ull << lane) - 1)), todo = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
      to += w < wave ? counts[w] : 0;
      todo += counts[w];
    }
    if (many) list[to] = threadIdx.x;
    __syncthreads();
    todo = uniform(todo) * kMany;
    for (int job = blockIdx.x; job < todo; job += gridDim.x)
      join(uniform(list[job / kMany]), job % kMany * (16 / kWide) + wave / kWide, wave % kWide, kWide);
  }
}

namespace {

// Row tiles of 16 that a workgroup takes.  us with 1, 2, 4 (64 sequences of 4096
// positions, 8 key heads): d 128, 20 rows each: 93, 70, 162; 64 rows: 183, 134, 166
// (4 fill the registers: one wave a SIMD); d 64, 30 rows: 66, 49, 78; 40: 95, 90,
// 79; 64: 126, 91, 80; d 256 (32 of 8192, 2 key heads), 24 rows: 54, 49.  The three
// pieces of fp32 queries leave room for two at 64 channels and one above.
int row_tiles(int D, bool in_bf16, bool out_bf16, int64_t rows) {
  if (!out_bf16 || rows <= 16 || (!in_bf16 && D > 64)) return 1;
  return D == 64 && in_bf16 && rows > 32 ? 4 : 2;
}

// Whether the chunk kernel takes a call: it reads keys and values once for 256
// rows, but computes for 256 where there are fewer, and takes longer to begin.  us
// there and here (sequences x rows of a key head behind 4096 positions unless said):
//   d 64, 8 key heads: 64 x 160: 198, 226; 64 x 256: 232, 298; 16 x 256: 97, 80;
//     1 x 4096: 112, 94; 1 x 8192: 208, 211; 4 x 2048: 159, 164
//   d 128, 8 key heads: 64 x 160: 384, 327; 64 x 224: 395, 463; 16 x 256: 130, 143;
//     1 x 4096: 146, 141; 1 x 8192: 284, 327; 4 x 2048: 219, 255
//   d 256, 2 key heads: 64 x 128: 148, 155; 64 x 160: 193, 209; 16 x 256: 113, 80;
//     1 x 4096: 90, 85, behind 16384 213, 281; 4 x 1024: 91, 80, behind 16384 251, 277
// (Its workgroups are the units, which have to fit a grid: kMostUnits.)
bool for_chunks(int D, const CacheArgs& c, int group, bool bf16, int64_t rows) {
  const int64_t all = c.n_tokens * c.heads * group;
  return bf16 && rows > (D == 128 ? 192 : 128) && all >= (D == 256 ? 8192 : 65536);
}

// Two a CU, or one where the registers leave room for one wave a SIMD (d 256, 24 rows
// as above: 49 us, with two 65; d 128, 64 rows, where two fit: 134, with one 173).
int workgroups(int D, int mt) { return kMostWorkgroups / 2 * waves_of(D, mt); }

// Rows of a key head of the longest sequence; where max_q is not known, those of
// the mean (256 sequences of one token at 8192 positions, 2 key heads of 256: 202
// us, and 906 when all tokens were counted as one sequence's, in the chunk kernel;
// one long chunk among many sequences goes to the first kernel for it).
int64_t rows_of(const CacheArgs& c, int group, int max_q) {
  return (max_q > 0 ? std::min<int64_t>(max_q, c.n_tokens) : (c.n_tokens + c.N - 1) / c.N) * group;
}

}  // namespace

hipError_t launch_join_parts(int D, const CacheArgs& c, int group, void* o, float* lse, const Split* joins,
                             float* pieces, int units, int stride, hipStream_t st) {
  constexpr int kRows = kChunkRows;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(static_cast<int64_t>(units) * (kRows / 4), 2 * kMostWorkgroups));
  switch (D) {
    case 64: join_pieces_kernel<64, kRows, true, true><<<grid, 1024, 0, st>>>(c.heads, group, o, lse, joins, pieces, units, stride); break;
    case 128: join_pieces_kernel<128, kRows, true, true><<<grid, 1024, 0, st>>>(c.heads, group, o, lse, joins, pieces, units, stride); break;
    case 256: join_pieces_kernel<256, kRows, true, true><<<grid, 1024, 0, st>>>(c.heads, group, o, lse, joins, pieces, units, stride); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

// At least what every call of fewer tokens, sequences or rows needs, whichever kernel it goes to.
size_t paged_attention_ws(int D, int N, int heads, int group, int64_t n_tokens, int max_q, bool in_bf16, bool out_bf16) {
  CacheArgs c{};
  c.n_tokens = n_tokens;
  c.N = N;
  c.heads = heads;
  const int64_t rows = rows_of(c, group, max_q > 0 ? max_q : static_cast<int>(std::max<int64_t>(n_tokens, 1)));
  size_t bytes = 0;
  for (int mt = row_tiles(D, in_bf16, out_bf16, rows); mt > 0; mt /= 2) {
    const size_t wgs = workgroups(D, mt);
    bytes = std::max(bytes, wgs * sizeof(Split) + 2 * wgs * (16 * mt) * (D + 2) * 4);
  }
  if (for_chunks(D, c, group, in_bf16 && out_bf16, rows))
    bytes = std::max(bytes, attention_chunk_ws(D, std::min(most_chunk_units(c, group), kMostUnits)));
  return bytes;
}

hipError_t launch_paged_attention(int D, const CacheArgs& c, const void* q, int group, float scale, int max_q, void* o,
                                  float* lse, void* ws, bool in_bf16, bool out_bf16, hipStream_t st) {
  const int64_t rows = rows_of(c, group, max_q);
  if (for_chunks(D, c, group, in_bf16 && out_bf16, rows) && most_chunk_units(c, group) <= kMostUnits)
    return launch_attention_chunk(D, c, q, group, scale * kLog2e, rows, o, lse, ws, st);
  const int mt = row_tiles(D, in_bf16, out_bf16, rows);
  const int wgs = workgroups(D, mt);
  Split* splits = static_cast<Split*>(ws);
  float* pieces = reinterpret_cast<float*>(splits + wgs);
  const size_t shared = (static_cast<size_t>(c.N) + 1) * 8;
  auto go = [&](auto d, auto t, auto ib, auto ob) {
    constexpr int kD = decltype(d)::value, kT = decltype(t)::value;
    constexpr bool kOut = decltype(ob)::value;
    paged_attention_kernel<kD, kT, decltype(ib)::value, kOut>
        <<<dim3(wgs), kWaves * 64, shared, st>>>(c, q, group, scale * kLog2e, o, lse, splits, pieces);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    join_pieces_kernel<kD, 16 * kT, kOut, false><<<kMostWorkgroups, 1024, 0, st>>>(c.heads, group, o, lse, splits, pieces, wgs, 0);
    return hipGetLastError();
  };
  using std::integral_constant;
  using std::false_type;
  using std::true_type;
  const integral_constant<int, 1> one;
  const integral_constant<int, 2> two;
  const integral_constant<int, 4> four;
  auto by_type = [&](auto d) {
    constexpr int kD = decltype(d)::value;
    if (!out_bf16) return in_bf16 ? go(d, one, true_type{}, false_type{}) : go(d, one, false_type{}, false_type{});
    auto by_rows = [&](auto ib) {
      constexpr bool kIn = decltype(ib)::value;
      if (mt == 1) return go(d, one, ib, true_type{});
      if constexpr (kIn || kD == 64) {
        if (mt == 2) return go(d, two, ib, true_type{});
      }
      if constexpr (kIn && kD == 64) {
        if (mt == 4) return go(d, four, ib, true_type{});
      }
      return hipErrorInvalidValue;
    };
    return in_bf16 ? by_rows(true_type{}) : by_rows(false_type{});
  };
  switch (D) {
    case 64: return by_type(integral_constant<int, 64>{});
    case 128: return by_type(integral_constant<int, 128>{});
    case 256: return by_type(integral_constant<int, 256>{});
    default: return hipErrorInvalidValue;
  }
}

}  // namespace kda
