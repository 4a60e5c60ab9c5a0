// From rows of logits: log probabilities, entropy, top alternatives, the
// divergence from a teacher's entries, and their gradients.
//
// A row is cut into parts of 2,048 columns, a wave to a part.  With c the row's
// scale times log2 e, a part's record is its largest logit m, l = sum 2^t and a =
// sum t 2^t over t = c (x - m); the records of a row are joined by one wave,
//   M = max m,  u = c (m - M),  l' = sum l 2^u,  a' = sum (a + l u) 2^u,
// in an order that the row's length fixes.  Then log q = scale (x - M) - log l'
// and the entropy is log l' - ln 2 a' / l'.  A record needs no running maximum: the
// wave holds its part in registers, so its maximum comes first.
//
// Top alternatives, by (logit, then lowest index): the parts also note the
// largest logit of every 128 columns.  The k best columns lie in the k best
// groups of 128 by (largest logit, lowest group): a column outside has k groups
// that each hold a better one.  So the joining wave picks the k best groups (of
// more than 64 parts, first the k best parts), and reads those again: k * 128
// columns of a row.  Short rows are read again whole.
//
// Bound by memory: the logits are read once (gradients: and written once).  A
// column costs 8 instructions, so the sums over 4,096 x 131,072 keep the vector
// units busy four fifths of the time; there is little room for more.
//
// Measured (a kernel that reads 1.07 GB and does nothing else: 154 us): log probabilities and
// entropy of 4,096 x 131,072, bf16, 155 us, 6.9 TB/s; of 256 rows with 20 alternatives 24.5 us (parts 14.2,
// join 11.0); gradient of 2,048 rows 164 us, 1.0 GB moved, 6.1 TB/s.  Divergence from 64 entries,
// 2,048 rows, 84.9 us, 538 MB, 6.3 TB/s; its gradient 175 us, 1.07 GB, 6.1 TB/s, from 256 entries 187; in fp32
// 513 x 50,001 38.6 us, 205 MB, 5.3 TB/s.  Rows of one part, one launch: log probabilities and entropy of
// 60,000 x 900 52 us in bf16, 109 MB, 2.1 TB/s, and 50 in fp32, 217 MB, 4.4 TB/s: the vectors of a row's end are
// loaded one after the other, each waited for before the next, so latency bounds them.
#pragma once

#include "stack_device.hpp"

namespace stack {

constexpr int kPart = 2048;                     // columns of a record: 4 vectors of 8 to a lane
constexpr int kVecs = kPart / 512;
constexpr int kGroup = 128;                     // columns of a noted maximum
constexpr int kGroups = kPart / kGroup;
constexpr int kMaxParts = (1 << 20) / kPart;
constexpr int kWaves = 4;                       // waves of a work-group
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

struct LogitsArgs {
  const void* logits;
  int64_t stride;
  int64_t rows;
  int vocab, parts, top;
  const int32_t* targets;
  const float* scale;
  f32x4* rec;        // [rows][parts]: m, l, a
  float* group_max;  // [rows][parts][kGroups]
  float *logprobs, *entropy, *stats, *top_logprobs;
  int32_t* top_ids;
  // distill
  const int32_t* ids;
  const float* values;
  int given_logprobs;
  float* loss;
  // gradients
  const float *in_stats, *in_entropy, *d_logprobs, *d_entropy, *d_loss;
  void* d_logits;
  int64_t d_stride;
};

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// a lane's columns of a part: vector j holds 512 j + 8 lane .. + 7
template <class E, bool ONCE>
__device__ __forceinline__ void load_part(const typename E::T* p, int n, int lane, F8 (&x)[kVecs]) {
  typename E::RAW raw[kVecs];
  if (n >= kPart) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) raw[j] = E::template load<true, ONCE>(p + j * 512 + lane * 8);
#pragma unroll
    for (int j = 0; j < kVecs; ++j) x[j] = E::wide(raw[j]);
    return;
  }
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    const int c = j * 512 + lane * 8;
    const float none = -__builtin_inff();
    x[j] = F8{{none, none, none, none}, {none, none, none, none}};
    if (j * 512 >= n) continue;
    if (c + 8 <= n) {
      x[j] = E::wide(E::template load<true>(p + c));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < n) x[j][i] = E::one(p[c + i]);
    }
  }
}

__device__ __forceinline__ float max8(const F8& f) {
  return max3(max3(f.a[0], f.a[1], f.a[2]), max3(f.a[3], f.b[0], f.b[1]), max3(f.b[2], f.b[3], f.b[3]));
}

// row and part of this wave; false past the last
__device__ __forceinline__ bool my_part(const LogitsArgs& a, int64_t& row, int& part) {
  const uint32_t w = __builtin_amdgcn_readfirstlane(blockIdx.x * kWaves + (threadIdx.x >> 6));
  row = w / (uint32_t)a.parts;
  part = w - (uint32_t)row * a.parts;
  return row < a.rows;
}

__device__ __forceinline__ bool left_out(const LogitsArgs& a, int64_t row) {
  return a.targets && (uint32_t)a.targets[row] >= (uint32_t)a.vocab;
}

// The record of a part, the same in every lane; c: scale * log2 e.
template <class E, bool ENTROPY, bool TOP, bool ONCE>
__device__ __forceinline__ f32x4 part_record(const LogitsArgs& a, int64_t row, int part, float c, int lane) {
  const int n = a.vocab - part * kPart;  // a vector past the row's end has nothing to add
  F8 x[kVecs];
  load_part<E, ONCE>((const typename E::T*)a.logits + row * a.stride + part * kPart, n, lane, x);
  float m8[kVecs];
#pragma unroll
  for (int j = 0; j < kVecs; ++j) m8[j] = max8(x[j]);
  float m;
  if constexpr (TOP) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      m8[j] = max_16(m8[j]);
      if ((lane & 15) == 0) a.group_max[(row * a.parts + part) * kGroups + j * 4 + (lane >> 4)] = m8[j];
    }
    m = max_groups(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])));
  } else {
    m = max_groups(max_16(max3(max3(m8[0], m8[1], m8[2]), m8[3], m8[3])));
  }
  const float ref = m == -__builtin_inff() ? 0.f : m;
  // The exponent in one operation, t = c x - fl(c m): what rounding left of c m is
  // common to all and taken off the sums.  Where c m is so large that t would lose
  // its bits, in two.
  const float cm = c * ref, rest = __builtin_fmaf(c, ref, -cm);
  const bool large = __builtin_amdgcn_readfirstlane(!(__builtin_fabsf(cm) < 256.f));
  float l[kVecs], s[kVecs], lt, st = 0.f;
  if (!large) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      l[j] = s[j] = 0.f;
      if (j * 512 >= n) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float t = __builtin_fmaf(x[j][i], c, -cm), e = exp2_fast(t);
        l[j] += e;
        if constexpr (ENTROPY) s[j] = __builtin_fmaf(e, t, s[j]);
      }
    }
    lt = sum_lanes<64>((l[0] + l[1]) + (l[2] + l[3]));
    if constexpr (ENTROPY) {
      st = sum_lanes<64>((s[0] + s[1]) + (s[2] + s[3]));
      if (__builtin_amdgcn_readfirstlane(st != st)) {  // masked columns: 0 * -inf is to count 0
        float again = cm;
        asm("" : "+v"(again));  // or the exponentials above would be kept for this, in 64 more registers
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
          s[j] = 0.f;
          if (j * 512 >= n) continue;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float t = __builtin_fmaf(x[j][i], c, -again);
            s[j] = __builtin_fmaf(exp2_fast(t), fmaxf(t, -0x1p100f), s[j]);
          }
        }
        st = sum_lanes<64>((s[0] + s[1]) + (s[2] + s[3]));
      }
    }
    const float f = 1.f - rest * kLn2;
    st = (st - rest * lt) * f;
    lt *= f;
  } else {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      l[j] = s[j] = 0.f;
      if (j * 512 >= n) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float t = (x[j][i] - ref) * c, e = exp2_fast(t);
        l[j] += e;
        if constexpr (ENTROPY) s[j] = __builtin_fmaf(e, fmaxf(t, -0x1p100f), s[j]);
      }
    }
    lt = sum_lanes<64>((l[0] + l[1]) + (l[2] + l[3]));
    if constexpr (ENTROPY) st = sum_lanes<64>((s[0] + s[1]) + (s[2] + s[3]));
  }
  return f32x4{m, lt, st, 0.f};
}

template <class E, bool ENTROPY, bool TOP, bool ONCE>
__global__ __launch_bounds__(64 * kWaves) void k_stack_parts(const LogitsArgs a) {
  int64_t row;
  int part;
  if (!my_part(a, row, part) || left_out(a, row)) return;
  const int lane = threadIdx.x & 63;
  const f32x4 r = part_record<E, ENTROPY, TOP, ONCE>(a, row, part, (a.scale ? a.scale[row] : 1.f) * kLog2e, lane);
  if (lane == 0) a.rec[row * a.parts + part] = r;
}

// What a row's records add up to.
struct RowSum {
  float m, l, a;   // largest logit, sum of exponentials, sum of exponents times exponentials
  float log_l;     // 0 in a row of -inf only
  bool none;       // such a row
};

struct RowRecords {
  f32x4 r[kMaxParts / 64];
};

__device__ __forceinline__ void load_records(const LogitsArgs& a, int64_t row, int lane, RowRecords& q) {
  const f32x4* rec = a.rec + row * a.parts;
#pragma unroll
  for (int i = 0; i < kMaxParts / 64; ++i) {
    q.r[i] = f32x4{-__builtin_inff(), 0.f, 0.f, 0.f};
    if (i * 64 + lane < a.parts) q.r[i] = rec[i * 64 + lane];
  }
}

// What a row's wave does: joins the records that are there, or makes the one that
// there is, without or with the entropy's sum.
enum RowForm { kJoin, kMake, kMakeEntropy };

// A row of one part: its record is made by the wave that would join it, without a
// launch of its own (8,192 rows of 500: 7.2 us, 12.9 with; 300 of 2,000 with 20 entries 7.0 and 9.7).
// The entropy's sum is left out where it is not asked for, us without / with it: 60,000 x 900
// 43.3 / 51.3 in bf16, 43.3 / 47.9 in fp32, 60,000 x 2,000 52.5 / 63.6 and 80.2 / 82.1.
template <class E, bool ENTROPY>
__device__ __forceinline__ void make_record(const LogitsArgs& a, int64_t row, float c, int lane, RowRecords& q) {
#pragma unroll
  for (int i = 0; i < kMaxParts / 64; ++i) q.r[i] = f32x4{-__builtin_inff(), 0.f, 0.f, 0.f};
  const f32x4 r = part_record<E, ENTROPY, false, false>(a, row, 0, c, lane);
  if (lane == 0) q.r[0] = r;
}

__device__ __forceinline__ RowSum join_records(const LogitsArgs& a, float c, const RowRecords& q) {
  float m = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < kMaxParts / 64; ++i) m = fmaxf(m, q.r[i][0]);
  m = max_groups(max_16(m));
  float l = 0.f, s = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxParts / 64; ++i) {
    if (i * 64 >= a.parts) break;
    if (q.r[i][1] != 0.f) {  // a part of masked columns only has nothing to add
      const float t = (q.r[i][0] - m) * c, f = exp2_fast(t);
      l = __builtin_fmaf(q.r[i][1], f, l);
      s = __builtin_fmaf(__builtin_fmaf(q.r[i][1], fmaxf(t, -0x1p100f), q.r[i][2]), f, s);
    }
  }
  RowSum t;
  t.m = m;
  t.l = sum_lanes<64>(l);
  t.a = sum_lanes<64>(s);
  t.none = t.l == 0.f;
  if (t.l < 1.f && !t.none) t.l = 1.f;  // the largest logit's own share, but for rounding: log q is never above 0
  t.log_l = t.none ? 0.f : logf(t.l);
  return t;
}

// log q of a logit
__device__ __forceinline__ float log_q(const RowSum& t, float scale, float x) {
  return t.none ? -__builtin_inff() : __builtin_fmaf(x - t.m, scale, -t.log_l);
}

// A float's place in ascending order as a whole number; -0 is 0, a NaN is -inf.
__device__ __forceinline__ uint32_t order_of(float x) {
  x = x != x ? -__builtin_inff() : x + 0.f;
  const uint32_t u = __float_as_uint(x);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

__device__ __forceinline__ float of_order(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

__device__ __forceinline__ int lanes_below(uint64_t mask) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

// The wave's LDS writes before this are seen by its reads after it.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Sum over the lanes up to and with this one.
__device__ __forceinline__ int sum_up_to(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, true);   // row_shr:1
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, true);   // row_shr:2
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, true);   // row_shr:4
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, true);   // row_shr:8
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // row_bcast15: into rows 1 and 3
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);  // row_bcast31: into rows 2 and 3
  return x;
}

// The value of a key in units of STEP: the lower half of a bf16 value's order is
// its sign's.
template <uint32_t STEP>
__device__ __forceinline__ float value_of(uint32_t k) {
  return of_order(k * STEP + ((int32_t)(k * STEP) < 0 ? 0 : STEP - 1));
}

// Of up to 64 * N values (value N * lane + i in x[i], NaN where there is none)
// the `want` <= 64 largest, equal ones by ascending index: their indices go to
// `list` in ascending order.  None is above `best`.  Returns the key, in units
// of STEP, of a value that exactly they reach, or, where others are equal to
// the least of them, of that.  It is found by halving an interval of keys and
// counting, and the search ends once the count is right.  (Rolled up, as its
// code is run once and has to be fetched first.)
template <uint32_t STEP, int N>
__device__ __forceinline__ uint32_t select_largest(const float (&x)[N], int want, float best, int lane, int* list) {
  const auto reach = [&](float f) {
    int c = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) c += x[i] >= f;
    return __builtin_amdgcn_readlane(sum_up_to(c), 63);
  };
  // as many values as lanes have any reach the least of the lanes' largest
  float low = x[0];
#pragma unroll
  for (int i = 1; i < N; ++i) low = fmaxf(low, x[i]);
  low = __builtin_popcountll(__ballot(low == low)) < want ? -__builtin_inff() : -max_groups(max_16(-low));
  uint32_t lo = __builtin_amdgcn_readfirstlane(order_of(low) / STEP), hi = __builtin_amdgcn_readfirstlane(order_of(best) / STEP);
  int count = reach(value_of<STEP>(lo));
#pragma unroll 1
  while (lo < hi && count != want) {
    const uint32_t t = lo + (hi - lo + 1) / 2;
    const int c = reach(value_of<STEP>(t));
    if (c >= want) {
      lo = t;
      count = c;
    } else {
      hi = t - 1;
    }
  }
  uint32_t take = 0;
  const float f = value_of<STEP>(lo);
#pragma unroll
  for (int i = N - 1; i >= 0; --i) take = 2 * take + (x[i] >= f);
  if (count != want) {  // of those equal to the least, the first
    uint32_t above = 0;
    const float g = value_of<STEP>(lo + 1);
#pragma unroll
    for (int i = N - 1; i >= 0; --i) above = 2 * above + (x[i] >= g);
    const int over = __builtin_amdgcn_readlane(sum_up_to(__builtin_popcount(above)), 63);
    uint32_t equal = take & ~above;
    const int mine = __builtin_popcount(equal);
    int room = want - over - (sum_up_to(mine) - mine);
    take = above;
#pragma unroll 1
    for (; equal && room > 0; --room, equal &= equal - 1) take |= equal & -equal;
  }
  const int mine = __builtin_popcount(take);
  int at = sum_up_to(mine) - mine;
#pragma unroll 1
  for (; take && at < 64; take &= take - 1) list[at++] = N * lane + __builtin_ctz(take);
  return lo;
}

// Where a row's alternatives are sought: nowhere; among its columns themselves;
// among the largest of every 8 columns, then in the best of those; or among the
// noted largest of every 128, then in the best of those.
enum TopMode { kNoTop, kTopColumns, kTopEights, kTopGroups };

inline int top_mode(int vocab, int top) {
  return top == 0 ? kNoTop : vocab <= 1024 ? kTopColumns : vocab <= 8192 ? kTopEights : kTopGroups;
}

template <int MODE>
struct TopScratch {
  static constexpr int N = MODE == kTopColumns ? 64 : 1024;
  uint64_t found[N];  // columns held while the best are sought
  int parts[64], units[64];
};

// Keeps the `want` largest of the `count` different values found, in order.
template <int N>
__device__ __forceinline__ int keep_largest(uint64_t (&found)[N], int count, int want, int lane) {
  wave_sync();
  if (N == 64 || count <= 64) {  // the usual case: hardly more than are wanted
    const uint64_t v = lane < count ? found[lane] : 0;
    int rank = 0;
#pragma unroll 1
    for (int t = 0; t < count; ++t) {
      const uint64_t o = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), t) << 32 |
                         (uint32_t)__builtin_amdgcn_readlane((int)v, t);
      rank += o > v;
    }
    wave_sync();
    if (lane < count && rank < want) found[rank] = v;
    wave_sync();
    return min(count, want);
  }
  uint64_t v[N / 64];
  int rank[N / 64];
#pragma unroll
  for (int i = 0; i < N / 64; ++i) {
    rank[i] = 0;
    v[i] = i * 64 + lane < count ? found[i * 64 + lane] : 0;
  }
#pragma unroll 4
  for (int t = 0; t < count; ++t) {
    const uint64_t o = found[t];
#pragma unroll
    for (int i = 0; i < N / 64; ++i)
      if (i * 64 < count) rank[i] += o > v[i];
  }
  wave_sync();
#pragma unroll
  for (int i = 0; i < N / 64; ++i)
    if (v[i] && rank[i] < want) found[rank[i]] = v[i];
  wave_sync();
  return min(count, want);
}

constexpr int kHeld = 16;  // values of a lane among which the largest are sought

// A value to seek among: a NaN ranks as -inf, and there is none where it ends.
__device__ __forceinline__ float held(float x, bool there) {
  return there ? fmaxf(x, -__builtin_inff()) : __uint_as_float(0x7fc00000u);
}

// eight columns of a row; past its end 0
template <class E>
__device__ __forceinline__ F8 load_eight(const typename E::T* x, int c, int vocab) {
  F8 f = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  if (c + 8 <= vocab) {
    f = E::wide(E::template load<true>(x + c));
  } else if (c < vocab) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < vocab) f[i] = E::one(x[c + i]);
  }
  return f;
}

// The noted maxima of a part of a row.
__device__ __forceinline__ void load_groups(const LogitsArgs& a, int64_t row, int part, bool there, float (&x)[kHeld]) {
  const f32x4* gm = (const f32x4*)(a.group_max + (row * a.parts + part) * kGroups);
#pragma unroll
  for (int i = 0; i < kHeld / 4; ++i) {
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (there) v = gm[i];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[4 * i + e] = held(v[e], there && part * kPart + (4 * i + e) * kGroup < a.vocab);
  }
}

// The values of a row's first search: lane l's are those of columns 16 l .. 16 l
// + 15, of units 16 l .. of 8 columns, or of part l (of up to 64 parts).  turn:
// LDS for 1,024 of them.
template <class E, int MODE>
__device__ __forceinline__ void load_values(const LogitsArgs& a, int64_t row, int lane, float* turn, float (&x)[kHeld]) {
  const typename E::T* p = (const typename E::T*)a.logits + row * a.stride;
  if constexpr (MODE == kTopColumns) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      F8 f = load_eight<E>(p, kHeld * lane + 8 * h, a.vocab);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[8 * h + i] = held(f[i], kHeld * lane + 8 * h + i < a.vocab);
    }
  } else if constexpr (MODE == kTopEights) {
    // read unit by unit along the row, handed to their lanes through LDS
#pragma unroll 8
    for (int i = 0; i < kHeld; ++i) {
      const int c = (i * 64 + lane) * 8;
      F8 f = load_eight<E>(p, c, a.vocab);
      float m = -__builtin_inff();
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e < a.vocab) m = fmaxf(m, f[e]);
      turn[i * 64 + lane] = m;
    }
    wave_sync();
#pragma unroll
    for (int i = 0; i < kHeld; ++i) x[i] = held(turn[kHeld * lane + i], (kHeld * lane + i) * 8 < a.vocab);
    wave_sync();
  } else if constexpr (MODE == kTopGroups) {
    if (a.parts <= 64) load_groups(a, row, min(lane, a.parts - 1), lane < a.parts, x);
  }
}

// The row's a.top best columns, in order, in found[]: order_of(logit) above the
// index's complement.  v: load_values.
template <class E, int MODE>
__device__ __forceinline__ void top_columns(const LogitsArgs& a, int64_t row, int lane, const RowRecords& q,
                                            float (&v)[kHeld], float best, TopScratch<MODE>& t) {
  constexpr uint32_t STEP = 1u << (32 - 8 * sizeof(typename E::T));  // keys of bf16 values are so far apart
  const typename E::T* x = (const typename E::T*)a.logits + row * a.stride;
  const auto entry = [&](float f, int c) { return (uint64_t)order_of(f) << 32 | (uint32_t)~c; };
  const bool direct = MODE != kTopGroups || a.parts <= 64;
  if (!direct) {  // the best parts first, as many as there are alternatives
    float* m = (float*)t.found;
#pragma unroll
    for (int i = 0; i < kMaxParts / 64; ++i) m[i * 64 + lane] = q.r[i][0];
    wave_sync();
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int at = kHeld * lane + i;
      v[i] = held(m[at & (kMaxParts - 1)], at < a.parts);
    }
  }
  uint32_t least = 0;
#pragma unroll 1
  for (int level = direct; level < 2; ++level) {
    least = select_largest<STEP, kHeld>(v, a.top, best, lane, t.units);
    wave_sync();
    if (level == 0) {  // then the groups of part l of those in lane l
      t.parts[lane] = lane < a.top ? t.units[lane] : 0;
      load_groups(a, row, min((uint32_t)t.parts[lane], (uint32_t)a.parts - 1), lane < a.top, v);
    } else if (!direct && lane < a.top) {
      const int at = t.units[lane];
      t.units[lane] = t.parts[(at / kGroups) & 63] * kGroups + at % kGroups;
    }
    wave_sync();
  }
  if constexpr (MODE == kTopColumns) {
    if (lane < a.top) {
      const int c = min((uint32_t)t.units[lane], (uint32_t)a.vocab - 1);
      t.found[lane] = entry(E::one(x[c]), c);
    }
    keep_largest(t.found, a.top, a.top, lane);
    return;
  }
  // Their columns.  At least as many as asked for reach the least of as many
  // units; of those equal to it, no more than asked for are needed, the first
  // ones, and the units come in ascending order.
  constexpr int W = MODE == kTopGroups ? 16 : 1, U = 64 / W;  // lanes to a unit, units at a time
  const float exact = value_of<STEP>(least);
  uint64_t bar = 0;
  int count = 0, equal = 0;
  const auto column = [&](int which) {
    which += lane / W;
    return which < a.top ? (int)min(((uint32_t)t.units[which] * W + lane % W) * 8, (uint32_t)a.vocab) : a.vocab;
  };
  constexpr int B = MODE == kTopGroups ? 4 : 1;  // loads of a lane under way: one is used, the others are ahead
  typename E::RAW raw[B];
  int col[B];
#pragma unroll
  for (int j = 0; j < B; ++j) {
    col[j] = column(U * j);
    if (col[j] + 8 <= a.vocab) raw[j] = E::template load<true>(x + col[j]);
  }
#pragma unroll 1
  for (int s = 0;; s += U) {
    if (count > t.N - 512 - 64 || s >= a.top) {
      count = keep_largest(t.found, count, a.top, lane);
      if (count == a.top) bar = t.found[count - 1];
    }
    if (s >= a.top) break;
    const int c = col[0];
    F8 f = E::wide(raw[0]);
#pragma unroll
    for (int j = 1; j < B; ++j) {
      col[j - 1] = col[j];
      raw[j - 1] = raw[j];
    }
    if constexpr (B > 1) {
      col[B - 1] = column(s + U * B);
      if (col[B - 1] + 8 <= a.vocab) raw[B - 1] = E::template load<true>(x + col[B - 1]);
    }
    if (c + 8 > a.vocab) f = load_eight<E>(x, c, a.vocab);
    uint32_t some = 0, same = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float g = held(f[i], c + i < a.vocab);
      some |= g > exact ? 1u << i : 0u;
      same |= g == exact ? 1u << i : 0u;
    }
    if (equal < a.top && __ballot(same != 0)) {
      const int mine = __builtin_popcount(same), upto = sum_up_to(mine);
      int room = a.top - equal - (upto - mine);
#pragma unroll 1
      for (; same && room > 0; --room, same &= same - 1) some |= same & -same;
      equal += __builtin_amdgcn_readlane(upto, 63);
    }
    // few are left: a lane's are taken one after the other
#pragma unroll 1
    while (__ballot(some != 0)) {
      const int at = __builtin_ctz(some | 256u);
      float g = f[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) g = at == i ? f[i] : g;
      const uint64_t e = entry(g, c + at);
      const bool take = some != 0 && e > bar;
      const uint64_t taken = __ballot(take);
      if (take) t.found[count + lanes_below(taken)] = e;
      count += __builtin_popcountll(taken);
      some &= some - 1;
    }
  }
}

template <class E, int MODE, RowForm FORM>
__global__ __launch_bounds__(64 * kWaves) void k_stack_logprobs(const LogitsArgs a) {
  __shared__ TopScratch<MODE> scratch[MODE ? kWaves : 1];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * kWaves + wave;
  if (row >= a.rows) return;
  RowRecords q;
  if (FORM == kJoin) load_records(a, row, lane, q);
  if (left_out(a, row)) {
    if (lane == 0) {
      a.logprobs[row] = 0.f;
      if (a.entropy) a.entropy[row] = 0.f;
      if (a.stats) a.stats[2 * row] = a.stats[2 * row + 1] = 0.f;
    }
    if (MODE && lane < a.top) {
      a.top_ids[row * a.top + lane] = -1;
      a.top_logprobs[row * a.top + lane] = 0.f;
    }
    return;
  }
  float v[kHeld];
  load_values<E, MODE>(a, row, lane, (float*)scratch[MODE ? wave : 0].found, v);
  const float scale = a.scale ? a.scale[row] : 1.f;
  const typename E::T* x = (const typename E::T*)a.logits + row * a.stride;
  const float at_target = a.targets ? E::one(x[a.targets[row]]) : 0.f;
  if (FORM != kJoin) make_record<E, FORM == kMakeEntropy>(a, row, scale * kLog2e, lane, q);
  const RowSum t = join_records(a, scale * kLog2e, q);
  if (lane == 0) {
    if (a.targets) a.logprobs[row] = log_q(t, scale, at_target);
    if (a.entropy) a.entropy[row] = t.none ? 0.f : t.log_l - kLn2 * (t.a / t.l);
    if (a.stats) {
      a.stats[2 * row] = t.m;
      a.stats[2 * row + 1] = t.log_l;
    }
  }
  if constexpr (MODE != kNoTop) {
    TopScratch<MODE>& s = scratch[wave];
    top_columns<E, MODE>(a, row, lane, q, v, t.m, s);
    if (lane < a.top) {
      const uint64_t e = s.found[lane];
      a.top_ids[row * a.top + lane] = (int32_t)~(uint32_t)e;
      a.top_logprobs[row * a.top + lane] = log_q(t, scale, of_order((uint32_t)(e >> 32)));
    }
  }
}

// Gradients: a wave to a part, column by column, so a lane's columns may be
// others: as many runs of 16 bytes as its eight elements are, a wave's runs side
// by side.  (Two loads of a lane side by side, as above, share their lines; read
// or written past the caches those would move twice.)
template <class E>
struct Runs {
  static constexpr int N = 16 / (int)sizeof(typename E::T), R = 8 / N;  // elements of a run, runs of a vector
  static __device__ __forceinline__ int column(int j, int r, int lane) { return j * 512 + r * (512 / R) + lane * N; }
};

template <class E, bool ONCE>
__device__ __forceinline__ void load_runs(const typename E::T* p, int n, int lane, F8 (&x)[kVecs]) {
  typedef Runs<E> L;
  u32x4 raw[kVecs * L::R];
#pragma unroll
  for (int j = 0; j < kVecs; ++j)
#pragma unroll
    for (int r = 0; r < L::R; ++r) {
      const int c = L::column(j, r, lane);
      if (n >= kPart || c + L::N <= n) {
        const auto* at = (const typename Pick<true>::U*)(p + c);
        raw[j * L::R + r] = ONCE ? __builtin_nontemporal_load(at) : *at;
      }
    }
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    E::widen(x[j], raw + j * L::R);
    if (n >= kPart) continue;
#pragma unroll
    for (int r = 0; r < L::R; ++r) {
      const int c = L::column(j, r, lane);
      if (c + L::N > n) {
#pragma unroll
        for (int i = 0; i < L::N; ++i) x[j][r * L::N + i] = c + i < n ? E::one(p[c + i]) : -__builtin_inff();
      }
    }
  }
}

template <class E, bool ONCE>
__device__ __forceinline__ void store_runs(typename E::T* p, int n, int lane, F8 (&x)[kVecs]) {
  typedef Runs<E> L;
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    u32x4 raw[L::R];
    E::narrow_to(x[j], raw);
#pragma unroll
    for (int r = 0; r < L::R; ++r) {
      const int c = L::column(j, r, lane);
      if (c + L::N <= n) {
        auto* at = (typename Pick<true>::U*)(p + c);
        if constexpr (ONCE)
          __builtin_nontemporal_store(raw[r], at);
        else
          *at = raw[r];
      } else {
#pragma unroll
        for (int i = 0; i < L::N; ++i)
          if (c + i < n) p[c + i] = E::round(x[j][r * L::N + i]);
      }
    }
  }
}

// Gradient of log probability and entropy.
template <class E, bool ENTROPY, bool ONCE>
__global__ __launch_bounds__(64 * kWaves) void k_stack_logprobs_bwd(const LogitsArgs a) {
  int64_t row;
  int part;
  if (!my_part(a, row, part)) return;
  const int lane = threadIdx.x & 63, n = a.vocab - part * kPart;
  typename E::T* out = (typename E::T*)a.d_logits + row * a.d_stride + part * kPart;
  const float m = a.in_stats[2 * row], log_l = a.in_stats[2 * row + 1];
  const bool zero = left_out(a, row) || (m == -__builtin_inff() && log_l == 0.f);
  const float scale = a.scale ? a.scale[row] : 1.f;
  const float g = a.d_logprobs ? a.d_logprobs[row] * scale : 0.f;
  const float f = ENTROPY ? a.d_entropy[row] * scale : 0.f, h = ENTROPY ? a.in_entropy[row] : 0.f;
  F8 x[kVecs];
  if (zero) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) x[j] = F8{{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  } else {
    load_runs<E, ONCE>((const typename E::T*)a.logits + row * a.stride + part * kPart, n, lane, x);
    const float c = scale * kLog2e, off = -log_l * kLog2e, up = h - log_l;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = x[j][i] - m;
        const float p = exp2_fast(__builtin_fmaf(d, c, off));
        float k = g;
        // where q is 0 (log q below -104, as of a masked column) log q + h is held to -128, so that
        // no f makes an infinity of it: 0 * inf would be NaN
        if constexpr (ENTROPY) k = __builtin_fmaf(f, fmaxf(__builtin_fmaf(d, scale, up), -128.f), g);
        x[j][i] = -p * k;
      }
    }
    if (a.targets && a.d_logprobs) {
      const int at = a.targets[row] - part * kPart;
      if (at >= 0 && at < kPart) {
        typedef Runs<E> L;
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
#pragma unroll
          for (int r = 0; r < L::R; ++r) {
            const int e = at - L::column(j, r, lane);
            if (e >= 0 && e < L::N) {
#pragma unroll
              for (int i = 0; i < L::N; ++i) x[j][r * L::N + i] += e == i ? g : 0.f;
            }
          }
      }
    }
  }
  store_runs<E, ONCE>(out, n, lane, x);
}

// ---------------------------------------------------------------------------
// distillation

constexpr int kEntries = 256 / 64;  // teacher's entries to a lane

struct Teacher {
  int id[kEntries];       // -1: not there
  float logp[kEntries];   // -inf: not there
};

__device__ __forceinline__ void load_teacher(const LogitsArgs& a, int64_t row, int lane, Teacher& t) {
#pragma unroll
  for (int i = 0; i < kEntries; ++i) {
    const int e = i * 64 + lane;
    int id = -1;
    float value = 0.f;
    if (e < a.top) {
      id = a.ids[row * a.top + e];
      value = a.values[row * a.top + e];
    }
    const bool there = (uint32_t)id < (uint32_t)a.vocab;
    t.id[i] = there ? id : -1;
    t.logp[i] = there ? value : -__builtin_inff();
  }
}

__device__ __forceinline__ void normalise(Teacher& t, float scale, float m, float log_l) {
#pragma unroll
  for (int i = 0; i < kEntries; ++i) t.logp[i] = __builtin_fmaf(t.logp[i] - m, scale, -log_l);
}

template <class E, RowForm FORM>
__global__ __launch_bounds__(64 * kWaves) void k_stack_distill(const LogitsArgs a) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * kWaves + wave;
  if (row >= a.rows) return;
  const float scale = a.scale ? a.scale[row] : 1.f;
  const typename E::T* x = (const typename E::T*)a.logits + row * a.stride;
  RowRecords q;
  if (FORM == kJoin) load_records(a, row, lane, q);
  Teacher te;
  load_teacher(a, row, lane, te);
  float s[kEntries];
#pragma unroll
  for (int i = 0; i < kEntries; ++i) s[i] = te.id[i] >= 0 ? E::one(x[te.id[i]]) : 0.f;
  if (FORM != kJoin) make_record<E, FORM == kMakeEntropy>(a, row, scale * kLog2e, lane, q);
  const RowSum t = join_records(a, scale * kLog2e, q);
  float m = 0.f, log_l = 0.f;
  if (!a.given_logprobs) {
    m = te.logp[0];
#pragma unroll
    for (int i = 1; i < kEntries; ++i) m = fmaxf(m, te.logp[i]);
    m = max_groups(max_16(m));
    if (m == -__builtin_inff()) m = 0.f;
    float l = 0.f;
#pragma unroll
    for (int i = 0; i < kEntries; ++i) l += expf((te.logp[i] - m) * scale);
    l = sum_lanes<64>(l);
    log_l = l == 0.f ? 0.f : logf(l);
    normalise(te, scale, m, log_l);
  }
  float loss = 0.f;
#pragma unroll
  for (int i = 0; i < kEntries; ++i) {
    const float p = expf(te.logp[i]);
    if (p != 0.f) loss = __builtin_fmaf(p, te.logp[i] - log_q(t, scale, s[i]), loss);
  }
  loss = sum_lanes<64>(loss);
  if (lane == 0) {
    a.loss[row] = loss;
    if (a.stats) *(f32x4*)(a.stats + 4 * row) = f32x4{t.m, t.log_l, m, log_l};
  }
}

// The wave's stores before this are done when those after it begin.  The fences keep
// the compiler from moving any across; that of a work-group makes no wait for stores on this
// target, whose waves' stores to an address stay in order, so the wait is one of its
// own (2,048 x 131,072, bf16, 64 entries: 175.8 us, without 178.6).
__device__ __forceinline__ void stores_done() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
}

// Gradient.  Every column is first stored as if it were no entry; the wave then
// writes over those that are.
template <class E, bool ONCE>
__global__ __launch_bounds__(64 * kWaves) void k_stack_distill_bwd(const LogitsArgs a) {
  __shared__ uint16_t owner[kWaves][kPart];
  int64_t row;
  int part;
  if (!my_part(a, row, part)) return;
  const int lane = threadIdx.x & 63, n = a.vocab - part * kPart;
  const typename E::T* in = (const typename E::T*)a.logits + row * a.stride + part * kPart;
  typename E::T* out = (typename E::T*)a.d_logits + row * a.d_stride + part * kPart;
  const f32x4 st = *(const f32x4*)(a.in_stats + 4 * row);
  const float m = st[0], log_l = st[1];
  const float scale = a.scale ? a.scale[row] : 1.f, g = a.d_loss[row] * scale;
  F8 x[kVecs];
  load_runs<E, ONCE>(in, n, lane, x);
  Teacher te;
  load_teacher(a, row, lane, te);
  if (!a.given_logprobs) normalise(te, scale, st[2], st[3]);
  float p[kEntries], s[kEntries], total = 0.f;
  uint64_t here[kEntries], any = 0;
#pragma unroll
  for (int i = 0; i < kEntries; ++i) {
    p[i] = expf(te.logp[i]);
    total += p[i];
    te.id[i] -= part * kPart;
    const bool mine = (uint32_t)te.id[i] < kPart;
    here[i] = __ballot(mine);
    any |= here[i];
    s[i] = mine ? E::one(in[te.id[i]]) : 0.f;
  }
  total = sum_lanes<64>(total);
  const bool zero = total == 0.f || (m == -__builtin_inff() && log_l == 0.f);
  const float c = scale * kLog2e, off = -log_l * kLog2e, k = g * total;
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[j][i] = zero ? 0.f : exp2_fast(__builtin_fmaf(x[j][i] - m, c, off)) * k;
  }
  store_runs<E, ONCE>(out, n, lane, x);
  if (any == 0 || zero) return;
  // An index that comes once takes its own p.  Entries of one index see another's
  // number where they left theirs; then the part's entries go one after the other,
  // each adds up the p of those of its index, and the first of them stores.
  float sum[kEntries];
  bool later[kEntries], twice = false;
  uint16_t* left = owner[threadIdx.x >> 6];
#pragma unroll
  for (int i = 0; i < kEntries; ++i) {
    if ((uint32_t)te.id[i] < kPart) left[te.id[i]] = i * 64 + lane;
    sum[i] = p[i];
    later[i] = false;
  }
  wave_sync();
#pragma unroll
  for (int i = 0; i < kEntries; ++i)
    if ((uint32_t)te.id[i] < kPart) twice |= left[te.id[i]] != i * 64 + lane;
  if (__ballot(twice)) {
#pragma unroll
    for (int i = 0; i < kEntries; ++i) sum[i] = 0.f;
#pragma unroll
    for (int i = 0; i < kEntries; ++i) {
#pragma unroll 1
      for (uint64_t rest = here[i]; rest; rest &= rest - 1) {
        const int who = __builtin_ctzll(rest);
        const int id = __builtin_amdgcn_readlane(te.id[i], who);
        const float pe = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(p[i]), who));
#pragma unroll
        for (int j = 0; j < kEntries; ++j) {
          const bool same = te.id[j] == id;
          sum[j] += same ? pe : 0.f;
          later[j] |= same && (j > i || (j == i && lane > who));
        }
      }
    }
  }
  stores_done();  // other lanes write to the same places now
#pragma unroll
  for (int i = 0; i < kEntries; ++i)
    if ((uint32_t)te.id[i] < kPart && !later[i]) out[te.id[i]] = E::round(g * (exp2_fast(__builtin_fmaf(s[i] - m, c, off)) * total - sum[i]));
}

}  // namespace stack
