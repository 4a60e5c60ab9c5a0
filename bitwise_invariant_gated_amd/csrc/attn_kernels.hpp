// Causal attention over the 8-bit cache: prefill (any number of new tokens
// per sequence) and the decode step.
//
// Arithmetic, the same in every kernel, per query row and in this order:
//   keys in partitions of 512; in a partition the 8-bit blocks before the
//   row's own in ascending order, then, in the last one, the own block's
//   tokens up to the row in the input type.  A block of 64 keys is one tile:
//     s    = K q, v_mfma_f32_16x16x32_bf16, k steps ascending (dims 64 kp +
//            16 g + 8 h .. + 7 in slot group g of step 2 kp + h)
//     m'   = max(m, c max(s)), c = scale * log2(e)
//     p    = exp2(fma(s, c, -m')), alpha = exp2(m - m')
//     l    = fma(l, alpha, sum p)   four partial sums per row, by lane group
//     O    = alpha O + V^T p, p in bf16, two MFMA k steps
//   partitions: (m, l, O) = fold of the total and the partition, left to
//   right: O = fma(Op, exp2(mp - m'), O exp2(m - m')).
//   o = O (1 / l), l's partial sums added as (0 + 1) + (2 + 3).
// A masked tile leaves a row's state as it is (alpha = 1, p = 0), so which
// tiles a kernel walks through for a row beyond its own does not matter,
// and neither does which work-group does which partition.
//
// Operand layout: the tile is computed transposed, S^T = K Q^T, so that a
// lane (r = lane % 16, g = lane / 16) holds scores of one query row r: of the
// keys 16 g + 4 a + i for register i of sub-tile a, if sub-tile a's A
// rows are the keys 16 (x / 4) + 4 a + x % 4.  Then a lane's p are of 16
// consecutive keys and are the B operand of O^T = V^T P^T as they stand, with
// V^T rows (the cache holds V per dim) giving the A operand in 16 consecutive
// bytes: softmax statistics are one value per lane, and neither S nor P nor V
// is ever transposed or moved between lanes.
#pragma once

#include <type_traits>

#include "attn_cache_kernels.hpp"

namespace attn {

constexpr int kPart = 512;               // keys of a partition
constexpr int kPartBlocks = kPart / 64;  // tiles of a partition
constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// key of a sub-tile's A row x
__device__ __forceinline__ int key_of(int a, int x) { return 16 * (x >> 2) + 4 * a + (x & 3); }

// max of a lane's 16 scores
__device__ __forceinline__ float max16(const f32x4 (&s)[4]) {
  float m = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3]));
#pragma unroll
  for (int a = 1; a < 4; ++a) m = fmaxf(m, fmaxf(fmaxf(s[a][0], s[a][1]), fmaxf(s[a][2], s[a][3])));
  return m;
}

// scores -> p: their bf16 B fragments for the two PV steps, and their sum
__device__ __forceinline__ float probabilities(const f32x4 (&s)[4], float c, float m, u32x4 (&p)[2]) {
  float sum[4];
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    float e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = exp2_(__builtin_fmaf(s[a][i], c, -m));
    sum[a] = (e[0] + e[1]) + (e[2] + e[3]);
    p[a >> 1][2 * (a & 1)] = pack2(e[0], e[1]);
    p[a >> 1][2 * (a & 1) + 1] = pack2(e[2], e[3]);
  }
  return (sum[0] + sum[1]) + (sum[2] + sum[3]);
}

// the running max as a reference for exp2 (a row that has seen nothing: 0)
__device__ __forceinline__ float ref_of(float m) { return m == kNegInf ? 0.f : m; }

// Weights of the total and of a partition in their fold, and the new max.
__device__ __forceinline__ void fold_weights(float& m, float mp, float& a, float& b) {
  const float mn = fmaxf(m, mp), ref = ref_of(mn);
  a = exp2_(m - ref);
  b = exp2_(mp - ref);
  m = mn;
}

// ---------------------------------------------------------------------------
// prefill

// Rows of a (sequence, key/value head): row r is token r / G, query head
// hk G + r % G.  A work-group takes kRows of them, a wave 16 kRT, and all of it
// walks the keys together: a tile is converted to bf16 once per work-group
// into LDS, in the order the MFMA operands are read (conflict-free, 16
// bytes per lane), while the bytes of the next one are in flight from memory.
//
// The 8-bit blocks come first, all in one loop (those from the work-group's
// first own block on are masked per row), then the rows' own blocks, kRaw of
// them staged at once, so that every wave does its own without waiting for
// the others'.
template <int D>
struct PrefillTile {
  static constexpr int kRT = D == 256 ? 1 : 2;   // 16-row tiles of a wave
  static constexpr int kWaves = 8;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kRows = 16 * kRT * kWaves;
  static constexpr int kFrags = 4 * (D / 32);    // 1 KiB each, K; as many for V
  static constexpr int kUnits = 4 * (D / 64);    // 1 KiB loads of an 8-bit block, K; as many for V
  static constexpr bool kSplit = kUnits < kWaves;  // d = 64: half of the waves load K, half V
  static constexpr int kPer = kSplit ? 1 : kUnits / kWaves;  // units of a wave, K and V each
  static constexpr int kRaw = D == 64 ? 4 : 2;  // LDS buffers
  // dim tiles of the folded total that are kept in LDS (each thread its own), for want of registers
  static constexpr int kOtLds = D == 128 ? 4 : 0;
};

template <int D>
struct PrefillLds {
  u32x4 k[PrefillTile<D>::kFrags * 64];
  u32x4 v[PrefillTile<D>::kFrags * 64];
};

// Where V's fragment (dt, h) keeps a lane's 16 bytes: rows change places by dt in
// groups of four, so that writing four keys of neighbouring dims (own blocks) spreads over the banks.
__device__ __forceinline__ int v_slot(int dt, int h, int lane) { return (dt * 2 + h) * 64 + (lane ^ (dt & 3)); }

// Pool blocks and scales of 64 blocks of a row at a time, one per lane: the
// loop over the blocks then waits for none of the two dependent loads.
struct BlockRun {
  int id;
  float ks, vs;
};

__device__ __forceinline__ BlockRun load_run(const StepArgs& a, int row, int hk, int b, int lane) {
  BlockRun x;
  x.id = pool_block(a, row, b + lane);
  const int64_t at = (int64_t)x.id * a.Hk + hk;
  x.ks = a.cache.k_scale[at];
  x.vs = a.cache.v_scale[at];
  return x;
}

__device__ __forceinline__ float lane_of(float x, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), lane));
}

template <int D>
struct Bytes {  // a wave's share of an 8-bit block in flight
  u32x4 k[PrefillTile<D>::kPer], v[PrefillTile<D>::kPer];
  float ks, vs;
};

template <int D>
__device__ __forceinline__ void load_block(const StepArgs& a, const BlockRun& run, int hk, int b, Bytes<D>& y, int wave,
                                           int lane) {
  typedef PrefillTile<D> P;
  const int r = lane & 15, g = lane >> 4;
  const int64_t at = (int64_t)__builtin_amdgcn_readlane(run.id, b & 63) * a.Hk + hk;
  y.ks = lane_of(run.ks, b & 63);
  y.vs = lane_of(run.vs, b & 63);
#pragma unroll
  for (int n = 0; n < P::kPer; ++n) {
    const int unit = (wave + P::kWaves * n) % P::kUnits;
    const int sub = unit & 3, kp = unit >> 2;
    if (!P::kSplit || wave < P::kUnits)
      y.k[n] = *(const u32x4*)(a.cache.k8 + at * (64 * D) + kp * 4096 + key_of(sub, r) * 64 + g * 16);
    if (!P::kSplit || wave >= P::kUnits)
      y.v[n] = *(const u32x4*)(a.cache.v8 + at * (64 * D) + (unit * 16 + r) * 64 + g * 16);
  }
}

// V that is not finite must not reach rows that do not see it: in a masked
// tile 0 * NaN would.  keys16: bit e is set if the lane's key 16 g + e has such a value
// in one of the lane's dims; returns the wave's 64 keys.
__device__ __forceinline__ uint64_t bad_keys(uint32_t keys16) {
  if (!__any(keys16 != 0)) return 0;
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) keys16 |= (uint32_t)__shfl_xor((int)keys16, o);
  uint64_t m = 0;
#pragma unroll
  for (int g = 0; g < 4; ++g) m |= (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)keys16, 16 * g) << (16 * g);
  return m;
}

// The A fragment of V^T step h with the keys of `drop` set to zero.
__device__ __forceinline__ u32x4 drop_keys(u32x4 v, uint64_t drop, int g, int h) {
  const uint32_t d = (uint32_t)(drop >> (16 * g + 8 * h)) & 0xffu;
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] &= ((d >> (2 * j)) & 1 ? 0u : 0xffffu) | ((d >> (2 * j + 1)) & 1 ? 0u : 0xffff0000u);
  return v;
}

template <int D>
__device__ __forceinline__ void store_block(const Bytes<D>& y, PrefillLds<D>& sm, int wave, int lane) {
  typedef PrefillTile<D> P;
#pragma unroll
  for (int n = 0; n < P::kPer; ++n) {
    const int unit = (wave + P::kWaves * n) % P::kUnits;
    const int sub = unit & 3, kp = unit >> 2;
    u32x4 lo, hi;
    if (!P::kSplit || wave < P::kUnits) {
      from_e4m3(y.k[n], y.ks, lo, hi);
      sm.k[(sub * (D / 32) + 2 * kp) * 64 + lane] = lo;
      sm.k[(sub * (D / 32) + 2 * kp + 1) * 64 + lane] = hi;
    }
    if (!P::kSplit || wave >= P::kUnits) {
      from_e4m3(y.v[n], y.vs, lo, hi);
      sm.v[v_slot(unit, 0, lane)] = lo;
      sm.v[v_slot(unit, 1, lane)] = hi;
    }
  }
}

// The keys of this wave's share of V that are not finite.
template <int D>
__device__ __forceinline__ uint64_t bad_in_block(const Bytes<D>& y, int wave) {
  typedef PrefillTile<D> P;
  uint32_t nan16 = 0;
  if (!P::kSplit || wave >= P::kUnits) {
#pragma unroll
    for (int n = 0; n < P::kPer; ++n)
#pragma unroll
      for (int e = 0; e < 16; ++e) nan16 |= ((y.v[n][e >> 2] >> (8 * (e & 3))) & 0x7f) == 0x7f ? 1u << e : 0u;
  }
  return bad_keys(nan16);
}

// A block in the input type: the call's tokens, and the tail as it was for
// the ones before.  Past the sequence's end: zeros.  K goes as it is; of V a
// thread takes four keys of four dims and writes them turned.  Returns the
// wave's keys with a V that is not finite.
template <int D>
__device__ __forceinline__ uint64_t stage_raw(const StepArgs& a, int i, int hk, int ctx, int end, int c0, int b,
                                              PrefillLds<D>& sm, int wave, int lane) {
  typedef PrefillTile<D> P;
  constexpr int NK = (P::kUnits + P::kWaves - 1) / P::kWaves, NV = (64 / 4) * (D / 4) / P::kThreads;
  const int r = lane & 15, g = lane >> 4;
  const int64_t tail = ((int64_t)i * a.Hk + hk) * (64 * D);
  const int64_t from = (int64_t)c0 - ctx;
  u32x4 lo[NK], hi[NK];
  u32x2 x[NV < 1 ? 1 : NV][4];
  constexpr int NVR = NV < 1 ? 1 : NV;
#pragma unroll
  for (int n = 0; n < NK; ++n) {
    const int unit = wave + P::kWaves * n, sub = unit & 3, kp = unit >> 2, key = key_of(sub, r), p = b * 64 + key;
    lo[n] = hi[n] = u32x4{0, 0, 0, 0};
    if (unit < P::kUnits && p < end) {
      const uint16_t* src = (p >= ctx ? a.k + (from + p) * a.k_stride + (int64_t)hk * D : a.old_k + tail + key * D) + kp * 64 + g * 16;
      lo[n] = *(const u32x4*)src;
      hi[n] = *(const u32x4*)(src + 8);
    }
  }
  uint64_t bad = 0;
#pragma unroll
  for (int n = 0; n < NVR; ++n) {
    const int it = wave * 64 + lane + P::kThreads * n, kq = it / (D / 4), dim = it % (D / 4) * 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int key = 4 * kq + j, p = b * 64 + key;
      x[n][j] = u32x2{0, 0};
      if (kq < 16 && p < end) {
        if (p >= ctx) {
          x[n][j] = *(const u32x2*)(a.v + (from + p) * a.v_stride + (int64_t)hk * D + dim);
        } else {
          const uint16_t* tv = a.old_v + tail + dim * 64 + key;
          x[n][j] = u32x2{tv[0] | (uint32_t)tv[64] << 16, tv[128] | (uint32_t)tv[192] << 16};
        }
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NK; ++n) {
    const int unit = wave + P::kWaves * n, sub = unit & 3, kp = unit >> 2;
    if (unit < P::kUnits) {
      sm.k[(sub * (D / 32) + 2 * kp) * 64 + lane] = lo[n];
      sm.k[(sub * (D / 32) + 2 * kp + 1) * 64 + lane] = hi[n];
    }
  }
#pragma unroll
  for (int n = 0; n < NVR; ++n) {
    const int it = wave * 64 + lane + P::kThreads * n, kq = it / (D / 4), dim = it % (D / 4) * 4;
    uint32_t nan4 = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w0 = x[n][j][0] & 0x7f807f80u, w1 = x[n][j][1] & 0x7f807f80u;
      if ((w0 & 0xffffu) == 0x7f80u || w0 >> 16 == 0x7f80u || (w1 & 0xffffu) == 0x7f80u || w1 >> 16 == 0x7f80u) nan4 |= 1u << j;
    }
    if (__any(nan4 != 0)) {
      uint64_t m = kq < 16 ? (uint64_t)nan4 << (4 * kq) : 0;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) m |= (uint64_t)__shfl_xor((long long)m, o);
      bad |= m;
    }
    if (kq < 16) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // dim + e of the four keys
        const uint32_t w0 = x[n][0][e >> 1], w1 = x[n][1][e >> 1], w2 = x[n][2][e >> 1], w3 = x[n][3][e >> 1];
        const u32x2 t = e & 1 ? u32x2{w0 >> 16 | (w1 & 0xffff0000u), w2 >> 16 | (w3 & 0xffff0000u)}
                              : u32x2{(w0 & 0xffffu) | w1 << 16, (w2 & 0xffffu) | w3 << 16};
        const int dd = dim + e;
        ((u32x2*)&sm.v[v_slot(dd >> 4, (kq >> 1) & 1, (kq >> 2) * 16 + (dd & 15))])[kq & 1] = t;
      }
    }
  }
  return bad;
}

// A work-group's rows [row0, row0 + kRows) of sequence i.  SLOW: a block that is
// masked for some of them holds a V that is not finite.
template <int D, bool SLOW>
__device__ __forceinline__ void prefill_rows(const StepArgs& a, PrefillLds<D>* sm, f32x4 (*s_ot)[PrefillTile<D>::kThreads],
                                             uint64_t (*s_bad)[PrefillTile<D>::kWaves],
                                             int hk, int i, int cache_row, uint32_t row0, uint32_t rows, int c0, int ctx,
                                             int end) {
  typedef PrefillTile<D> P;
  constexpr int RT = P::kRT, KS = D / 32, DT = D / 16;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const uint32_t G = (uint32_t)a.G, last_row = min(row0 + P::kRows, rows) - 1;
  const uint32_t w0 = row0 + wave * RT * 16;
  u32x4 q[RT][KS];
  int pos[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const uint32_t row = min(w0 + t * 16 + r, rows - 1);
    const int token = (int)(row / G), head = hk * a.G + (int)(row % G);
    pos[t] = ctx + token;
    const uint16_t* qp = a.q + (int64_t)(c0 + token) * a.q_stride + (int64_t)head * D;
#pragma unroll
    for (int x = 0; x < KS; ++x) q[t][x] = *(const u32x4*)(qp + (x >> 1) * 64 + g * 16 + (x & 1) * 8);
  }
  // own blocks: of the work-group's rows and of this wave's
  const int b_lo = (ctx + (int)(row0 / G)) >> 6, b_hi = (ctx + (int)(last_row / G)) >> 6;
  const bool has = w0 <= last_row;
  const int w_lo = (ctx + (int)(min(w0, last_row) / G)) >> 6;
  const int w_hi = (ctx + (int)(min(w0 + RT * 16 - 1, last_row) / G)) >> 6;

  constexpr int OL = P::kOtLds, OR = DT - OL;
  f32x4 O[RT][DT], Ot[RT][OR];
  float m[RT], l[RT], mt[RT], lt[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    m[t] = mt[t] = kNegInf;
    l[t] = lt[t] = 0.f;
#pragma unroll
    for (int x = 0; x < DT; ++x) O[t][x] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int x = 0; x < DT; ++x) (x < OR ? Ot[t][x < OR ? x : 0] : s_ot[t * OL + x - OR][threadIdx.x]) = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // one tile from LDS; MASKED: rows see keys up to upto[t] of it
  auto tile = [&](auto masked_, int buf, const int (&upto)[RT]) {
    constexpr bool MASKED = decltype(masked_)::value;
    const PrefillLds<D>& s_ = sm[buf];
    f32x4 s[RT][4];
#pragma unroll
    for (int x = 0; x < KS; ++x)  // sub-tiles inside: neighbouring MFMAs do not wait for each other
#pragma unroll
      for (int sub = 0; sub < 4; ++sub) {
        const u32x4 kf = s_.k[(sub * KS + x) * 64 + lane];
#pragma unroll
        for (int t = 0; t < RT; ++t) s[t][sub] = mma(kf, q[t][x], x ? s[t][sub] : f32x4{0.f, 0.f, 0.f, 0.f});
      }
    u32x4 p[RT][2];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      if (MASKED) {
#pragma unroll
        for (int sub = 0; sub < 4; ++sub)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[t][sub][e] = 16 * g + 4 * sub + e <= upto[t] ? s[t][sub][e] : kNegInf;
      }
      const float mn = fmaxf(m[t], max_over_groups(max16(s[t])) * a.c), ref = ref_of(mn);
      const float alpha = exp2_(m[t] - ref);
      m[t] = mn;
      l[t] = __builtin_fmaf(l[t], alpha, probabilities(s[t], a.c, ref, p[t]));
      if (__any(alpha != 1.f)) {
#pragma unroll
        for (int x = 0; x < DT; ++x) O[t][x] *= alpha;
      }
    }
    if (!(MASKED && SLOW)) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int x = 0; x < DT; ++x) {
          const u32x4 vf = s_.v[v_slot(x, h, lane)];
#pragma unroll
          for (int t = 0; t < RT; ++t) O[t][x] = mma(vf, p[t][h], O[t][x]);
        }
    } else {
      // keys with a V that is not finite: one product for every number n of
      // them that a row may see, the first n as they are, the others zero; a row takes its own
      uint64_t bad = 0;
#pragma unroll
      for (int w = 0; w < P::kWaves; ++w) bad |= s_bad[buf][w];
      int sees[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t) sees[t] = upto[t] < 0 ? 0 : __popcll(bad & (~0ull >> (63 - upto[t])));
#pragma unroll
      for (int x = 0; x < DT; ++x) {
        f32x4 base[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) base[t] = O[t][x];
        uint64_t drop = bad;
#pragma unroll 1
        for (int n = 0; n <= __popcll(bad); ++n, drop &= drop - 1) {
          const u32x4 v0 = drop_keys(s_.v[v_slot(x, 0, lane)], drop, g, 0);
          const u32x4 v1 = drop_keys(s_.v[v_slot(x, 1, lane)], drop, g, 1);
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            const f32x4 y_ = mma(v1, p[t][1], mma(v0, p[t][0], base[t]));
#pragma unroll
            for (int e = 0; e < 4; ++e) O[t][x][e] = sees[t] == n ? y_[e] : O[t][x][e];
          }
        }
      }
    }
  };
  // the end of a partition; rows whose own block is in it go on (MASKED)
  auto fold = [&](auto masked_, int b) {
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      if (decltype(masked_)::value && b >= pos[t] >> 6) continue;
      float wa, wb;
      fold_weights(mt[t], m[t], wa, wb);
      lt[t] = __builtin_fmaf(l[t], wb, lt[t] * wa);
      m[t] = kNegInf;
      l[t] = 0.f;
#pragma unroll
      for (int x = 0; x < DT; ++x) {
        f32x4& to = x < OR ? Ot[t][x < OR ? x : 0] : s_ot[t * OL + x - OR][threadIdx.x];
        f32x4 y_ = to;
#pragma unroll
        for (int e = 0; e < 4; ++e) y_[e] = __builtin_fmaf(O[t][x][e], wb, y_[e] * wa);
        to = y_;
        O[t][x] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
    }
  };

  // the 8-bit blocks that every row sees
  Bytes<D> y;
  BlockRun run;
  auto fetch = [&](int b) {
    if ((b & 63) == 0) run = load_run(a, cache_row, hk, b, lane);
    load_block<D>(a, run, hk, b, y, wave, lane);
  };
  int upto[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) upto[t] = 63;
  if (b_hi > 0) {
    fetch(0);
    store_block<D>(y, sm[0], wave, lane);
    if (SLOW && b_lo == 0) {
      const uint64_t bad = bad_in_block<D>(y, wave);
      if (lane == 0) s_bad[0][wave] = bad;
    }
    if (b_hi > 1) fetch(1);
  }
  __syncthreads();
#pragma unroll 1
  for (int b = 0; b < b_lo; ++b) {
    if (b + 1 < b_hi) {
      store_block<D>(y, sm[(b + 1) & 1], wave, lane);
      if (SLOW && b + 1 == b_lo) {
        const uint64_t bad = bad_in_block<D>(y, wave);
        if (lane == 0) s_bad[(b + 1) & 1][wave] = bad;
      }
    }
    if (b + 2 < b_hi) fetch(b + 2);
    if (has) tile(std::false_type{}, b & 1, upto);
    if ((b + 1) % kPartBlocks == 0) fold(std::false_type{}, b);
    __syncthreads();
  }
  // those that only later rows see
#pragma unroll 1
  for (int b = b_lo; b < b_hi; ++b) {
    if (b + 1 < b_hi) {
      store_block<D>(y, sm[(b + 1) & 1], wave, lane);
      if (SLOW) {
        const uint64_t bad = bad_in_block<D>(y, wave);
        if (lane == 0) s_bad[(b + 1) & 1][wave] = bad;
      }
    }
    if (b + 2 < b_hi) fetch(b + 2);
    if (has && b < w_hi) {
#pragma unroll
      for (int t = 0; t < RT; ++t) upto[t] = b < pos[t] >> 6 ? 63 : -1;
      tile(std::true_type{}, b & 1, upto);
    }
    if ((b + 1) % kPartBlocks == 0) fold(std::true_type{}, b);
    __syncthreads();
  }
  // the own blocks
#pragma unroll 1
  for (int b0 = b_lo; b0 <= b_hi; b0 += P::kRaw) {
    if (b0 > b_lo) __syncthreads();
#pragma unroll 1
    for (int n = 0; n < P::kRaw && b0 + n <= b_hi; ++n) {
      const uint64_t bad = stage_raw<D>(a, i, hk, ctx, end, c0, b0 + n, sm[n], wave, lane);
      if (SLOW && lane == 0) s_bad[n][wave] = bad;
    }
    __syncthreads();
#pragma unroll 1
    for (int n = 0; has && n < P::kRaw; ++n) {
      const int b = b0 + n;
      if (b < w_lo || b > w_hi) continue;
#pragma unroll
      for (int t = 0; t < RT; ++t) upto[t] = pos[t] >> 6 == b ? pos[t] & 63 : -1;
      tile(std::true_type{}, n, upto);
    }
  }
  fold(std::false_type{}, 0);
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const float inv = 1.f / sum_over_groups(lt[t]);
    const uint32_t row = w0 + t * 16 + r;
    if (row >= rows) continue;
    uint16_t* o = a.o + ((int64_t)(c0 + (int)(row / G)) * a.H + hk * a.G + (int)(row % G)) * D + g * 4;
#pragma unroll
    for (int x = 0; x < DT; ++x) {
      const f32x4 y_ = x < OR ? Ot[t][x < OR ? x : 0] : s_ot[t * OL + x - OR][threadIdx.x];
      *(u32x2*)(o + x * 16) = u32x2{pack2(y_[0] * inv, y_[1] * inv), pack2(y_[2] * inv, y_[3] * inv)};
    }
  }
}

template <int D>
__global__ __launch_bounds__(PrefillTile<D>::kThreads) void k_attn_prefill(const StepArgs a) {
  typedef PrefillTile<D> P;
  __shared__ PrefillLds<D> sm[P::kRaw];
  __shared__ f32x4 s_ot[P::kOtLds ? P::kRT * P::kOtLds : 1][P::kThreads];
  __shared__ uint64_t s_bad[P::kRaw][P::kWaves];
  // neighbouring work-groups take different heads: with 2, 4, 8 .. heads each
  // chiplet, and its L2, sees the keys of some of them only
  const int hk = blockIdx.x % a.Hk;
  // which sequence and rows: sequence i has the row-tile slots floor(cu[i] G / kRows) + i ..
  const int item = (int)((gridDim.x - 1 - blockIdx.x) / a.Hk);  // later rows, which see more keys, first
  int lo = 0, hi = a.N - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((int)((int64_t)a.cu[mid] * a.G / P::kRows) + mid <= item)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int i = lo, c0 = a.cu[i], len = a.cu[i + 1] - c0;
  const int64_t row0 = (int64_t)(item - ((int)((int64_t)c0 * a.G / P::kRows) + i)) * P::kRows;
  const int64_t rows = (int64_t)len * a.G;
  if (row0 >= rows) return;
  const int ctx = a.ctx_len[i], cache_row = row_of(a.slot, i, a.cache.num_slots);
  if (ctx < 0 || cache_row < 0) {  // refused: o = 0
    const int n = (int)min(rows - row0, (int64_t)P::kRows);
    for (int x = threadIdx.x; x < n * (D / 8); x += P::kThreads) {
      const uint32_t row = (uint32_t)row0 + x / (D / 8);
      u32x4* o = (u32x4*)(a.o + ((int64_t)(c0 + (int)(row / a.G)) * a.H + hk * a.G + (int)(row % a.G)) * D);
      o[x % (D / 8)] = u32x4{0, 0, 0, 0};
    }
    return;
  }
  // does one of the rows' own blocks hold a V that is not finite?
  const int b_lo = (ctx + (int)((uint32_t)row0 / (uint32_t)a.G)) >> 6;
  const int b_hi = (ctx + (int)((uint32_t)(min(row0 + P::kRows, rows) - 1) / (uint32_t)a.G)) >> 6;
  int bad = 0;
  for (int b = b_lo; b <= b_hi; ++b) bad |= a.bad[(int64_t)((c0 >> 6) + 2 * i + b - (ctx >> 6)) * a.Hk + hk];
  if (bad == 0)
    prefill_rows<D, false>(a, sm, s_ot, s_bad, hk, i, cache_row, (uint32_t)row0, (uint32_t)rows, c0, ctx, ctx + len);
  else
    prefill_rows<D, true>(a, sm, s_ot, s_bad, hk, i, cache_row, (uint32_t)row0, (uint32_t)rows, c0, ctx, ctx + len);
}

// ---------------------------------------------------------------------------
// decode

// Records that join work-groups' shares of a row: per flat partition index
// and key/value head, O [rows][D] and per row m and the four partial l.
struct DecodeArgs {
  StepArgs s;
  float* rec_o;
  float* rec_ml;  // [..][rows][8]: m, l of the four lane groups
  int32_t *base, *total;  // first flat partition of every sequence; how many there are
  int max_parts;          // records that fit
};

__device__ __forceinline__ int parts_of(int ctx) { return ctx < 0 ? 0 : ctx / kPart + 1; }

// All partitions of the batch in a row, sequence by sequence, are dealt out
// in equal runs to the W work-groups of a key/value head (blockIdx.x of
// gridDim.x): a batch of any lengths is balanced to one partition.  A run
// that begins a sequence folds its partitions as it goes; one that begins
// inside a sequence must leave each partition by itself, because the fold goes
// left to right.  If the batch has more partitions than there is room for
// records (sequences that share blocks), sequences are dealt out whole.
//
// In a work-group the four waves share a partition, four tiles at a time: wave
// w computes the scores and p of tile w; p goes through LDS and every wave
// adds all four tiles to its own quarter of the dims.  So a partition's
// bytes are spread over four waves' loads, and no byte is loaded twice.
template <int D>
__global__ __launch_bounds__(256) void k_attn_decode(const DecodeArgs da) {
  const StepArgs& a = da.s;
  constexpr int KS = D / 32, KP = D / 64, DT = D / 64;  // DT: dim tiles of a wave
  __shared__ u32x4 s_p[4][2][64];
  __shared__ float s_max[4][16], s_sum[4][64];
  __shared__ int s_scan[4], s_at[3];
  __shared__ uint32_t s_red[4];
  const int hk = blockIdx.y, tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int W = gridDim.x, head0 = blockIdx.z * 16;  // of this key/value head's group

  // the run [g0, g1) of flat partitions, and the sequence it begins in
  const int per = (a.N + 255) / 256, n0 = min(tid * per, a.N), n1 = min(n0 + per, a.N);
  int mine = 0;
  for (int n = n0; n < n1; ++n) mine += parts_of(a.ctx_len[n]);
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 63) s_scan[wave] = upto;
  __syncthreads();
  const int total = s_scan[0] + s_scan[1] + s_scan[2] + s_scan[3];
  for (int w = 0; w < wave; ++w) upto += s_scan[w];
  const bool whole_seqs = total > da.max_parts;
  const int g0 = (int)((int64_t)blockIdx.x * total / W), g1 = (int)((int64_t)(blockIdx.x + 1) * total / W);
  if (blockIdx.x == 0 && hk == 0 && blockIdx.z == 0 && tid == 0) *da.total = total;
  if (g0 >= g1 && !whole_seqs) return;
  if (g0 >= upto - mine && g0 < upto) {
    int at = upto - mine, n = n0;
    for (; n < n1 - 1; ++n) {
      const int x = parts_of(a.ctx_len[n]);
      if (g0 < at + x) break;
      at += x;
    }
    s_at[0] = n;
    s_at[1] = at;
  }
  __syncthreads();
  int i = whole_seqs ? blockIdx.x : s_at[0], base = whole_seqs ? 0 : s_at[1];

  for (int f = g0; whole_seqs ? i < a.N : f < g1;) {
    const int ctx = a.ctx_len[i], np = parts_of(ctx);
    if (np == 0) {
      i += whole_seqs ? W : 1;
      continue;
    }
    const int own = ctx >> 6;  // the block of the new token
    const int p_lo = whole_seqs ? 0 : f - base, p_hi = whole_seqs ? np : min(np, g1 - base);
    const int cache_row = max(row_of(a.slot, i, a.cache.num_slots), 0);
    if (p_lo == 0 && hk == 0 && blockIdx.z == 0 && tid == 0) da.base[i] = base;
    const int head = head0 + r;
    const bool live = head < a.G;
    u32x4 q[KS];
    {
      const uint16_t* qp = a.q + (int64_t)i * a.q_stride + (int64_t)(hk * a.G + (live ? head : a.G - 1)) * D;
#pragma unroll
      for (int x = 0; x < KS; ++x) q[x] = *(const u32x4*)(qp + (x >> 1) * 64 + g * 16 + (x & 1) * 8);
    }
    f32x4 Ot[DT];
    float mt = kNegInf, lt = 0.f;
#pragma unroll
    for (int x = 0; x < DT; ++x) Ot[x] = f32x4{0.f, 0.f, 0.f, 0.f};

    for (int p = p_lo; p < p_hi; ++p) {
      f32x4 O[DT];
      float m = kNegInf, l = 0.f;
#pragma unroll
      for (int x = 0; x < DT; ++x) O[x] = f32x4{0.f, 0.f, 0.f, 0.f};
      const int b_end = min((p + 1) * kPartBlocks, own);
#pragma unroll 1
      for (int b0 = p * kPartBlocks; b0 < b_end; b0 += 4) {
        const bool mytile = b0 + wave < b_end;
        // V of all four tiles for this wave's dims; K of its own tile
        u32x4 kb[4][KP], vb[4][DT];
        float ks = 1.f, vs[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int64_t at = (int64_t)pool_block(a, cache_row, min(b0 + t, b_end - 1)) * a.Hk + hk;
          vs[t] = a.cache.v_scale[at];
          const uint8_t* vp = a.cache.v8 + at * (64 * D) + (wave * DT * 16 + r) * 64 + g * 16;
#pragma unroll
          for (int x = 0; x < DT; ++x) vb[t][x] = *(const u32x4*)(vp + x * 1024);
        }
        {
          const int64_t at = (int64_t)pool_block(a, cache_row, min(b0 + wave, b_end - 1)) * a.Hk + hk;
          ks = a.cache.k_scale[at];
          const uint8_t* kp_ = a.cache.k8 + at * (64 * D) + g * 16;
#pragma unroll
          for (int sub = 0; sub < 4; ++sub)
#pragma unroll
            for (int x = 0; x < KP; ++x) kb[sub][x] = *(const u32x4*)(kp_ + x * 4096 + key_of(sub, r) * 64);
        }
        f32x4 s[4];
#pragma unroll
        for (int sub = 0; sub < 4; ++sub) {
          s[sub] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int x = 0; x < KP; ++x) {
            u32x4 k0, k1;
            from_e4m3(kb[sub][x], ks, k0, k1);
            s[sub] = mma(k0, q[2 * x], s[sub]);
            s[sub] = mma(k1, q[2 * x + 1], s[sub]);
          }
        }
        const float smax = max_over_groups(max16(s));
        if (g == 0) s_max[wave][r] = smax;
        __syncthreads();
        float mm[5];  // the running max before and after every tile
        mm[0] = m;
#pragma unroll
        for (int t = 0; t < 4; ++t) mm[t + 1] = b0 + t < b_end ? fmaxf(mm[t], s_max[t][r] * a.c) : mm[t];
        if (mytile) {
          u32x4 pf[2];
          const float mine_ = wave == 0 ? mm[1] : wave == 1 ? mm[2] : wave == 2 ? mm[3] : mm[4];
          s_sum[wave][lane] = probabilities(s, a.c, ref_of(mine_), pf);
          s_p[wave][0][lane] = pf[0];
          s_p[wave][1][lane] = pf[1];
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          if (b0 + t >= b_end) break;
          const float alpha = exp2_(mm[t] - ref_of(mm[t + 1]));
          l = __builtin_fmaf(l, alpha, s_sum[t][lane]);
          const u32x4 p0 = s_p[t][0][lane], p1 = s_p[t][1][lane];
#pragma unroll
          for (int x = 0; x < DT; ++x) {
            u32x4 v0, v1;
            from_e4m3(vb[t][x], vs[t], v0, v1);
            O[x] *= alpha;
            O[x] = mma(v0, p0, O[x]);
            O[x] = mma(v1, p1, O[x]);
          }
        }
        m = mm[4];
      }
      if (p == np - 1) {
        // the own block, in the input type: the tail, and the new token in
        // its place; every wave computes all of its scores
        const int at = ctx & 63;
        const uint16_t* tk = a.cache.tail_k + ((int64_t)cache_row * a.Hk + hk) * (64 * D);
        const uint16_t* tv = a.cache.tail_v + ((int64_t)cache_row * a.Hk + hk) * (64 * D);
        const uint16_t* nk = a.k + (int64_t)i * a.k_stride + (int64_t)hk * D;
        const uint16_t* nv = a.v + (int64_t)i * a.v_stride + (int64_t)hk * D;
        u32x4 vb[DT][2];
        uint32_t nvx[DT];
#pragma unroll
        for (int x = 0; x < DT; ++x) {
          const int dim = (wave * DT + x) * 16 + r;
          vb[x][0] = *(const u32x4*)(tv + dim * 64 + g * 16);
          vb[x][1] = *(const u32x4*)(tv + dim * 64 + g * 16 + 8);
          nvx[x] = nv[dim];
        }
        f32x4 s[4];
#pragma unroll
        for (int sub = 0; sub < 4; ++sub) {
          const int key = key_of(sub, r);
          const uint16_t* kr = (key == at ? nk : tk + key * D) + g * 16;
          s[sub] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int x = 0; x < KS; ++x) s[sub] = mma(*(const u32x4*)(kr + (x >> 1) * 64 + (x & 1) * 8), q[x], s[sub]);
#pragma unroll
          for (int e = 0; e < 4; ++e) s[sub][e] = 16 * g + 4 * sub + e <= at ? s[sub][e] : kNegInf;
        }
        const float mn = fmaxf(m, max_over_groups(max16(s)) * a.c), ref = ref_of(mn);
        const float alpha = exp2_(m - ref);
        m = mn;
        u32x4 pf[2];
        l = __builtin_fmaf(l, alpha, probabilities(s, a.c, ref, pf));
        // V: keys past the new one are not there yet (whatever the tail
        // holds), the new one comes from the call
#pragma unroll
        for (int x = 0; x < DT; ++x) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int key = 16 * g + 2 * j;
            uint32_t w = vb[x][j >> 2][j & 3];
            w = key > at ? 0u : key + 1 > at ? w & 0xffffu : w;
            w = key == at ? nvx[x] : key + 1 == at ? (w & 0xffffu) | nvx[x] << 16 : w;
            vb[x][j >> 2][j & 3] = w;
          }
          O[x] *= alpha;
          O[x] = mma(vb[x][0], pf[0], O[x]);
          O[x] = mma(vb[x][1], pf[1], O[x]);
        }
        if (blockIdx.z == 0) {
          // append: the tail's row and column; a full block is quantised
          __syncthreads();  // every wave has read the tail
          uint16_t* wk = (uint16_t*)tk;
          uint16_t* wv = (uint16_t*)tv;
          if (tid < D / 8) *(u32x4*)(wk + at * D + tid * 8) = *(const u32x4*)(nk + tid * 8);
          for (int x = tid; x < D; x += 256) wv[x * 64 + at] = nv[x];
          if (at == 63) {
            __threadfence_block();
            __syncthreads();
            quantise_block<D>(
                a.cache, (int64_t)pool_block(a, cache_row, own) * a.Hk + hk,
                [&](int x) { return ((const u32x4*)wk)[x]; }, [&](int x) { return ((const u32x4*)wv)[x]; }, s_red);
          }
        }
      }
      if (p_lo == 0) {
        float wa, wb;
        fold_weights(mt, m, wa, wb);
        lt = __builtin_fmaf(l, wb, lt * wa);
#pragma unroll
        for (int x = 0; x < DT; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) Ot[x][e] = __builtin_fmaf(O[x][e], wb, Ot[x][e] * wa);
      }
      const bool whole = p_lo == 0 && p == np - 1;
      if (whole) {
        const float inv = 1.f / sum_over_groups(lt);
        if (live) {
          uint16_t* o = a.o + ((int64_t)i * a.H + hk * a.G + head) * D + wave * DT * 16 + g * 4;
#pragma unroll
          for (int x = 0; x < DT; ++x)
            *(u32x2*)(o + x * 16) = u32x2{pack2(Ot[x][0] * inv, Ot[x][1] * inv), pack2(Ot[x][2] * inv, Ot[x][3] * inv)};
        }
      } else if (p_lo > 0 || p == p_hi - 1) {
        const int64_t rec = ((int64_t)(base + (p_lo > 0 ? p : 0)) * a.Hk + hk) * a.G + head;
        if (live) {
          float* o = da.rec_o + rec * D + wave * DT * 16 + g * 4;
#pragma unroll
          for (int x = 0; x < DT; ++x) *(f32x4*)(o + x * 16) = p_lo > 0 ? O[x] : Ot[x];
          if (wave == 0) {
            if (g == 0) da.rec_ml[rec * 8] = p_lo > 0 ? m : mt;
            da.rec_ml[rec * 8 + 4 + g] = p_lo > 0 ? l : lt;
          }
        }
      }
    }
    if (whole_seqs) {
      i += W;
    } else {
      f = base + p_hi;
      base += np;
      ++i;
    }
  }
}

// Joins what several work-groups did of a sequence, left to right; sequences
// that one work-group did alone are finished, refused ones get o = 0.
template <int D>
__global__ __launch_bounds__(256) void k_attn_join(const DecodeArgs da, int W) {
  const StepArgs& a = da.s;
  const int i = blockIdx.x, hk = blockIdx.y;
  const int np = parts_of(a.ctx_len[i]);
  uint16_t* o = a.o + ((int64_t)i * a.H + hk * a.G) * D;
  if (np == 0) {
    for (int x = threadIdx.x; x < a.G * D / 4; x += 256) *(u32x2*)(o + x * 4) = u32x2{0, 0};
    return;
  }
  const int base = da.base[i], total = *da.total;
  if (total > da.max_parts) return;
  // the work-group of the sequence's first partition, and where its run ends
  const int w = (int)((((int64_t)base + 1) * W - 1) / total);
  const int cut = (int)((int64_t)(w + 1) * total / W);
  if (cut >= base + np) return;
  const int n = base + np - cut;  // records after the first
  for (int x = blockIdx.z * 256 + threadIdx.x; x < a.G * D / 4; x += 256 * gridDim.z) {
    const int head = x / (D / 4), dim = x % (D / 4) * 4;
    const int64_t row = (int64_t)hk * a.G + head, step = (int64_t)a.Hk * a.G;
    const float* ml = da.rec_ml + ((int64_t)base * step + row) * 8;
    f32x4 O = *(const f32x4*)(da.rec_o + ((int64_t)base * step + row) * D + dim);
    float m = ml[0];
    f32x4 l = *(const f32x4*)(ml + 4);
    const float* po = da.rec_o + ((int64_t)cut * step + row) * D + dim;
    const float* pm = da.rec_ml + ((int64_t)cut * step + row) * 8;
#pragma unroll 8
    for (int j = 0; j < n; ++j) {
      const f32x4 Op = *(const f32x4*)(po + (int64_t)j * step * D);
      const float mp = pm[(int64_t)j * step * 8];
      const f32x4 lp = *(const f32x4*)(pm + (int64_t)j * step * 8 + 4);
      float wa, wb;
      fold_weights(m, mp, wa, wb);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        l[e] = __builtin_fmaf(lp[e], wb, l[e] * wa);
        O[e] = __builtin_fmaf(Op[e], wb, O[e] * wa);
      }
    }
    const float inv = 1.f / ((l[0] + l[1]) + (l[2] + l[3]));
    *(u32x2*)(o + head * D + dim) = u32x2{pack2(O[0] * inv, O[1] * inv), pack2(O[2] * inv, O[3] * inv)};
  }
}

}  // namespace attn
