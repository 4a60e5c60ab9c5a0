// Causal attention over the 8-bit cache: prefill (any number of new tokens
// per sequence) and the decode step.
//
// Arithmetic, the same in every kernel, per query row and in this order:
//   keys in partitions of 512; in a partition the 8-bit blocks before the
//   row's own in ascending order, then, in the last one, the own block's
//   tokens up to the row in the input type.  A block of 64 keys is one tile:
//     s    = K q, v_mfma_f32_16x16x32_bf16, k steps ascending (dims 64 kp +
//            16 g + 8 h .. + 7 in slot group g of step 2 kp + h)
//     m'   = c max(s) if that is more than m + 8, m if not; c = scale * log2(e)
//     p    = exp2(fma(s, c, -m')), alpha = exp2(m - m')
//     O    = alpha O + V^T p, p in bf16, two MFMA k steps
//     l    = the same with V = 1, so numerator and denominator have the same p
//   partitions: (m, l, O) = fold of the total and the partition, left to
//   right: O = fma(Op, exp2(mp - m'), O exp2(m - m')).
//   o = O (1 / l).
// p is rounded to bf16 because the second product takes bf16 operands; that is the
// largest error of o beside its own rounding (5 x 2,048: 0.0020 of its size against 64
// bits, where 32 bits throughout and one rounding at the end give 0.0016).
// m is a reference for the exponents, not the maximum itself: it moves, and O
// and l are scaled, only when p would pass 2^8, which bf16 and the 32-bit sums hold
// as exactly as 1.  Of random scores a partition's first tile sets it for the rest,
// where a true running maximum moves for some row of 16 in nearly every tile
// (prefill, 5 x 2,048 at d = 128: 172 us a call, with the maximum 179; 1 x 10,240 at
// d = 256: 1,109 and 1,167).
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

// Waits here for a load whose first use would otherwise be inside a loop: the
// wait counts loads, so in the loop it would also wait for every load that
// the loop itself keeps in flight.
__device__ __forceinline__ void settle(u32x4& x) { asm volatile("" : "+v"(x)); }

// key of a sub-tile's A row x
__device__ __forceinline__ int key_of(int a, int x) { return 16 * (x >> 2) + 4 * a + (x & 3); }

// For inline assembly that reads MFMA results: the hardware does not wait for
// them, the compiler puts the wait states (11 at most for these shapes) before
// its own instructions only.  Nothing is moved over the barriers.
__device__ __forceinline__ void mfma_done() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 15\ns_nop 3");
  __builtin_amdgcn_sched_barrier(0);
}

// max of a lane's 16 scores, after mfma_done().  v_max3_f32 by name: of fmaxf
// the compiler makes one more instruction per score, to quiet NaNs that
// v_max3_f32 passes over by itself.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float m;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(m) : "v"(a), "v"(b), "v"(c));
  return m;
}

__device__ __forceinline__ float max16(const f32x4 (&s)[4]) {
  const float a = max3(s[0][0], s[0][1], s[0][2]), b = max3(s[0][3], s[1][0], s[1][1]), c = max3(s[1][2], s[1][3], s[2][0]);
  const float d = max3(s[2][1], s[2][2], s[2][3]), e = max3(s[3][0], s[3][1], s[3][2]);
  return max3(max3(a, b, c), max3(d, e, s[3][3]), s[3][3]);
}

// scores -> p: their bf16 B fragments for the two PV steps
__device__ __forceinline__ void probabilities(const f32x4 (&s)[4], float c, float m, u32x4 (&p)[2]) {
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    float e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = exp2_(__builtin_fmaf(s[a][i], c, -m));
    p[a >> 1][2 * (a & 1)] = pack2(e[0], e[1]);
    p[a >> 1][2 * (a & 1) + 1] = pack2(e[2], e[3]);
  }
}

// l += sum p, as one more dim whose V is 1: every lane of a row gets the sum
// over all 64 keys (in element 0; the others are not kept up).
__device__ __forceinline__ void add_sum(const u32x4 (&p)[2], f32x4& l) {
  const u32x4 ones = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
  l = mma(ones, p[1], mma(ones, p[0], l));
}

// the reference after a tile whose scores have the maximum x / c
__device__ __forceinline__ float move_ref(float m, float x) { return x > m + 8.f ? x : m; }

// as an exponent's reference (a row that has seen nothing: 0)
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
// walks the keys together through tiles in LDS, in the order the MFMA operands
// are read (conflict-free, 16 bytes per lane), while the bytes of the next one
// are in flight from memory.  The accumulators' registers allow two waves on a
// SIMD.  Of a long prompt what bounds it is their issue of instructions, one a SIMD in
// 6 to 7 cycles at d = 256 with the MFMAs busy a third of the time; of 2,048
// tokens at d = 128 it is one in 11, MFMAs busy for a quarter, and the start, the masked
// tiles and the own blocks count for as much.  So a tile is converted to bf16 once per work-group,
// before it is written to LDS, at d = 64 and 128 (5 x 2,048 at d = 128: 172 us a call;
// with 8-bit tiles, which every wave converts as it reads, 185).  At d = 256 the 8-bit
// tiles leave LDS for more of the folded total, which otherwise goes to scratch memory in
// the loop (1 x 10,240: 1,109 us a call; bf16 tiles 1,616).
//
// The 8-bit blocks come first, all in one loop (those from the work-group's
// first own block on are masked per row), then the rows' own blocks.
//
// Measured: 5 x 2,048, 16 heads, d = 128: 145 us, 85.9 GFLOP, 590 TFLOP/s; 1 x 10,240, 16 heads over 2,
// d = 256: 1,076 us, 859 GFLOP, 800 TFLOP/s; a library product of two 8,192 x 8,192
// matrices reaches 1,210.  Two more tries at the issue of instructions changed nothing: half of the
// waves half a tile behind the others, and half of the exponentials between the MFMAs.
template <int D>
struct PrefillTile {
  static constexpr int kRT = D == 256 ? 1 : 2;   // 16-row tiles of a wave: as the accumulators' registers allow
  static constexpr int kWaves = 8;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kRows = 16 * kRT * kWaves;
  static constexpr int kUnits = 4 * (D / 64);    // 1 KiB loads of an 8-bit block, K; as many for V
  static constexpr bool kSplit = kUnits < kWaves;  // d = 64: half of the waves load K, half V
  static constexpr int kPer = kSplit ? 1 : kUnits / kWaves;  // units of a wave, K and V each
  static constexpr bool kLds8 = D == 256;          // tiles in LDS: 8 bits, or bf16
  // dim tiles of the folded total that are kept in LDS (each thread its own), for want of registers
  static constexpr int kOtLds = D == 64 ? 0 : D == 128 ? 5 : 8;
};

template <int D>
struct PrefillLds {
  static constexpr int kPart = PrefillTile<D>::kUnits * (PrefillTile<D>::kLds8 ? 1 : 2) * 64;
  u32x4 x[2 * kPart];  // K and V of a tile in 1 KiB units or bf16 fragments
  __device__ u32x4* k() { return x; }
  __device__ u32x4* v() { return x + kPart; }
};

// Of the two tiles' LDS, where V of an own block lies (bf16): slots of them fit.
template <int D>
constexpr int kRawSlots = PrefillTile<D>::kLds8 ? 2 : 4;

template <int D>
__device__ __forceinline__ u32x4* raw_slot(PrefillLds<D>* sm, int n) { return (u32x4*)sm + n * (D / 16 * 2 * 64); }

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
  asm volatile("" : "+v"(x.ks), "+v"(x.vs));  // as settle()
  return x;
}

__device__ __forceinline__ float lane_of(float x, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), lane));
}

template <int D>
struct Bytes {  // a wave's share of an 8-bit block in flight
  u32x4 k[PrefillTile<D>::kPer], v[PrefillTile<D>::kPer];
};

template <int D>
__device__ __forceinline__ void load_k8(const StepArgs& a, const BlockRun& run, int hk, int b, Bytes<D>& y, int wave, int lane) {
  typedef PrefillTile<D> P;
  if (P::kSplit && wave >= P::kUnits) return;
  const int r = lane & 15, g = lane >> 4;
  const int64_t at = (int64_t)__builtin_amdgcn_readlane(run.id, b & 63) * a.Hk + hk;
#pragma unroll
  for (int n = 0; n < P::kPer; ++n) {
    const int unit = (wave + P::kWaves * n) % P::kUnits;
    y.k[n] = *(const u32x4*)(a.cache.k8 + at * (64 * D) + (unit >> 2) * 4096 + key_of(unit & 3, r) * 64 + g * 16);
  }
}

template <int D>
__device__ __forceinline__ void load_v8(const StepArgs& a, const BlockRun& run, int hk, int b, Bytes<D>& y, int wave, int lane) {
  typedef PrefillTile<D> P;
  if (P::kSplit && wave < P::kUnits) return;
  const int r = lane & 15, g = lane >> 4;
  const int64_t at = (int64_t)__builtin_amdgcn_readlane(run.id, b & 63) * a.Hk + hk;
#pragma unroll
  for (int n = 0; n < P::kPer; ++n) {
    const int unit = (wave + P::kWaves * n) % P::kUnits;
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
__device__ __forceinline__ void put_k8(const Bytes<D>& y, float scale, PrefillLds<D>& sm, int wave, int lane) {
  typedef PrefillTile<D> P;
  if (P::kSplit && wave >= P::kUnits) return;
#pragma unroll
  for (int n = 0; n < P::kPer; ++n) {
    const int unit = (wave + P::kWaves * n) % P::kUnits, sub = unit & 3, kp = unit >> 2;
    if constexpr (P::kLds8) {
      sm.k()[unit * 64 + lane] = y.k[n];
    } else {
      u32x4 lo, hi;
      from_e4m3(y.k[n], scale, lo, hi);
      sm.k()[(sub * (D / 32) + 2 * kp) * 64 + lane] = lo;
      sm.k()[(sub * (D / 32) + 2 * kp + 1) * 64 + lane] = hi;
    }
  }
}

template <int D>
__device__ __forceinline__ void put_v8(const Bytes<D>& y, float scale, PrefillLds<D>& sm, int wave, int lane) {
  typedef PrefillTile<D> P;
  if (P::kSplit && wave < P::kUnits) return;
#pragma unroll
  for (int n = 0; n < P::kPer; ++n) {
    const int unit = (wave + P::kWaves * n) % P::kUnits;
    if constexpr (P::kLds8) {
      sm.v()[unit * 64 + lane] = y.v[n];
    } else {
      u32x4 lo, hi;
      from_e4m3(y.v[n], scale, lo, hi);
      sm.v()[v_slot(unit, 0, lane)] = lo;
      sm.v()[v_slot(unit, 1, lane)] = hi;
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

// V of the own blocks b and b + 1, in the input type, into slots n and n + 1:
// the call's tokens, and the tail as it was for the ones before.  From token
// `end` on: zeros.  A thread takes four keys of four dims and writes them turned.
// s_bad gets the wave's keys with a V that is not finite.
template <int D, bool SLOW>
__device__ __forceinline__ void stage_raw(const StepArgs& a, int i, int hk, int ctx, int end, int c0, int b, PrefillLds<D>* sm,
                                          int n, uint64_t (*s_bad)[PrefillTile<D>::kWaves], int wave, int lane) {
  typedef PrefillTile<D> P;
  constexpr int NV = (16 * (D / 4) + P::kThreads - 1) / P::kThreads;
  const int64_t tail = ((int64_t)i * a.Hk + hk) * (64 * D);
  const int64_t from = (int64_t)c0 - ctx;
  u32x2 x[2][NV][4];
#pragma unroll
  for (int z = 0; z < 2; ++z)
#pragma unroll
    for (int m = 0; m < NV; ++m) {
      const int it = wave * 64 + lane + P::kThreads * m, kq = it / (D / 4), dim = it % (D / 4) * 4;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = 4 * kq + j, p = (b + z) * 64 + key;
        x[z][m][j] = u32x2{0, 0};
        if (kq < 16 && p < end) {
          if (p >= ctx) {
            x[z][m][j] = *(const u32x2*)(a.v + (from + p) * a.v_stride + (int64_t)hk * D + dim);
          } else {
            const uint16_t* tv = a.old_v + tail + dim * 64 + key;
            x[z][m][j] = u32x2{tv[0] | (uint32_t)tv[64] << 16, tv[128] | (uint32_t)tv[192] << 16};
          }
        }
      }
    }
#pragma unroll
  for (int z = 0; z < 2; ++z) {
    uint64_t bad = 0;
#pragma unroll
    for (int m = 0; m < NV; ++m) {
      const int it = wave * 64 + lane + P::kThreads * m, kq = it / (D / 4), dim = it % (D / 4) * 4;
      if (SLOW) {
        uint32_t nan4 = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t w0 = x[z][m][j][0] & 0x7f807f80u, w1 = x[z][m][j][1] & 0x7f807f80u;
          if ((w0 & 0xffffu) == 0x7f80u || w0 >> 16 == 0x7f80u || (w1 & 0xffffu) == 0x7f80u || w1 >> 16 == 0x7f80u) nan4 |= 1u << j;
        }
        if (__any(nan4 != 0)) {
          uint64_t w = kq < 16 ? (uint64_t)nan4 << (4 * kq) : 0;
#pragma unroll
          for (int o = 1; o < 64; o <<= 1) w |= (uint64_t)__shfl_xor((long long)w, o);
          bad |= w;
        }
      }
      if (kq < 16) {
        u32x2 turned[4];
        transpose4(x[z][m], turned);
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // dim + e of the four keys
          const int dd = dim + e;
          ((u32x2*)&raw_slot<D>(sm, n + z)[v_slot(dd >> 4, (kq >> 1) & 1, (kq >> 2) * 16 + (dd & 15))])[kq & 1] = turned[e];
        }
      }
    }
    if (SLOW && lane == 0) s_bad[n + z][wave] = bad;
  }
}

// A work-group's rows [row0, row0 + kRows) of sequence i.  SLOW: a block that is
// masked for some of them holds a V that is not finite.
template <int D, bool SLOW>
__device__ __forceinline__ void prefill_rows(const StepArgs& a, PrefillLds<D>* sm, f32x4 (*s_ot)[PrefillTile<D>::kThreads],
                                             uint64_t (*s_bad)[PrefillTile<D>::kWaves], float (*s_scale)[2],
                                             int hk, int i, int cache_row, uint32_t row0, uint32_t rows, int c0, int ctx,
                                             int end) {
  typedef PrefillTile<D> P;
  constexpr int RT = P::kRT, KS = D / 32, DT = D / 16;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const uint32_t G = (uint32_t)a.G, last_row = min(row0 + P::kRows, rows) - 1;
  const uint32_t w0 = row0 + wave * RT * 16;
  // own blocks: of the work-group's rows
  const int b_lo = (ctx + (int)(row0 / G)) >> 6, b_hi = (ctx + (int)(last_row / G)) >> 6;

  Bytes<D> y;
  float ks = 1.f, vs = 1.f;
  BlockRun run;
  const int n_tiles = b_hi;
  auto fetch = [&](int t) __attribute__((always_inline)) {
    if ((t & 63) == 0) run = load_run(a, cache_row, hk, t, lane);
    load_k8<D>(a, run, hk, t, y, wave, lane);
    load_v8<D>(a, run, hk, t, y, wave, lane);
    ks = lane_of(run.ks, t & 63);
    vs = lane_of(run.vs, t & 63);
  };
  if (n_tiles > 0) fetch(0);

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
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int x = 0; x < KS; ++x) settle(q[t][x]);
  // own blocks of this wave's rows
  const bool has = w0 <= last_row;
  const int w_lo = (ctx + (int)(min(w0, last_row) / G)) >> 6;
  const int w_hi = (ctx + (int)(min(w0 + RT * 16 - 1, last_row) / G)) >> 6;

  constexpr int OL = P::kOtLds, OR = DT - OL;
  f32x4 O[RT][DT], Ot[RT][OR], l[RT];
  float m[RT], mt[RT], lt[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    m[t] = mt[t] = kNegInf;
    lt[t] = 0.f;
    l[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int x = 0; x < DT; ++x) O[t][x] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int x = 0; x < DT; ++x) (x < OR ? Ot[t][x < OR ? x : 0] : s_ot[t * OL + x - OR][threadIdx.x]) = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // The three parts of a tile.  LDS is read a group ahead of the MFMAs that
  // use it; the barriers keep the compiler from moving a read to its use,
  // where its latency would show.
  constexpr int PF = P::kLds8 ? 2 : 1;             // fragments of 16 bytes in LDS
  constexpr int GS = (RT == 1 ? 8 : 4) / PF;       // 16-byte reads of a group
  f32x4 s[RT][4];
  u32x4 p[RT][2];
  int upto[RT];  // the last key of the tile that a row sees
  auto scores = [&](int buf) __attribute__((always_inline)) {
    constexpr int NG = 4 * KS / PF / GS;
    const u32x4* s_ = sm[buf].k();
    const float ks = P::kLds8 ? s_scale[buf][0] : 1.f;
    u32x4 u[2][GS];
    auto read = [&](int n) __attribute__((always_inline)) {
#pragma unroll
      for (int e = 0; e < GS; ++e) {
        const int f = n * GS + e;  // sub-tiles inside: neighbouring MFMAs do not wait for each other
        u[n & 1][e] = s_[(P::kLds8 ? f : (f & 3) * KS + (f >> 2)) * 64 + lane];
      }
    };
    read(0);
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      if (n + 1 < NG) read(n + 1);
      __builtin_amdgcn_sched_barrier(0);
      u32x4 k[GS][PF];
#pragma unroll
      for (int e = 0; e < GS; ++e) {
        if constexpr (P::kLds8)
          from_e4m3(u[n & 1][e], ks, k[e][0], k[e][1]);
        else
          k[e][0] = u[n & 1][e];
      }
#pragma unroll
      for (int h = 0; h < PF; ++h)
#pragma unroll
        for (int e = 0; e < GS; ++e) {
          const int sub = (n * GS + e) & 3, x = (n * GS + e) / 4 * PF + h;
#pragma unroll
          for (int t = 0; t < RT; ++t) s[t][sub] = mma(k[e][h], q[t][x], x ? s[t][sub] : f32x4{0.f, 0.f, 0.f, 0.f});
        }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // scores of own block b: K from memory, as it is, a sub-tile ahead
  auto raw_scores = [&](int b) __attribute__((always_inline)) {
    u32x4 k[2][KS];
    auto load = [&](int sub) __attribute__((always_inline)) {
      const int key = key_of(sub, r), pk = b * 64 + key;
      const uint16_t* src = (pk >= ctx ? a.k + ((int64_t)c0 - ctx + min(pk, end - 1)) * a.k_stride + (int64_t)hk * D
                                       : a.old_k + ((int64_t)i * a.Hk + hk) * (64 * D) + key * D) + g * 16;
#pragma unroll
      for (int x = 0; x < KS; ++x) k[sub & 1][x] = *(const u32x4*)(src + (x >> 1) * 64 + (x & 1) * 8);
    };
    load(0);
#pragma unroll
    for (int sub = 0; sub < 4; ++sub) {
      if (sub < 3) load(sub + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int x = 0; x < KS; ++x)
#pragma unroll
        for (int t = 0; t < RT; ++t) s[t][sub] = mma(k[sub & 1][x], q[t][x], x ? s[t][sub] : f32x4{0.f, 0.f, 0.f, 0.f});
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto softmax = [&](bool masked) __attribute__((always_inline)) {
    mfma_done();
    if (masked) {
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const int lim = upto[t] - 16 * g;
#pragma unroll
        for (int sub = 0; sub < 4; ++sub)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[t][sub][e] = 4 * sub + e <= lim ? s[t][sub][e] : kNegInf;
      }
    }
    float alpha[RT];
    bool moved = false;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const float mn = move_ref(m[t], max_over_groups(max16(s[t])) * a.c);
      moved |= mn != m[t];
      alpha[t] = exp2_(m[t] - ref_of(mn));
      m[t] = mn;
    }
    if (__any(moved)) {
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        l[t][0] *= alpha[t];
#pragma unroll
        for (int x = 0; x < DT; ++x) O[t][x] *= alpha[t];
      }
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) probabilities(s[t], a.c, ref_of(m[t]), p[t]);
  };
  // O += V^T p of a tile with keys whose V is not finite (s_bad): one product
  // for every number n of them that a row may see, the first n as they
  // are, the others zero; a row takes its own
  auto slow_products = [&](int buf, auto&& fragments) __attribute__((always_inline)) {
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
      u32x4 f0, f1;
      fragments(x, f0, f1);
      uint64_t drop = bad;
#pragma unroll 1
      for (int n = 0; n <= __popcll(bad); ++n, drop &= drop - 1) {
        const u32x4 v0 = drop_keys(f0, drop, g, 0), v1 = drop_keys(f1, drop, g, 1);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          const f32x4 y_ = mma(v1, p[t][1], mma(v0, p[t][0], base[t]));
#pragma unroll
          for (int e = 0; e < 4; ++e) O[t][x][e] = sees[t] == n ? y_[e] : O[t][x][e];
        }
      }
    }
  };
  auto products = [&](int buf, bool masked) __attribute__((always_inline)) {
    constexpr int NG = 2 * DT / PF / GS;
    const u32x4* s_ = sm[buf].v();
    const float vs = P::kLds8 ? s_scale[buf][1] : 1.f;
#pragma unroll
    for (int t = 0; t < RT; ++t) add_sum(p[t], l[t]);
    if (SLOW && masked) {
      slow_products(buf, [&](int x, u32x4& f0, u32x4& f1) {
        if constexpr (P::kLds8) {
          from_e4m3(s_[x * 64 + lane], vs, f0, f1);
        } else {
          f0 = s_[v_slot(x, 0, lane)];
          f1 = s_[v_slot(x, 1, lane)];
        }
      });
      return;
    }
    u32x4 u[2][GS];
    auto read = [&](int n) __attribute__((always_inline)) {
#pragma unroll
      for (int e = 0; e < GS; ++e) {
        const int f = n * GS + e;
        u[n & 1][e] = s_[P::kLds8 ? f * 64 + lane : v_slot(f % DT, f / DT, lane)];
      }
    };
    read(0);
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      if (n + 1 < NG) read(n + 1);
      __builtin_amdgcn_sched_barrier(0);
      u32x4 v[GS][PF];
#pragma unroll
      for (int e = 0; e < GS; ++e) {
        if constexpr (P::kLds8)
          from_e4m3(u[n & 1][e], vs, v[e][0], v[e][1]);
        else
          v[e][0] = u[n & 1][e];
      }
#pragma unroll
      for (int h = 0; h < PF; ++h)
#pragma unroll
        for (int e = 0; e < GS; ++e) {
          const int f = n * GS + e, x = f % DT, step = P::kLds8 ? h : f / DT;
#pragma unroll
          for (int t = 0; t < RT; ++t) O[t][x] = mma(v[e][h], p[t][step], O[t][x]);
        }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto raw_products = [&](u32x4* s_, int slot) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < RT; ++t) add_sum(p[t], l[t]);
    if (SLOW) {
      slow_products(slot, [&](int x, u32x4& f0, u32x4& f1) {
        f0 = s_[v_slot(x, 0, lane)];
        f1 = s_[v_slot(x, 1, lane)];
      });
      return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int x = 0; x < DT; ++x) {
        const u32x4 vf = s_[v_slot(x, h, lane)];
#pragma unroll
        for (int t = 0; t < RT; ++t) O[t][x] = mma(vf, p[t][h], O[t][x]);
      }
  };
  // the end of a partition; rows whose own block is in it go on (MASKED)
  auto fold = [&](auto masked_, int b) {
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      if (decltype(masked_)::value && b >= pos[t] >> 6) continue;
      float wa, wb;
      fold_weights(mt[t], m[t], wa, wb);
      lt[t] = __builtin_fmaf(l[t][0], wb, lt[t] * wa);
      m[t] = kNegInf;
      l[t] = f32x4{0.f, 0.f, 0.f, 0.f};
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

  // the 8-bit blocks, a tile ahead in LDS and another on its way
  auto put = [&](int t) __attribute__((always_inline)) {
    put_k8<D>(y, ks, sm[t & 1], wave, lane);
    put_v8<D>(y, vs, sm[t & 1], wave, lane);
    if (P::kLds8 && threadIdx.x == 0) {
      s_scale[t & 1][0] = ks;
      s_scale[t & 1][1] = vs;
    }
    if (SLOW && t >= b_lo) {
      const uint64_t bad = bad_in_block<D>(y, wave);
      if (lane == 0) s_bad[t & 1][wave] = bad;
    }
  };
  if (n_tiles > 0) {
    put(0);
    if (n_tiles > 1) fetch(1);
  }
  __syncthreads();
#pragma unroll 1
  for (int b = 0; b < n_tiles; ++b) {
    if (b + 1 < n_tiles) put(b + 1);
    if (b + 2 < n_tiles) fetch(b + 2);
    if (has && b < w_hi) {
#pragma unroll
      for (int t = 0; t < RT; ++t) upto[t] = b < pos[t] >> 6 ? 63 : -1;
      // MFMAs first: a wave that has some to issue goes before one in its
      // softmax (1 x 10,240 at d = 256: 1,109 us a call; all alike 1,156)
      __builtin_amdgcn_s_setprio(1);
      scores(b & 1);
      __builtin_amdgcn_s_setprio(0);
      softmax(b >= w_lo);
      __builtin_amdgcn_s_setprio(1);
      products(b & 1, b >= w_lo);
      __builtin_amdgcn_s_setprio(0);
    }
    if ((b + 1) % kPartBlocks == 0) fold(std::true_type{}, b);
    __syncthreads();
  }
  // the own blocks, as many at once as LDS holds
  constexpr int kSlots = kRawSlots<D>;
#pragma unroll 1
  for (int b0 = b_lo; b0 <= b_hi; b0 += kSlots) {
    if (b0 > b_lo) __syncthreads();
#pragma unroll 1
    for (int n = 0; n < kSlots && b0 + n <= b_hi; n += 2)
      stage_raw<D, SLOW>(a, i, hk, ctx, min(end, (b_hi + 1) * 64), c0, b0 + n, sm, n, s_bad, wave, lane);
    __syncthreads();
#pragma unroll 1
    for (int b = max(b0, w_lo); has && b <= min(b0 + kSlots - 1, w_hi); ++b) {
#pragma unroll
      for (int t = 0; t < RT; ++t) upto[t] = pos[t] >> 6 == b ? pos[t] & 63 : -1;
      raw_scores(b);
      softmax(true);
      raw_products(raw_slot<D>(sm, b - b0), b - b0);
    }
  }
  fold(std::false_type{}, 0);
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const float inv = 1.f / lt[t];
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
  __shared__ PrefillLds<D> sm[2];
  __shared__ f32x4 s_ot[P::kOtLds ? P::kRT * P::kOtLds : 1][P::kThreads];
  __shared__ uint64_t s_bad[kRawSlots<D>][P::kWaves];
  __shared__ float s_scale[2][2];
  // neighbouring work-groups take different heads: with 2, 4, 8 .. heads each
  // chiplet, and its L2, sees the keys of some of them only
  const int hk = blockIdx.x % a.Hk;
  // which sequence and rows, longest first (order_tiles)
  const i32x2 item = a.order[blockIdx.x / a.Hk];
  const int i = item[0];
  if (i < 0) return;
  const Entry e_ = entry_of(a, i);
  int c0 = e_.c0, len = e_.len, ctx = e_.ctx, cache_row = e_.row;
  // settled here, or their limits are worked out again where they are used
  // (1 x 10,240 at d = 256: 1,109 us a call, with this 1,100)
  asm volatile("" : "+s"(c0), "+s"(len), "+s"(ctx), "+s"(cache_row));
  const int64_t row0 = (int64_t)item[1] * P::kRows;
  const int64_t rows = (int64_t)len * a.G;
  if (ctx < 0) {  // no request: o = 0
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
    prefill_rows<D, false>(a, sm, s_ot, s_bad, s_scale, hk, i, cache_row, (uint32_t)row0, (uint32_t)rows, c0, ctx, ctx + len);
  else
    prefill_rows<D, true>(a, sm, s_ot, s_bad, s_scale, hk, i, cache_row, (uint32_t)row0, (uint32_t)rows, c0, ctx, ctx + len);
}

// ---------------------------------------------------------------------------
// few rows per sequence: the decode step, and prefill of few new tokens

// Records that join work-groups' shares of a row: per partition's unit
// and key/value head, O [rec_rows][D], and per row m and l.
struct RowsArgs {
  StepArgs s;
  float* rec_o;
  float* rec_ml;  // [..][rec_rows][2]: m, l
  int32_t* base;  // first unit of every sequence
  int32_t* total;  // how many units there are
  int max_parts;  // records that fit
  int rec_rows;   // rows of a record
  int chunk_rows;  // rows of a chunk, 16 RT
};

// A sequence's rows are cut into chunks.  A chunk's partitions reach to the
// last row's own block.
__device__ __forceinline__ int chunks_of(const RowsArgs& a, int len) {
  return (int)(((uint32_t)len * (uint32_t)a.s.G + a.chunk_rows - 1) / a.chunk_rows);
}

__device__ __forceinline__ int parts_of(const RowsArgs& a, int ctx, int len, int c) {
  const uint32_t last = min((uint32_t)(c + 1) * a.chunk_rows, (uint32_t)len * a.s.G) - 1;
  return ((ctx + (int)(last / (uint32_t)a.s.G)) >> 9) + 1;
}

__device__ __forceinline__ int len_of(const RowsArgs& a, int i) { return entry_of(a.s, i).len; }

// What a chunk costs, in units of a partition: its partitions, and its own
// block, first loads and outputs, which take about as long as two (two, one, none:
// 16 x 37 new tokens, 4 query heads to each of 8, d = 64 after 5,000 tokens 110, 115 and
// 118 us, d = 128 after 3,000 127, 134 and 134; decode of 256 x 4,096 161.7, 162.2 and
// 162.6; ragged turns after 4,000 to 8,000, whose contexts weigh more, 118, 112 and 113).
constexpr int kChunkCost = 2;

// units of all chunks of sequence i
__device__ __forceinline__ int all_units_of(const RowsArgs& a, int i) {
  const Entry e_ = entry_of(a.s, i);
  const int ctx = e_.ctx, len = e_.len;
  if (ctx < 0 || len <= 0) return 0;
  const int n = chunks_of(a, len);
  if ((ctx >> 9) == (ctx + len - 1) >> 9) return n * ((ctx >> 9) + 1 + kChunkCost);
  int sum = 0;
  for (int c = 0; c < n; ++c) sum += parts_of(a, ctx, len, c) + kChunkCost;
  return sum;
}

// Work-group w's run of `total` things dealt to W of them: the first total % W get one more.
__device__ __forceinline__ int run_begin(int total, int W, int w) {
  return w * (total / W) + min(w, total % W);
}
__device__ __forceinline__ int run_of(int total, int W, int x) {
  const int per = total / W, more = total % W, first = more * (per + 1);
  return x < first ? x / (per + 1) : more + (x - first) / per;
}

// Work-groups of k_attn_rows that share a CU.  With one its waves have all
// registers, and what hides the memory's latency are the loads that a wave has in
// flight (decode, 256 x 4,096 at d = 128: 162 us a call, with two 166; 16 x 16 new tokens,
// 8 query heads to each of 2, d = 256, after 5,000: 116, with two 149); fewer runs also leave
// fewer records.  Several new tokens at d = 64 and 128 keep the MFMAs busier with two (16 x 37
// tokens, 4 query heads to each of 8, d = 64, after 5,000: 110 us; one 171, three 116;
// d = 128, after 3,000: 127 and one 163).
//
// Bound by memory in decode: 256 x 4,096, 823 MB, 155 us, 5.3 TB/s, where a
// copy moves 4.65 and a kernel that only reads 6.1; 3 x 100,003, 307 MB, 58 us.  Few new
// tokens are bound by neither: 88 us of the ragged turns at d = 64 are 9.4 VALU instructions to
// an MFMA, one instruction a SIMD in 10 cycles and MFMAs busy a sixth of the time, so
// the two barriers and the dependent parts of a step count beside the issue.
template <int D, bool MULTI>
constexpr int kRowsPerCu = MULTI && D < 256 ? 2 : 1;

// All units of the batch in a row, sequence by sequence and chunk by chunk,
// are dealt out in equal runs to the W work-groups of a key/value head
// (blockIdx.x of gridDim.x): a batch of any lengths is balanced to one
// partition.  A chunk's first units are its partitions.  A run that begins a
// chunk folds its partitions as it goes; one that begins inside a chunk must
// leave each partition by itself, because the fold goes left to right.  If the
// batch has more units than there is room for records, chunks (decode:
// sequences) are dealt out whole.
//
// In a work-group the four waves share a partition, four tiles at a time: wave
// w computes the scores and p of tile w; p goes through LDS and every wave
// adds all four tiles to its own quarter of the dims.  So a partition's
// bytes are spread over four waves' loads, and no byte is loaded twice.  The
// own block's scores are shared out by 16 keys.
//
// MULTI: any number of new tokens, which k_attn_append has put into the tail
// (last block) or raw_k, raw_v (blocks that they filled).  Otherwise one each,
// which this kernel appends itself.
//
// STREAM: no other chunk reads the keys, and the caches need not keep them (decode,
// 256 x 4,096 at d = 128: 162 us instead of 178; 64 x 4 new tokens after 3,000: 98 instead of 119; but 5
// chunks a sequence, 16 x 37 tokens after 3,000: 151 instead of 127).
template <int D, int RT, bool MULTI, bool STREAM>
__global__ __launch_bounds__(256, (kRowsPerCu<D, MULTI>)) void k_attn_rows(const RowsArgs ra) {
  const StepArgs& a = ra.s;
  constexpr int KS = D / 32, KP = D / 64, DT = D / 64, R = 16 * RT;  // DT: dim tiles of a wave
  __shared__ u32x4 s_p[4][RT][2][64];
  __shared__ f32x4 s_raw[4][RT][64];
  __shared__ float s_max[4][RT][16];
  __shared__ int s_scan[4], s_at[2];
  __shared__ uint32_t s_red[4];
  const int hk = blockIdx.y, tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int W = gridDim.x;

  // the run [g0, g1) of units, and the sequence it begins in
  const int per = (a.N + 255) / 256, n0 = min(tid * per, a.N), n1 = min(n0 + per, a.N);
  int mine = 0;
  for (int n = n0; n < n1; ++n) mine += all_units_of(ra, n);
  int upto_ = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(upto_, o);
    if (lane >= o) upto_ += y;
  }
  if (lane == 63) s_scan[wave] = upto_;
  __syncthreads();
  const int total = s_scan[0] + s_scan[1] + s_scan[2] + s_scan[3];
  for (int w = 0; w < wave; ++w) upto_ += s_scan[w];
  const bool whole = total > ra.max_parts;
  const int g0 = run_begin(total, W, blockIdx.x), g1 = run_begin(total, W, blockIdx.x + 1);
  if (blockIdx.x == 0 && hk == 0 && tid == 0) *ra.total = total;
  if (g0 >= g1 && !whole) return;
  if (g0 >= upto_ - mine && g0 < upto_) {
    int at = upto_ - mine, n = n0;
    for (; n < n1 - 1; ++n) {
      const int x = all_units_of(ra, n);
      if (g0 < at + x) break;
      at += x;
    }
    s_at[0] = n;
    s_at[1] = at;
  }
  __syncthreads();
  int i = whole ? (MULTI ? 0 : blockIdx.x) : s_at[0], base = whole ? 0 : s_at[1], c = 0;
  auto skip = [&](int n) {  // n chunks further
    c += n;
    for (int k; i < a.N && c >= (k = max(1, chunks_of(ra, len_of(ra, i)))); ++i) c -= k;
  };
  if (MULTI && whole) skip(blockIdx.x);

  for (int f = g0; whole ? i < a.N : f < g1;) {
    const Entry e_ = entry_of(a, i);
    const int c0 = MULTI ? e_.c0 : i, len = MULTI ? e_.len : 1, ctx = e_.ctx, cache_row = e_.row;
    const int np = ctx < 0 || len <= 0 ? 0 : parts_of(ra, ctx, len, c);
    if (c == 0 && np > 0 && !whole && hk == 0 && tid == 0 && f == base) ra.base[i] = base;
    if (np == 0 || (!whole && f >= base + np)) {  // nothing there, or behind it
      if (np) base += np + kChunkCost;
      f = max(f, base);
      if (MULTI && whole) {
        skip(W);
      } else if (np && c + 1 < chunks_of(ra, len)) {
        ++c;
      } else {
        c = 0;
        i += !MULTI && whole ? W : 1;
      }
      continue;
    }
    const int end = ctx + len;
    const uint32_t rows = (uint32_t)len * (uint32_t)a.G, row0 = (uint32_t)c * R;
    const uint32_t last_row = min(row0 + R, rows) - 1;
    const int p_lo = whole ? 0 : f - base, p_hi = whole ? np : min(np, g1 - base);
    // own blocks of the chunk's rows (there are two at most)
    const int b_lo = (ctx + (int)(row0 / (uint32_t)a.G)) >> 6, b_hi = (ctx + (int)(last_row / (uint32_t)a.G)) >> 6;
    const int b_end = min(p_hi * kPartBlocks, b_hi);  // the 8-bit blocks end here

    u32x4 q[RT][KS];
    int pos[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const uint32_t row = min(row0 + t * 16 + r, rows - 1);
      const int token = (int)(row / (uint32_t)a.G), head = hk * a.G + (int)(row % (uint32_t)a.G);
      pos[t] = ctx + token;
      const uint16_t* qp = a.q + (int64_t)(c0 + token) * a.q_stride + (int64_t)head * D;
#pragma unroll
      for (int x = 0; x < KS; ++x) q[t][x] = *(const u32x4*)(qp + (x >> 1) * 64 + g * 16 + (x & 1) * 8);
    }
    f32x4 O[RT][DT], Ot[RT][DT], l[RT];  // the partition's, the folded total
    float m[RT], mt[RT], lt[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      m[t] = mt[t] = kNegInf;
      lt[t] = 0.f;
      l[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int x = 0; x < DT; ++x) O[t][x] = Ot[t][x] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    auto record = [&](int p, const f32x4 (&o)[RT][DT], const float (&mr)[RT], const float (&lr)[RT]) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        if (row0 + t * 16 + r > last_row) continue;
        const int64_t rec = ((int64_t)(base + p) * a.Hk + hk) * ra.rec_rows + t * 16 + r;
        float* to = ra.rec_o + rec * D + wave * DT * 16 + g * 4;
#pragma unroll
        for (int x = 0; x < DT; ++x) *(f32x4*)(to + x * 16) = o[t][x];
        if (wave == 0 && g == 0) {
          ra.rec_ml[rec * 2] = mr[t];
          ra.rec_ml[rec * 2 + 1] = lr[t];
        }
      }
    };
    auto end_partition = [&](int p) __attribute__((always_inline)) {
      if (p_lo > 0) {
        float l0[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) l0[t] = l[t][0];
        record(p, O, m, l0);
      }
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        if (p_lo == 0) {
          float wa, wb;
          fold_weights(mt[t], m[t], wa, wb);
          lt[t] = __builtin_fmaf(l[t][0], wb, lt[t] * wa);
#pragma unroll
          for (int x = 0; x < DT; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) Ot[t][x][e] = __builtin_fmaf(O[t][x][e], wb, Ot[t][x][e] * wa);
        }
        m[t] = kNegInf;
        l[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < DT; ++x) O[t][x] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
    };
    // O += V^T p for a tile that some rows see less of (keys up to upto[t]):
    // a key whose V is not finite must not reach them as 0 * NaN.  One
    // product for every number n of such keys that a row may see.
    auto masked_pv = [&](const u32x4 (&v)[DT][2], const u32x4 (&p)[RT][2], const int (&upto)[RT], uint64_t bad) __attribute__((always_inline)) {
      int sees[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t) sees[t] = upto[t] < 0 ? 0 : __popcll(bad & (~0ull >> (63 - upto[t])));
#pragma unroll
      for (int x = 0; x < DT; ++x) {
        f32x4 was[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) was[t] = O[t][x];
        uint64_t drop = bad;
#pragma unroll 1
        for (int n = 0; n <= __popcll(bad); ++n, drop &= drop - 1) {
          const u32x4 v0 = drop_keys(v[x][0], drop, g, 0), v1 = drop_keys(v[x][1], drop, g, 1);
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            const f32x4 y_ = mma(v1, p[t][1], mma(v0, p[t][0], was[t]));
#pragma unroll
            for (int e = 0; e < 4; ++e) O[t][x][e] = sees[t] == n ? y_[e] : O[t][x][e];
          }
        }
      }
    };

    // ---- the 8-bit blocks, four a step.  K of a step is asked for as soon as
    // the scores of the step before have been taken from its registers, V
    // as soon as its products have, so loads are in flight all the time.
    BlockRun run;
    u32x4 kb[4][KP], vb[4][DT];
    auto fetch_ids = [&](int b) __attribute__((always_inline)) { run.id = pool_block(a, cache_row, b + lane); };
    auto fetch_scales = [&]() __attribute__((always_inline)) {
      const int64_t at = (int64_t)run.id * a.Hk + hk;
      run.ks = a.cache.k_scale[at];
      run.vs = a.cache.v_scale[at];
    };
    auto fetch_k = [&](int b0) __attribute__((always_inline)) {  // of this wave's own tile
      const int bt = __builtin_amdgcn_readfirstlane(min(b0 + wave, b_end - 1) & 63);
      const int64_t at = (int64_t)__builtin_amdgcn_readlane(run.id, bt) * a.Hk + hk;
      const uint8_t* kp_ = a.cache.k8 + at * (64 * D) + g * 16;
#pragma unroll
      for (int sub = 0; sub < 4; ++sub)
#pragma unroll
        for (int x = 0; x < KP; ++x) kb[sub][x] = load<STREAM>((const u32x4*)(kp_ + x * 4096 + key_of(sub, r) * 64));
    };
    auto fetch_v = [&](int b0) __attribute__((always_inline)) {  // of all four, this wave's dims
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int64_t at = (int64_t)__builtin_amdgcn_readlane(run.id, min(b0 + t, b_end - 1) & 63) * a.Hk + hk;
        const uint8_t* vp = a.cache.v8 + at * (64 * D) + (wave * DT * 16 + r) * 64 + g * 16;
#pragma unroll
        for (int x = 0; x < DT; ++x) vb[t][x] = load<STREAM>((const u32x4*)(vp + x * 1024));
      }
    };
    // ---- an own block in the input type: this wave's 16 keys and its dims of V
    u32x4 rk[KS], rv[DT][2];
    uint32_t rn[DT];  // decode: V of the new token
    auto fetch_raw = [&](int b) __attribute__((always_inline)) {
      const bool in_tail = !MULTI || b == (end - 1) >> 6;
      const int64_t at = in_tail ? ((int64_t)cache_row * a.Hk + hk) * (64 * D)
                                 : ((int64_t)((c0 >> 6) + 2 * i + b - (ctx >> 6)) * a.Hk + hk) * (64 * D);
      const uint16_t* tk = (in_tail ? a.cache.tail_k : a.raw_k) + at;
      const uint16_t* tv = (in_tail ? a.cache.tail_v : a.raw_v) + at;
      const int key = key_of(wave, r);
      const uint16_t* kr = (!MULTI && key == (ctx & 63) ? a.k + (int64_t)i * a.k_stride + (int64_t)hk * D : tk + key * D) + g * 16;
#pragma unroll
      for (int x = 0; x < KS; ++x) rk[x] = *(const u32x4*)(kr + (x >> 1) * 64 + (x & 1) * 8);
#pragma unroll
      for (int x = 0; x < DT; ++x) {
        const int dim = (wave * DT + x) * 16 + r;
        rv[x][0] = *(const u32x4*)(tv + dim * 64 + g * 16);
        rv[x][1] = *(const u32x4*)(tv + dim * 64 + g * 16 + 8);
        if (!MULTI) rn[x] = a.v[(int64_t)i * a.v_stride + (int64_t)hk * D + dim];
      }
    };
    auto do_raw = [&](int b) __attribute__((always_inline)) {
      if (MULTI) __syncthreads();  // the scores of a raw block before have been read
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        f32x4 y_ = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < KS; ++x) y_ = mma(rk[x], q[t][x], y_);
        s_raw[wave][t][lane] = y_;
      }
      __syncthreads();
      u32x4 p[RT][2];
      int upto[RT];
      float alpha[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        f32x4 s[4];
        upto[t] = pos[t] >> 6 == b ? pos[t] & 63 : -1;
#pragma unroll
        for (int sub = 0; sub < 4; ++sub) {
          s[sub] = s_raw[sub][t][lane];
#pragma unroll
          for (int e = 0; e < 4; ++e) s[sub][e] = 16 * g + 4 * sub + e <= upto[t] ? s[sub][e] : kNegInf;
        }
        const float mn = move_ref(m[t], max_over_groups(max16(s)) * a.c), ref = ref_of(mn);
        alpha[t] = exp2_(m[t] - ref);
        m[t] = mn;
        probabilities(s, a.c, ref, p[t]);
        l[t][0] *= alpha[t];
        add_sum(p[t], l[t]);
      }
      // V: keys past the sequence's end are not there yet (whatever the tail
      // holds); decode's new one comes from the call
      const int at = end - 1 - b * 64;
      uint32_t nan16 = 0;
#pragma unroll
      for (int x = 0; x < DT; ++x) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int key = 16 * g + 2 * j;
          uint32_t w = rv[x][j >> 2][j & 3];
          w = key > at ? 0u : key + 1 > at ? w & 0xffffu : w;
          if (!MULTI) w = key == at ? rn[x] : key + 1 == at ? (w & 0xffffu) | rn[x] << 16 : w;
          if (MULTI) {
            nan16 |= (w & 0x7f80u) == 0x7f80u ? 1u << (2 * j) : 0u;
            nan16 |= (w & 0x7f800000u) == 0x7f800000u ? 2u << (2 * j) : 0u;
          }
          rv[x][j >> 2][j & 3] = w;
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) O[t][x] *= alpha[t];
      }
      const uint64_t bad = MULTI ? bad_keys(nan16) : 0;
      if (bad) {
        masked_pv(rv, p, upto, bad);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int x = 0; x < DT; ++x)
#pragma unroll
            for (int t = 0; t < RT; ++t) O[t][x] = mma(rv[x][h], p[t][h], O[t][x]);
      }
    };

    auto step = [&](int b0, auto more_) __attribute__((always_inline)) {
      constexpr bool more = decltype(more_)::value;
      f32x4 s[RT][4];
      const float ks = lane_of(run.ks, __builtin_amdgcn_readfirstlane(min(b0 + wave, b_end - 1) & 63));
      float vs[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) vs[t] = lane_of(run.vs, min(b0 + t, b_end - 1) & 63);
#pragma unroll
      for (int sub = 0; sub < 4; ++sub) {
#pragma unroll
        for (int x = 0; x < KP; ++x) {
          u32x4 k0, k1;
          from_e4m3(kb[sub][x], ks, k0, k1);
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            s[t][sub] = mma(k0, q[t][2 * x], x ? s[t][sub] : f32x4{0.f, 0.f, 0.f, 0.f});
            s[t][sub] = mma(k1, q[t][2 * x + 1], s[t][sub]);
          }
        }
      }
      if (more) {
        if (((b0 + 4) & 63) == 0) {
          fetch_ids(b0 + 4);
          fetch_scales();
          asm volatile("" : "+v"(run.ks), "+v"(run.vs));
        }
        fetch_k(b0 + 4);
      } else if (!MULTI) {
        fetch_raw(b_hi);
      }
      const bool mytile = more || b0 + wave < b_end;
      mfma_done();
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        if (MULTI && b0 + wave >= b_lo) {  // only rows whose own block comes later see it
          const bool sees = b0 + wave < pos[t] >> 6;
#pragma unroll
          for (int sub = 0; sub < 4; ++sub)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[t][sub][e] = sees ? s[t][sub][e] : kNegInf;
        }
        const float smax = max_over_groups(max16(s[t]));
        if (g == 0) s_max[wave][t][r] = smax;
      }
      __syncthreads();
      float mm[RT][5];  // the reference before and after every tile
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        mm[t][0] = m[t];
#pragma unroll
        for (int n = 0; n < 4; ++n) mm[t][n + 1] = more || b0 + n < b_end ? move_ref(mm[t][n], s_max[n][t][r] * a.c) : mm[t][n];
        if (mytile) {
          u32x4 pf[2];
          const float mine_ = wave == 0 ? mm[t][1] : wave == 1 ? mm[t][2] : wave == 2 ? mm[t][3] : mm[t][4];
          probabilities(s[t], a.c, ref_of(mine_), pf);
          s_p[wave][t][0][lane] = pf[0];
          s_p[wave][t][1][lane] = pf[1];
        }
      }
      __syncthreads();
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        if (!more && b0 + n >= b_end) break;
        u32x4 p[RT][2], v[DT][2];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          const float alpha = exp2_(mm[t][n] - ref_of(mm[t][n + 1]));
          p[t][0] = s_p[n][t][0][lane];
          p[t][1] = s_p[n][t][1][lane];
          l[t][0] *= alpha;
          add_sum(p[t], l[t]);
#pragma unroll
          for (int x = 0; x < DT; ++x) O[t][x] *= alpha;
        }
        uint64_t bad = 0;
        if (MULTI && b0 + n >= b_lo) {
          uint32_t nan16 = 0;
#pragma unroll
          for (int x = 0; x < DT; ++x)
#pragma unroll
            for (int e = 0; e < 16; ++e) nan16 |= ((vb[n][x][e >> 2] >> (8 * (e & 3))) & 0x7f) == 0x7f ? 1u << e : 0u;
          bad = bad_keys(nan16);
        }
#pragma unroll
        for (int x = 0; x < DT; ++x) from_e4m3(vb[n][x], vs[n], v[x][0], v[x][1]);
        if (MULTI && bad) {
          int upto[RT];
#pragma unroll
          for (int t = 0; t < RT; ++t) upto[t] = b0 + n < pos[t] >> 6 ? 63 : -1;
          masked_pv(v, p, upto, bad);
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int x = 0; x < DT; ++x)
#pragma unroll
              for (int t = 0; t < RT; ++t) O[t][x] = mma(v[x][h], p[t][h], O[t][x]);
        }
      }
#pragma unroll
      for (int t = 0; t < RT; ++t) m[t] = mm[t][4];
      if (more) fetch_v(b0 + 4);
      if (((b0 + 4) & (kPartBlocks - 1)) == 0 && b0 + 4 <= b_hi) {
        const int p = b0 / kPartBlocks;
        if (MULTI && b_lo / kPartBlocks == p) {  // the partition's last block is a row's own
          fetch_raw(b_lo);
          do_raw(b_lo);
        }
        end_partition(p);
      }
    };
    if (p_lo * kPartBlocks < b_end) {
      int b0 = p_lo * kPartBlocks;
      fetch_ids(b0 & ~63);
      fetch_scales();
      fetch_k(b0);
      fetch_v(b0);
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int x = 0; x < KS; ++x) settle(q[t][x]);
      asm volatile("" : "+v"(run.ks), "+v"(run.vs));
#pragma unroll 1
      for (; b0 + 4 < b_end; b0 += 4) step(b0, std::true_type{});
      // by itself, so that in the loop every load is followed by the others
      // (if it might not be, a wait for K would be one for V as well)
      step(b0, std::false_type{});
    } else if (!MULTI) {
      fetch_raw(b_hi);
    }
    if (p_hi == np) {
      if (MULTI) {
        if (b_lo < b_hi && b_lo / kPartBlocks == np - 1) {
          fetch_raw(b_lo);
          do_raw(b_lo);
        }
        fetch_raw(b_hi);
      }
      do_raw(b_hi);
      if (!MULTI && c == 0) {
        // append: the tail's row and column; a full block is quantised
        const int at = ctx & 63;
        uint16_t* wk = a.cache.tail_k + ((int64_t)cache_row * a.Hk + hk) * (64 * D);
        uint16_t* wv = a.cache.tail_v + ((int64_t)cache_row * a.Hk + hk) * (64 * D);
        const uint16_t* nk = a.k + (int64_t)i * a.k_stride + (int64_t)hk * D;
        const uint16_t* nv = a.v + (int64_t)i * a.v_stride + (int64_t)hk * D;
        if (tid < D / 8) *(u32x4*)(wk + at * D + tid * 8) = *(const u32x4*)(nk + tid * 8);
        for (int x = tid; x < D; x += 256) wv[x * 64 + at] = nv[x];
        const int block = at == 63 ? block_to_write(a, cache_row, b_hi) : -1;
        if (block >= 0) {
          __threadfence_block();
          __syncthreads();
          quantise_block<D>(
              a.cache, (int64_t)block * a.Hk + hk,
              [&](int x) { return ((const u32x4*)wk)[x]; }, [&](int x) { return ((const u32x4*)wv)[x]; }, s_red);
        }
      }
      end_partition(np - 1);
    }
    if (p_lo == 0 && p_hi < np) record(0, Ot, mt, lt);
    if (p_lo == 0 && p_hi == np) {
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const float inv = 1.f / lt[t];
        const uint32_t row = row0 + t * 16 + r;
        if (row > last_row) continue;
        uint16_t* o = a.o + ((int64_t)(c0 + (int)(row / (uint32_t)a.G)) * a.H + hk * a.G + (int)(row % (uint32_t)a.G)) * D +
                      wave * DT * 16 + g * 4;
#pragma unroll
        for (int x = 0; x < DT; ++x)
          *(u32x2*)(o + x * 16) = u32x2{pack2(Ot[t][x][0] * inv, Ot[t][x][1] * inv), pack2(Ot[t][x][2] * inv, Ot[t][x][3] * inv)};
      }
    }
    __syncthreads();  // LDS is used again by the next chunk
    if (MULTI && whole) {
      skip(W);
      continue;
    }
    f = whole ? 0 : base + p_hi;
    if (whole || p_hi == np) {
      base += np + kChunkCost;
      f = max(f, base);
      if (c + 1 < chunks_of(ra, len)) {
        ++c;
      } else {
        c = 0;
        i += whole ? W : 1;
      }
    }
  }
}

// Joins what several work-groups did of a chunk, left to right; chunks that
// one work-group did alone are finished, rows of entries without a request get o = 0.
// A wave takes a row, a lane D / 64 of its dims.  The fold is a chain over the
// records, but what it needs of each is not: the weights of 64 folds come
// from prefix maxima (exact in any order), a lane each, and many records are
// asked for before the first is used, so the chain is two operations a record
// (195 records a row, 3 x 100,003 at d = 128: 18 us; where it was 20, two batches in turn, the
// next asked for during the fold, took 26, weights through LDS and a wave to a work-group 59).
template <int D>
__global__ __launch_bounds__(256) void k_attn_join(const RowsArgs ra, int W) {
  constexpr int V = D / 64;
  typedef float fv __attribute__((ext_vector_type(V)));
  const StepArgs& a = ra.s;
  const int i = blockIdx.x, hk = blockIdx.y, lane = threadIdx.x & 63;
  const Entry e_ = entry_of(a, i);
  const int c0 = e_.c0, len = e_.len, ctx = e_.ctx;
  const int x_ = __builtin_amdgcn_readfirstlane(blockIdx.z * 4 + (threadIdx.x >> 6));
  const int c = x_ / ra.rec_rows, rr = x_ % ra.rec_rows;
  const uint32_t row = (uint32_t)c * ra.chunk_rows + rr, G = (uint32_t)a.G;
  if (len <= 0 || row >= (uint32_t)len * G) return;
  uint16_t* o = a.o + ((int64_t)(c0 + (int)(row / G)) * a.H + hk * a.G + (int)(row % G)) * D + lane * V;
  if (ctx < 0) {
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = 0;
    return;
  }
  const int total = *ra.total;
  if (total > ra.max_parts) return;
  int base = ra.base[i];
  for (int x = 0; x < c; ++x) base += parts_of(ra, ctx, len, x) + kChunkCost;
  // where the run of the work-group with the chunk's first partition ends
  const int cut = run_begin(total, W, run_of(total, W, base) + 1);
  const int n = base + parts_of(ra, ctx, len, c) - cut + 1;  // records
  if (n <= 1) return;
  const int64_t step = (int64_t)a.Hk * ra.rec_rows, at = (int64_t)hk * ra.rec_rows + rr;
  const int64_t rec0 = base * step + at;
  fv O = *(const fv*)(ra.rec_o + rec0 * D + lane * V);
  float m = ra.rec_ml[rec0 * 2], l = ra.rec_ml[rec0 * 2 + 1];
  // the others follow each other
  const int k = n - 1;
  const float* po = ra.rec_o + (cut * step + at) * D;
  const float* pm = ra.rec_ml + (cut * step + at) * 2;
  const int64_t so = step * D, sm = step * 2;
  auto batch = [&](auto size_, int j0, int u0, float mp, float& wa, float& wb) __attribute__((always_inline)) {
    constexpr int S = decltype(size_)::value;  // records asked for at once
    fv Op[S];
    float lp[S];
    const float *to = po + (j0 + u0) * so, *tm = pm + (j0 + u0) * sm;
#pragma unroll
    for (int u = 0; u < S; ++u) {
      Op[u] = *(const fv*)(to + lane * V);
      lp[u] = tm[1];
      if (j0 + u0 + u + 1 < k) {  // past the last: the last again
        to += so;
        tm += sm;
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // or the loads are moved to where they are used
    if (u0 == 0) {  // weights of the next 64 folds
      float up = mp;
#pragma unroll
      for (int y = 1; y < 64; y <<= 1) {
        const float z = __shfl_up(up, y);
        if (lane >= y) up = fmaxf(up, z);
      }
      const float prev = __shfl_up(up, 1);
      float before = lane ? fmaxf(m, prev) : m;
      fold_weights(before, mp, wa, wb);
      m = fmaxf(m, __shfl(up, 63));
    }
    auto folds = [&](auto all_) __attribute__((always_inline)) {
#pragma unroll
      for (int u = 0; u < S; ++u) {
        const bool there = decltype(all_)::value || j0 + u0 + u < k;
        const float ya = lane_of(wa, u0 + u), yb = lane_of(wb, u0 + u);
        l = there ? __builtin_fmaf(lp[u], yb, l * ya) : l;
#pragma unroll
        for (int e = 0; e < V; ++e) O[e] = there ? __builtin_fmaf(Op[u][e], yb, O[e] * ya) : O[e];
      }
    };
    if (j0 + u0 + S <= k)
      folds(std::true_type{});
    else
      folds(std::false_type{});
  };
  for (int j0 = 0; j0 < k; j0 += 64) {
    const float mp = j0 + lane < k ? pm[(j0 + lane) * sm] : kNegInf;
    float wa = 0.f, wb = 0.f;
    if (k - j0 > 16) {
      constexpr int S = 32;  // with 64 more of the last batch is in vain (3 x 100,003: 82 us a call, with 32 77)
#pragma unroll 1
      for (int u0 = 0; u0 < 64 && j0 + u0 < k; u0 += S) batch(std::integral_constant<int, S>{}, j0, u0, mp, wa, wb);
    } else {
      batch(std::integral_constant<int, 16>{}, j0, 0, mp, wa, wb);
    }
  }
  const float inv = 1.f / l;
#pragma unroll
  for (int e = 0; e < V; ++e) o[e] = (uint16_t)pack2(O[e] * inv, 0.f);
}

}  // namespace attn
