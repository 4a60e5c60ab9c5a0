// The attention cache's write side (tails, block quantisation) and its
// read-out.
//
// A block is quantised from its 64 tokens at once: the largest finite
// magnitude gives the scale's exponent, then every element is scaled (exactly,
// by a power of two) and rounded to e4m3.  All of it is bound by memory and
// small beside the attention that reads the cache: per token and head 4 d bytes in
// and 2 d out.
#pragma once

#include "attn_device.hpp"

namespace attn {

struct CacheArgs {
  uint8_t *k8, *v8;
  float *k_scale, *v_scale;
  uint16_t *tail_k, *tail_v;
  int num_blocks, num_slots;
};

// The tokens of a call and where they belong.
struct StepArgs {
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const int32_t *cu, *ctx_len, *table, *slot;
  int N, T, H, Hk, G, max_blocks;
  uint16_t* o;
  float c;  // softmax scale * log2(e)
  CacheArgs cache;
  uint16_t *old_k, *old_v;  // [N, Hk, 64, d], [N, Hk, d, 64]: the tails as they were before the call
  uint16_t *raw_k, *raw_v;  // as the old tails, per touched block: those that the call fills, in the input type
  int32_t* bad;             // per touched block and head: does its V hold a value that is not finite?
  i32x2* order;             // prefill: (sequence, tile of tile_rows rows), (-1, 0) for none, in the order they are begun
  int tile_rows;
};

// Batch entry i: its packed tokens [c0, c0 + len), the tokens in its cache and its
// cache row.  An entry without a request (context -1, a row that the cache does not
// have, or more full blocks than a row of the table is wide) has ctx = row = -1
// in every kernel: o = 0, nothing is written.  So positions fit 32 bits, and the
// work that a wrong context can ask for is held to the table's width.
struct Entry {
  int c0, len, ctx, row;
};

// cu[i], held to the call's tokens
__device__ __forceinline__ int cu_at(const StepArgs& a, int i) { return min(max(a.cu[i], 0), a.T); }

__device__ __forceinline__ Entry entry_of(const StepArgs& a, int i) {
  Entry e;
  e.c0 = a.cu ? cu_at(a, i) : i;
  e.len = a.cu ? max(cu_at(a, i + 1) - e.c0, 0) : 1;
  e.ctx = a.ctx_len[i];
  e.row = row_of(a.slot, i, a.cache.num_slots);
  const bool fits = e.ctx <= 0x7fffffff - kBlock - e.len && (e.ctx + e.len) >> 6 <= a.max_blocks;
  if (e.ctx < 0 || e.row < 0 || !fits) e.ctx = e.row = -1;
  return e;
}

// the pool block of a row's block b, held to the pool
__device__ __forceinline__ int pool_block(const StepArgs& a, int row, int b) {
  const int id = a.table[(size_t)row * a.max_blocks + min(b, a.max_blocks - 1)];
  return min(max(id, 0), a.cache.num_blocks - 1);
}

// the same for writing: -1 where the table has no block of the pool
__device__ __forceinline__ int block_to_write(const StepArgs& a, int row, int b) {
  const int id = b < a.max_blocks ? a.table[(size_t)row * a.max_blocks + b] : -1;
  return id < a.cache.num_blocks ? max(id, -1) : -1;
}

// largest finite magnitude among eight bf16, as its bits (ordered like the values)
__device__ __forceinline__ uint32_t amax8(u32x4 x, uint32_t m) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = x[i] & 0x7fffu, hi = (x[i] >> 16) & 0x7fffu;
    m = max(m, lo < 0x7f80u ? lo : 0u);
    m = max(m, hi < 0x7f80u ? hi : 0u);
  }
  return m;
}

// exponent e of the scale: the least e >= -100 with amax <= 448 * 2^e
// (448 = 1.75 * 2^8; amax as bf16 bits)
__device__ __forceinline__ int scale_exponent(uint32_t amax) {
  return max((int)(amax >> 7) - 127 - 8 + ((amax & 0x7fu) > 0x60u ? 1 : 0), -100);
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// whether one of eight bf16 is not finite
__device__ __forceinline__ bool not_finite8(u32x4 x) {
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) bad |= (x[i] & 0x7f80u) == 0x7f80u || (x[i] & 0x7f800000u) == 0x7f800000u;
  return bad;
}

// eight bf16 divided by 2^e -> eight e4m3, nearest even; what is not finite
// becomes NaN.  At the largest exponent, 120, e4m3 reaches past bf16: what would
// round to 256 * 2^120, which is infinite there, is held to 240 * 2^120.
__device__ __forceinline__ u32x2 to_e4m3(u32x4 x, int e) {
  const float inv = pow2(-e), most = e == 120 ? 240.f : 448.f;
  u32x2 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float f[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      f[2 * j] = __uint_as_float(x[2 * i + j] << 16) * inv;
      f[2 * j + 1] = __uint_as_float(x[2 * i + j] & 0xffff0000u) * inv;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      f[j] = __builtin_isfinite(f[j]) ? __builtin_amdgcn_fmed3f(f[j], -most, most) : __uint_as_float(0x7fc00000u);
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], w, true);
    r[i] = (uint32_t)w;
  }
  return r;
}

// 16 e4m3 times a power of two -> 16 bf16 (exact)
__device__ __forceinline__ void from_e4m3(u32x4 x, float scale, u32x4& lo, u32x4& hi) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[i], scale, false));
    const uint32_t b = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[i], scale, true));
    (i < 2 ? lo : hi)[2 * (i & 1)] = a;
    (i < 2 ? lo : hi)[2 * (i & 1) + 1] = b;
  }
}

// max over a work-group of 256 threads; `red` is reused by every call
__device__ __forceinline__ uint32_t block_max256(uint32_t m, uint32_t* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  return max(max(red[0], red[1]), max(red[2], red[3]));
}

// Quantises one block of one head by 256 threads.  kc(i) is K's chunk i (key
// i / (D / 8), dims 8 (i % (D / 8)) ..), vc(i) is V's chunk i (dim i / 8, keys 8 (i % 8) ..).
template <int D, class FK, class FV>
__device__ __forceinline__ void quantise_block(const CacheArgs& c, int64_t at, FK&& kc, FV&& vc, uint32_t* red) {
  constexpr int n = 64 * D / 8 / 256;
  u32x4 x[n];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < n; ++i) m = amax8(x[i] = kc(threadIdx.x + 256 * i), m);
  int e = scale_exponent(block_max256(m, red));
#pragma unroll
  for (int i = 0; i < n; ++i) {
    const int ch = threadIdx.x + 256 * i, key = ch / (D / 8), dim = ch % (D / 8) * 8;
    *(u32x2*)(c.k8 + at * (64 * D) + (dim >> 6) * 4096 + key * 64 + (dim & 63)) = to_e4m3(x[i], e);
  }
  if (threadIdx.x == 0) c.k_scale[at] = pow2(e);
  m = 0;
#pragma unroll
  for (int i = 0; i < n; ++i) m = amax8(x[i] = vc(threadIdx.x + 256 * i), m);
  e = scale_exponent(block_max256(m, red));
#pragma unroll
  for (int i = 0; i < n; ++i)
    *(u32x2*)(c.v8 + at * (64 * D) + (int64_t)(threadIdx.x + 256 * i) * 8) = to_e4m3(x[i], e);
  if (threadIdx.x == 0) c.v_scale[at] = pow2(e);
}

// The i with slots(i) <= x < slots(i + 1), slots(i) = cu[i] / 64 + per * i: room for every block that
// sequence i's tokens can touch, found without a prefix sum over the batch.  0 if x lies before slots(0).
__device__ __forceinline__ int seq_of_item(const StepArgs& a, int x) {
  int lo = 0, hi = a.N - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((cu_at(a, mid) >> 6) + 2 * mid <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Four keys of four dims (two words a key) -> four dims of four keys.
__device__ __forceinline__ void transpose4(const u32x2 (&x)[4], u32x2 (&t)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t w0 = x[0][e >> 1], w1 = x[1][e >> 1], w2 = x[2][e >> 1], w3 = x[3][e >> 1];
    t[e] = e & 1 ? u32x2{w0 >> 16 | (w1 & 0xffff0000u), w2 >> 16 | (w3 & 0xffff0000u)}
                 : u32x2{(w0 & 0xffffu) | w1 << 16, (w2 & 0xffffu) | w3 << 16};
  }
}

// The order in which the attention kernel begins its row tiles: those with the
// most keys first, whatever sequence they are of, so that the short ones fill the
// end (call of 5 x 2,048, 640 tiles on 256 CUs: 172 us; sequence by sequence 196).
// Sequence i has the tiles floor(cu[i] G / tile_rows) + i and on, one too many
// for some.  A counting sort by keys in kClasses classes; which tile of a class
// comes first is not defined, and nothing but time depends on it.
constexpr int kClasses = 512;

template <int TH>
__device__ void order_tiles(const StepArgs& a, int* hist /* [kClasses] */, int* most) {
  const int tid = threadIdx.x, n = (int)((int64_t)a.T * a.G / a.tile_rows) + a.N;
  for (int x = tid; x < kClasses; x += TH) hist[x] = 0;
  if (tid == 0) *most = 0;
  __syncthreads();
  int m = 0;
  for (int i = tid; i < a.N; i += TH) {
    const Entry e = entry_of(a, i);
    m = max(m, (e.ctx + e.len) >> 6);
  }
  atomicMax(most, m);
  __syncthreads();
  const int shift = max(0, 32 - __builtin_clz(*most + 1) - 9);  // (most + 1) >> shift < kClasses
  auto item = [&](int x, i32x2& to) -> int {  // its class
    int lo = 0, hi = a.N - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((int)((int64_t)cu_at(a, mid) * a.G / a.tile_rows) + mid <= x)
        lo = mid;
      else
        hi = mid - 1;
    }
    const Entry e = entry_of(a, lo);
    const int tile = x - ((int)((int64_t)e.c0 * a.G / a.tile_rows) + lo);
    const int64_t rows = (int64_t)e.len * a.G, row0 = (int64_t)tile * a.tile_rows;
    const bool none = tile < 0 || row0 >= rows;
    to = none ? i32x2{-1, 0} : i32x2{lo, tile};
    const int keys = e.ctx + (int)((min(row0 + a.tile_rows, rows) - 1) / a.G);  // -1 in a refused sequence at least
    return kClasses - 1 - (none ? 0 : min(((max(keys, 0) >> 6) + 1) >> shift, kClasses - 1));
  };
  i32x2 it;
  for (int x = tid; x < n; x += TH) atomicAdd(&hist[item(x, it)], 1);
  __syncthreads();
  if (tid < 64) {  // exclusive sums, by one wave
    int own[kClasses / 64], sum = 0;
#pragma unroll
    for (int e = 0; e < kClasses / 64; ++e) {
      own[e] = sum;
      sum += hist[tid * (kClasses / 64) + e];
    }
    int upto = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int y = __shfl_up(upto, o);
      upto += tid >= o ? y : 0;
    }
#pragma unroll
    for (int e = 0; e < kClasses / 64; ++e) hist[tid * (kClasses / 64) + e] = upto - sum + own[e];
  }
  __syncthreads();
  for (int x = tid; x < n; x += TH) {
    const int at = atomicAdd(&hist[item(x, it)], 1);
    a.order[at] = it;
  }
}

// Appends a call's tokens: a work-group per (touched block, key/value head).
// Full blocks are quantised.  The work-group of a sequence's first touched
// block also keeps the tail as it was for the attention that follows (its
// rows are that block's earlier tokens) and then writes the new tail, so that
// no two work-groups touch one tail.  Every work-group notes whether its
// block's V has a value that is not finite.
//
// A block is read once, into registers: K in runs of 8 dims of a key, V in
// squares of four keys by four dims, which turn over in the thread; only V's
// bytes go through LDS, to leave in whole lines.
//
// RAW: for k_attn_rows, which reads no V by token: the blocks that the call
// fills, except a sequence's last, are left in raw_k and raw_v in the tail's
// layout.  Otherwise the first work-group of head 0 makes the order of the row
// tiles instead, and the rest count from the second.
//
// Bound by memory: 5 x 2,048, 16 heads, d = 128, 84 MB read and 42 written in 27 us, 4.7 TB/s.
template <int D>
constexpr int kAppendThreads = D == 256 ? 512 : 256;  // a thread's share of a block stays in registers

template <int D, bool RAW>
__global__ __launch_bounds__(kAppendThreads<D>, D == 256 ? 2 : 4) void k_attn_append(const StepArgs a) {
  constexpr int TH = kAppendThreads<D>;
  constexpr int n = 64 * D / 8 / TH, nsq = 64 * D / 16 / TH;  // K runs and V squares of a thread
  constexpr int kLd = 17;              // words of a dim's 64 bytes in LDS, and one so that dims start in different banks
  __shared__ uint32_t vt[D * kLd];
  __shared__ uint32_t red[TH / 64][3];
  const int hk = blockIdx.y, tid = threadIdx.x;
  const int at_block = (int)blockIdx.x - (RAW ? 0 : 1);
  if (at_block < 0) {
    static_assert(D * kLd >= kClasses, "");
    if (hk == 0) order_tiles<TH>(a, (int*)vt, (int*)red);
    return;
  }
  const int i = seq_of_item(a, at_block);
  const Entry e_ = entry_of(a, i);
  const int c0 = e_.c0, len = e_.len, ctx = e_.ctx, row = e_.row;
  if (ctx < 0 || len <= 0) return;
  const int first = ctx >> 6, last = (ctx + len - 1) >> 6;
  const int b = first + at_block - ((c0 >> 6) + 2 * i);
  if (b < first || b > last) return;
  uint16_t* tk = a.cache.tail_k + ((int64_t)row * a.Hk + hk) * (64 * D);
  uint16_t* tv = a.cache.tail_v + ((int64_t)row * a.Hk + hk) * (64 * D);
  const uint16_t* nk = a.k + (int64_t)hk * D;
  const uint16_t* nv = a.v + (int64_t)hk * D;
  const int old = b == first ? ctx & 63 : 0;  // tokens of this block that were there
  const int64_t from = (int64_t)c0 + (int64_t)b * 64 - ctx;  // packed row of the block's key 0
  const int keys = min(64, ctx + len - b * 64);
  const int block = keys == 64 ? block_to_write(a, row, b) : -1;

  // run i: key x / (D / 8), dims 8 (x % (D / 8)) ..; square i: keys 4 (x / (D / 4)) .., dims 4 (x % (D / 4)) ..,
  // x = thread + TH i
  u32x4 kx[n];
  u32x2 vx[nsq][4];
#pragma unroll
  for (int j = 0; j < n; ++j) {
    const int x = tid + TH * j, key = x / (D / 8), dim = x % (D / 8) * 8;
    kx[j] = u32x4{0, 0, 0, 0};
    if (key < keys) kx[j] = *(const u32x4*)(key < old ? tk + key * D + dim : nk + (from + key) * a.k_stride + dim);
  }
#pragma unroll
  for (int j = 0; j < nsq; ++j) {
    const int x = tid + TH * j, key = x / (D / 4) * 4, dim = x % (D / 4) * 4;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      vx[j][e] = u32x2{0, 0};
      if (key + e >= keys) continue;
      if (key + e >= old) {
        vx[j][e] = *(const u32x2*)(nv + (from + key + e) * a.v_stride + dim);
      } else {
        const uint16_t* t = tv + dim * 64 + key + e;
        vx[j][e] = u32x2{t[0] | (uint32_t)t[64] << 16, t[128] | (uint32_t)t[192] << 16};
      }
    }
  }
  if (old) {
    u32x4* ok = (u32x4*)(a.old_k + ((int64_t)i * a.Hk + hk) * (64 * D));
    u32x4* ov = (u32x4*)(a.old_v + ((int64_t)i * a.Hk + hk) * (64 * D));
    for (int x = tid; x < 64 * D / 8; x += TH) {
      ok[x] = ((const u32x4*)tk)[x];
      ov[x] = ((const u32x4*)tv)[x];
    }
  }
  uint32_t km = 0, vm = 0, bad = 0;
#pragma unroll
  for (int j = 0; j < n; ++j) km = amax8(kx[j], km);
#pragma unroll
  for (int j = 0; j < nsq; ++j) {
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const u32x4 w = {vx[j][e][0], vx[j][e][1], vx[j][e + 1][0], vx[j][e + 1][1]};
      vm = amax8(w, vm);
      bad |= not_finite8(w);
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    km = max(km, (uint32_t)__shfl_xor((int)km, o));
    vm = max(vm, (uint32_t)__shfl_xor((int)vm, o));
  }
  bad = __any(bad != 0);
  if ((tid & 63) == 0) {
    red[tid >> 6][0] = km;
    red[tid >> 6][1] = vm;
    red[tid >> 6][2] = bad;
  }
  __syncthreads();  // also: the old tail has been read
#pragma unroll
  for (int w = 0; w < TH / 64; ++w) {
    km = max(km, red[w][0]);
    vm = max(vm, red[w][1]);
    bad |= red[w][2];
  }
  const bool missing = keys == 64 && block < 0;  // it is read as some other one, whatever that holds
  if (tid == 0) a.bad[(int64_t)at_block * a.Hk + hk] = bad | missing;

  if (keys == 64) {  // full now
    const int64_t at = (int64_t)block * a.Hk + hk;
    const int ek = scale_exponent(km), ev = scale_exponent(vm);
    if (!missing && tid == 0) {
      a.cache.k_scale[at] = pow2(ek);
      a.cache.v_scale[at] = pow2(ev);
    }
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const int x = tid + TH * j, key = x / (D / 8), dim = x % (D / 8) * 8;
      if (!missing) *(u32x2*)(a.cache.k8 + at * (64 * D) + (dim >> 6) * 4096 + key * 64 + (dim & 63)) = to_e4m3(kx[j], ek);
      if (RAW && b != last) ((u32x4*)(a.raw_k + ((int64_t)at_block * a.Hk + hk) * (64 * D)))[x] = kx[j];
    }
#pragma unroll
    for (int j = 0; j < nsq; ++j) {
      const int x = tid + TH * j, kq = x / (D / 4), dim = x % (D / 4) * 4;
      u32x2 t[4];
      transpose4(vx[j], t);
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const u32x2 w = to_e4m3(u32x4{t[e][0], t[e][1], t[e + 1][0], t[e + 1][1]}, ev);
        vt[(dim + e) * kLd + kq] = w[0];
        vt[(dim + e + 1) * kLd + kq] = w[1];
      }
      if (RAW && b != last) {
        uint16_t* rv = a.raw_v + ((int64_t)at_block * a.Hk + hk) * (64 * D);
#pragma unroll
        for (int e = 0; e < 4; ++e) *(u32x2*)(rv + (dim + e) * 64 + kq * 4) = t[e];
      }
    }
    __syncthreads();
    for (int x = tid; !missing && x < D * 4; x += TH) {
      const uint32_t* w = vt + x / 4 * kLd + x % 4 * 4;
      *(u32x4*)(a.cache.v8 + at * (64 * D) + x * 16) = u32x4{w[0], w[1], w[2], w[3]};
    }
  }
  if (b != first) return;
  // the new tail: the tokens of the last block, from registers if that is this one
  if (last != first) {
    const int64_t src = (int64_t)c0 + (int64_t)last * 64 - ctx;
    const int there = ctx + len - last * 64;
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const int x = tid + TH * j, key = x / (D / 8), dim = x % (D / 8) * 8;
      if (key < there) kx[j] = *(const u32x4*)(nk + (src + key) * a.k_stride + dim);
    }
#pragma unroll
    for (int j = 0; j < nsq; ++j) {
      const int x = tid + TH * j, vkey = x / (D / 4) * 4, vdim = x % (D / 4) * 4;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (vkey + e < there) vx[j][e] = *(const u32x2*)(nv + (src + vkey + e) * a.v_stride + vdim);
    }
  }
  const int lo = last != first ? 0 : old, hi = last != first ? ctx + len - last * 64 : keys;  // keys to write
#pragma unroll
  for (int j = 0; j < n; ++j) {
    const int x = tid + TH * j, key = x / (D / 8), dim = x % (D / 8) * 8;
    if (key >= lo && key < hi) *(u32x4*)(tk + key * D + dim) = kx[j];
  }
#pragma unroll
  for (int j = 0; j < nsq; ++j) {
    const int x = tid + TH * j, vkey = x / (D / 4) * 4, vdim = x % (D / 4) * 4;
    u32x2 t[4];
    transpose4(vx[j], t);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint16_t* to = tv + (vdim + e) * 64 + vkey;
      if (vkey >= lo && vkey + 4 <= hi) {
        *(u32x2*)to = t[e];
      } else {
#pragma unroll
        for (int y = 0; y < 4; ++y)
          if (vkey + y >= lo && vkey + y < hi) to[y] = (uint16_t)(t[e][y >> 1] >> (16 * (y & 1)));
      }
    }
  }
}

// Read-out: a work-group per (touched block, key/value head) of the packed
// output; the block's bytes once in and its bf16 once out.  A simple kernel: a
// thread moves one element of K and one of V at a time, and V's neighbours are 64 bytes
// apart, so the number of loads bounds it and not their bytes (64 x 4,000 tokens, 4 heads,
// d = 128: 786 MB in 485 us, 1.6 TB/s; 8 heads, d = 64 409 us, 2 heads, d = 256 530).
template <int D>
__global__ __launch_bounds__(256) void k_attn_cache_read(const StepArgs a, uint16_t* k_out, uint16_t* v_out) {
  const int hk = blockIdx.y;
  const int i = seq_of_item(a, blockIdx.x);
  const int c0 = cu_at(a, i), len = cu_at(a, i + 1) - c0;
  const int b = (int)blockIdx.x - ((c0 >> 6) + 2 * i);
  if (len <= 0 || b < 0 || b > ((len - 1) >> 6)) return;
  const int row = row_of(a.slot, i, a.cache.num_slots);
  const bool full = (int64_t)(b + 1) * 64 <= len;
  const int64_t at = row < 0 ? 0 : (int64_t)(full ? pool_block(a, row, b) : row) * a.Hk + hk;
  const float ks = row >= 0 && full ? a.cache.k_scale[at] : 1.f, vs = row >= 0 && full ? a.cache.v_scale[at] : 1.f;
  for (int x = threadIdx.x; x < 64 * D; x += 256) {
    const int key = x / D, dim = x % D;
    if (b * 64 + key >= len) break;
    float kf = 0.f, vf = 0.f;
    if (row >= 0 && full) {
      const int kb = a.cache.k8[at * (64 * D) + (dim >> 6) * 4096 + key * 64 + (dim & 63)];
      const int vb = a.cache.v8[at * (64 * D) + dim * 64 + key];
      kf = __builtin_amdgcn_cvt_f32_fp8(kb, 0) * ks;
      vf = __builtin_amdgcn_cvt_f32_fp8(vb, 0) * vs;
    } else if (row >= 0) {
      kf = __uint_as_float((uint32_t)a.cache.tail_k[at * (64 * D) + key * D + dim] << 16);
      vf = __uint_as_float((uint32_t)a.cache.tail_v[at * (64 * D) + dim * 64 + key] << 16);
    }
    const int64_t to = ((int64_t)(c0 + b * 64 + key) * a.Hk + hk) * D + dim;
    k_out[to] = (uint16_t)pack2(kf, 0.f);
    v_out[to] = (uint16_t)pack2(vf, 0.f);
  }
}

}  // namespace attn
