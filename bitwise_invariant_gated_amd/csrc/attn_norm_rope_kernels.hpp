// Norm of every head's q and k with the position rotation, and its gradient.
//
// x -> n = x r w, r = rsqrt(mean(x^2) + eps), then the pair (n1, n2) of the
// first rd dims -> (n1 c - n2 s, n2 c + n1 s).  Gradient: dn is the incoming
// gradient rotated back (s -> -s), dw = sum dn x r and
// dx = r (dn w - x r (r / d) sum(dn w x)), from the two sums sum(x^2) and
// sum(dn w x) of one pass over the row.
//
// Bound by memory: a row is read once and written once, all else stays in
// registers.  A row takes d / 8 lanes.  A lane holds two runs of four
// elements, four apart in the pairing: dims 4l and rd/2 + 4l of a rotated
// head, so that both members of a pair meet in one lane and no element
// crosses lanes; the runs are 8 bytes (bf16) and neighbouring lanes'
// runs are contiguous.  Dims past rd, and adjacent pairs, take 8 dims in a row.
//
// Measured with inputs that no cache holds, 10,240 tokens, 32 heads in all, d = 128, bf16: 37 us,
// 173 MB, 4.7 TB/s; the gradient 59 us in two launches, 257 MB, 4.3 TB/s (a copy moves 4.65).
#pragma once

#include "attn_device.hpp"

namespace attn {

struct NormRopeArgs {
  const void *x[2], *dy[2];  // q, k
  void* out[2];
  const float* w[2];
  int64_t x_stride[2], dy_stride[2], out_stride[2];
  int heads[2];
  int64_t rows[2];
  const float* cos_sin;
  const int32_t* positions;
  int rd, interleaved, num_positions;
  float eps, w_add;
  int groups[2];    // forward: work-groups of q and of k
  float* partial;   // gradient: [work-group][2][d]
};

constexpr int kNormThreads = 256;

// Where a lane's eight elements sit in a row, and its pairs' place in the table.
struct RowLane {
  int o1, o2, c;  // offsets of the two runs; first pair
  bool rot, adj;
};

template <int D>
__device__ __forceinline__ RowLane row_lane(int l, int rd, int interleaved) {
  RowLane p;
  p.rot = l < rd / 8;
  p.adj = interleaved != 0;
  if (p.rot && !p.adj) {
    p.o1 = 4 * l;
    p.o2 = rd / 2 + 4 * l;
  } else {
    p.o1 = 8 * l;
    p.o2 = 8 * l + 4;
  }
  p.c = 4 * l;
  return p;
}

// cosines and sines of the lane's four pairs at the token's position
__device__ __forceinline__ void load_rotation(const NormRopeArgs& a, const RowLane& p, int64_t token, f32x4& c, f32x4& s) {
  c = f32x4{1.f, 1.f, 1.f, 1.f};
  s = f32x4{0.f, 0.f, 0.f, 0.f};
  if (!p.rot) return;
  const int pos = a.positions[token];
  if (pos >= 0 && pos < a.num_positions) {
    const float* row = a.cos_sin + (int64_t)pos * a.rd + p.c;
    c = *(const f32x4*)row;
    s = *(const f32x4*)(row + a.rd / 2);
  } else {
    const float nan = __uint_as_float(0x7fc00000u);
    c = f32x4{nan, nan, nan, nan};
    s = c;
  }
}

// (x1, x2) -> the rotated runs; back: by the opposite angle
__device__ __forceinline__ void rotate(const RowLane& p, f32x4& x1, f32x4& x2, f32x4 c, f32x4 s, bool back) {
  if (!p.rot) return;
  if (back) s = -s;
  const f32x4 a = p.adj ? f32x4{x1[0], x1[2], x2[0], x2[2]} : x1;
  const f32x4 b = p.adj ? f32x4{x1[1], x1[3], x2[1], x2[3]} : x2;
  f32x4 u, v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    u[i] = __builtin_fmaf(a[i], c[i], -(b[i] * s[i]));
    v[i] = __builtin_fmaf(b[i], c[i], a[i] * s[i]);
  }
  x1 = p.adj ? f32x4{u[0], v[0], u[1], v[1]} : u;
  x2 = p.adj ? f32x4{u[2], v[2], u[3], v[3]} : v;
}

__device__ __forceinline__ float dot8(f32x4 a, f32x4 b, f32x4 c, f32x4 d) {
  float s0 = a[0] * c[0], s1 = b[0] * d[0];
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    s0 = __builtin_fmaf(a[i], c[i], s0);
    s1 = __builtin_fmaf(b[i], d[i], s1);
  }
  return s0 + s1;
}

// U rows per lane group: their loads are all issued before the first is used.
template <class E, int D, int U, bool STREAM>
__global__ __launch_bounds__(kNormThreads) void k_attn_norm_rope(const NormRopeArgs a) {
  typedef typename E::T T;
  constexpr int L = D / 8, R = kNormThreads / L;
  const int which = (int)blockIdx.x >= a.groups[0];
  const int64_t group = (int64_t)blockIdx.x - (which ? a.groups[0] : 0);
  const RowLane p = row_lane<D>(threadIdx.x % L, a.rd, a.interleaved);
  const int heads = a.heads[which];
  const T* x = (const T*)a.x[which];
  T* out = (T*)a.out[which];
  f32x4 x1[U], x2[U], c[U], s[U];
  int64_t at[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = (group * U + u) * R + threadIdx.x / L;
    at[u] = -1;
    if (row < a.rows[which]) {
      const uint32_t token = (uint32_t)row / (uint32_t)heads, head = (uint32_t)row - token * heads;
      const T* r = x + token * a.x_stride[which] + head * D;
      x1[u] = E::load4(r + p.o1);
      x2[u] = E::load4(r + p.o2);
      load_rotation(a, p, token, c[u], s[u]);
      at[u] = token * a.out_stride[which] + head * D;
    }
  }
  const f32x4 w1 = *(const f32x4*)(a.w[which] + p.o1) + a.w_add, w2 = *(const f32x4*)(a.w[which] + p.o2) + a.w_add;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (at[u] < 0) continue;
    const float ss = sum_over_lanes<L>(dot8(x1[u], x2[u], x1[u], x2[u]));
    const float r = 1.f / __builtin_sqrtf(ss * (1.f / D) + a.eps);
    x1[u] = x1[u] * r * w1;
    x2[u] = x2[u] * r * w2;
    rotate(p, x1[u], x2[u], c[u], s[u], false);
    E::template store4<STREAM>(out + at[u] + p.o1, x1[u]);
    E::template store4<STREAM>(out + at[u] + p.o2, x2[u]);
  }
}

// Gradient.  Work-groups go over the rows of q, then over those of k, in
// steps of the grid; a lane keeps dw of its eight dims in registers for all
// of its rows, so dw costs one partial sum of 2 d floats per work-group.
template <class E, int D, bool STREAM>
__global__ __launch_bounds__(kNormThreads) void k_attn_norm_rope_bwd(const NormRopeArgs a) {
  typedef typename E::T T;
  constexpr int L = D / 8, R = kNormThreads / L;
  __shared__ f32x4 red[2 * kNormThreads];
  const int l = threadIdx.x % L, sub = threadIdx.x / L;
  const RowLane p = row_lane<D>(l, a.rd, a.interleaved);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const int heads = a.heads[which];
    const f32x4 w1 = *(const f32x4*)(a.w[which] + p.o1) + a.w_add, w2 = *(const f32x4*)(a.w[which] + p.o2) + a.w_add;
    f32x4 g1 = {0.f, 0.f, 0.f, 0.f}, g2 = g1;
    for (int64_t row = (int64_t)blockIdx.x * R + sub; row < a.rows[which]; row += (int64_t)gridDim.x * R) {
      const uint32_t token = (uint32_t)row / (uint32_t)heads, head = (uint32_t)row - token * heads;
      const T* xr = (const T*)a.x[which] + token * a.x_stride[which] + head * D;
      const T* yr = (const T*)a.dy[which] + token * a.dy_stride[which] + head * D;
      const f32x4 x1 = E::load4(xr + p.o1), x2 = E::load4(xr + p.o2);
      f32x4 y1 = E::load4(yr + p.o1), y2 = E::load4(yr + p.o2), c, s;
      load_rotation(a, p, token, c, s);
      rotate(p, y1, y2, c, s, true);
      const f32x4 h1 = y1 * w1, h2 = y2 * w2;
      const float ss = sum_over_lanes<L>(dot8(x1, x2, x1, x2));
      const float hx = sum_over_lanes<L>(dot8(h1, h2, x1, x2));
      const float r = 1.f / __builtin_sqrtf(ss * (1.f / D) + a.eps);
      const float m = hx * r * r * (1.f / D);
      T* o = (T*)a.out[which] + token * a.out_stride[which] + head * D;
      E::template store4<STREAM>(o + p.o1, r * (h1 - x1 * m));
      E::template store4<STREAM>(o + p.o2, r * (h2 - x2 * m));
      g1 += y1 * (x1 * r);
      g2 += y2 * (x2 * r);
    }
    // the work-group's rows, lane group by lane group
    __syncthreads();
    red[threadIdx.x] = g1;
    red[kNormThreads + threadIdx.x] = g2;
    __syncthreads();
    if (threadIdx.x < 2 * L) {
      const int half = threadIdx.x / L, ll = threadIdx.x % L;
      f32x4 t = red[half * kNormThreads + ll];
#pragma unroll 4
      for (int i = 1; i < R; ++i) t += red[half * kNormThreads + i * L + ll];
      const RowLane pp = row_lane<D>(ll, a.rd, a.interleaved);
      *(f32x4*)(a.partial + ((int64_t)blockIdx.x * 2 + which) * D + (half ? pp.o2 : pp.o1)) = t;
    }
  }
}

// dw = the partial sums added up: 32 columns per work-group, 32 runs of
// partials each, then the runs in order.
__global__ __launch_bounds__(1024) void k_attn_norm_rope_dw(const float* partial, int n, int D, float* dw_q, float* dw_k) {
  __shared__ float red[32][33];
  const int col = threadIdx.x & 31, run = threadIdx.x >> 5, at = blockIdx.x * 32 + col;
  float t = 0.f;
#pragma unroll 8
  for (int i = run; i < n; i += 32) t += partial[(int64_t)i * 2 * D + at];
  red[run][col] = t;
  __syncthreads();
  if (run == 0) {
    for (int i = 1; i < 32; ++i) t += red[i][col];
    if (at < D)
      dw_q[at] = t;
    else
      dw_k[at - D] = t;
  }
}

}  // namespace attn
