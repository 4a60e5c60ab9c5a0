// The residual's addition with the root-mean-square norm, and its gradient.
//
// h = x + residual, rounded as it is stored; r = 1 / sqrt(sum(h^2) / width + eps)
// (0 where the sum passes fp32's range, or is 0 without eps); n = h r w.  Gradient: dn = dy w, dh = d_residual_out + r (dn - h (r^2 / width)
// sum(dn h)), dw = sum over rows of dy h r: two sums over the row, sum(h^2) and
// sum(dn h), in one pass.
//
// Bound by memory: a row is read once, kept in registers and written once.  A row
// is the work of 16, 64 or 256 threads (gradient: up to 1,024), as its width
// says, so that a thread holds at most 64 columns, and so that its bits depend on
// the width alone.  The waves that share a SIMD, as their registers let them: eight or more
// where a lane has up to 16 columns (widths up to 1,024, and from 2,056 to 4,096), and in
// bf16 up to 8,192; with 32 columns seven in bf16 over a stream in fp32 (67 and 68
// registers) and four all in fp32 (97 and 100); with 64, past 8,192, four (102 and
// 124) and two (188).  The gradient is held to four.
//
// Measured (the card copies 256 MB at 5.5 TB/s, 2 GB at 5.0): 10,240 x 2,048, bf16, 32.4 us, 168 MB, 5.2 TB/s;
// 10,240 x 4,096 into 8 bits over a stream in fp32 85.5 us, 463 MB, 5.4 TB/s; one row 3.3 us (the
// call 6.0 to 7.0, of the host).  All in fp32 5,000 x 2,048 37.5 us, 164 MB, 4.4 TB/s, 1,250 x 8,192 35.8 us, 4.6; 1,200 x
// 16,384 30.4 us in bf16, 157 MB, 5.2 TB/s, 51.1 over a stream in fp32, 236 MB, 4.6, 73.8 all in fp32, 315 MB,
// 4.3.  Gradient of 10,240 x 2,048 32.0 us in two launches, 168 MB, 5.2 TB/s.
#pragma once

#include "stack_device.hpp"

namespace stack {

struct NormArgs {
  const void *x, *res, *dy;  // gradient: x is h, res is d_residual_out
  const float* w;
  void *h, *y;               // gradient: d_residual, dx
  uint8_t* y8;
  float* y_scale;
  int64_t x_stride, res_stride, dy_stride, h_stride, y_stride;
  int64_t rows;
  int width, group;
  float eps, w_add;
  float* partial;            // gradient: [work-group][width]
};

constexpr int kNormThreads = 256;

// What is read past the caches: in fp32 a lane's two loads share their lines,
// which would be fetched for each.
template <class E, bool ONCE>
constexpr bool once = ONCE && sizeof(typename E::T) == 2;


// Sum over the LANES threads of a row; `red`: 4 floats of LDS that no thread
// still reads from an earlier call.
template <int LANES>
__device__ __forceinline__ float row_sum(float x, float* red) {
  if constexpr (LANES <= 64) {
    return sum_lanes<LANES>(x);
  } else {
    x = sum_lanes<64>(x);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
  }
}

// two sums at once; red: LANES / 32 floats
template <int LANES>
__device__ __forceinline__ void row_sums(float& x, float& y, float* red) {
  constexpr int W = LANES / 64;
  x = sum_lanes<(LANES < 64 ? LANES : 64)>(x);
  y = sum_lanes<(LANES < 64 ? LANES : 64)>(y);
  if constexpr (W > 1) {
    const int wave = (threadIdx.x >> 6) % W;
    if ((threadIdx.x & 63) == 0) {
      red[wave] = x;
      red[W + wave] = y;
    }
    __syncthreads();
    x = red[0];
    y = red[W];
#pragma unroll
    for (int i = 1; i < W; ++i) {
      x += red[i];
      y += red[W + i];
    }
  }
}

// r of a row's sum of squares.  A row of zeros without eps: 0, so that its norm is.
__device__ __forceinline__ float root(float ss, float inv_width, float eps) {
  const float mean = ss * inv_width + eps;
  return mean == 0.f ? 0.f : 1.f / __builtin_sqrtf(mean);
}

template <int LANES>
__device__ __forceinline__ float row_max(float x, float* red) {
  x = max_16(x);
  if constexpr (LANES > 16) x = max_groups(x);
  if constexpr (LANES > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
    __syncthreads();
    x = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  }
  return x;
}

__device__ __forceinline__ float dot4(f32x4 a, f32x4 b, float s) {
#pragma unroll
  for (int i = 0; i < 4; ++i) s = __builtin_fmaf(a[i], b[i], s);
  return s;
}

__device__ __forceinline__ float amax8(const F8& f) {
  float m = max3(__builtin_fabsf(f.a[0]), __builtin_fabsf(f.a[1]), __builtin_fabsf(f.a[2]));
  m = max3(m, __builtin_fabsf(f.a[3]), __builtin_fabsf(f.b[0]));
  m = max3(m, __builtin_fabsf(f.b[1]), __builtin_fabsf(f.b[2]));
  return fmaxf(m, __builtin_fabsf(f.b[3]));
}

// Quotients by one s > 0, correctly rounded.  (A product with 1 / s has a rounding of
// its own: beside a border between two codes the other one would come out.)  In
// units of a power of two, so that remainders are exact: a product, a correction
// that leaves less than a step, and one that rounds as the quotient does (Markstein's
// theorem; inv is 1 / s rounded once).  By an infinity 0.  10,240 x 2,048 into 8 bits
// alone, us, with products / this / the compiler's division: 28.6 / 29.6 / 30.7.
struct Divisor {
  float s, inv;
  int shift;
  __device__ __forceinline__ explicit Divisor(float x) {
    const bool none = x > 0x1.fffffep127f;
    s = none ? 0.f : __builtin_amdgcn_frexp_mantf(x);
    inv = none ? 0.f : 1.f / s;
    shift = -__builtin_amdgcn_frexp_expf(x);
  }
  __device__ __forceinline__ float operator()(float n) const {
    n = __builtin_amdgcn_ldexpf(n, shift);
    float q = n * inv;
    q = __builtin_fmaf(__builtin_fmaf(-s, q, n), inv, q);
    return __builtin_fmaf(__builtin_fmaf(-s, q, n), inv, q);
  }
};

__device__ __forceinline__ u32x2 to_e4m3(const F8& f, const Divisor& by) {
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(by(f.a[0]), by(f.a[1]), 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(by(f.a[2]), by(f.a[3]), lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(by(f.b[0]), by(f.b[1]), 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(by(f.b[2]), by(f.b[3]), hi, true);
  return u32x2{(uint32_t)lo, (uint32_t)hi};
}

// A row to LANES threads, NV vectors of eight columns to a thread, the vectors
// LANES * 8 columns apart.
template <class X, class R, int LANES, int NV, bool ONCE>
__global__ __launch_bounds__(kNormThreads) void k_stack_add_norm(const NormArgs a) {
  __shared__ float red[8];
  const int l = threadIdx.x % LANES;
  const int64_t row = (int64_t)blockIdx.x * (kNormThreads / LANES) + threadIdx.x / LANES;
  if (row >= a.rows) return;  // with LANES = 256 there is none
  const typename X::T* x = (const typename X::T*)a.x + row * a.x_stride;
  const typename R::T* res = (const typename R::T*)a.res + row * a.res_stride;
  typename R::T* h_out = (typename R::T*)a.h + row * a.h_stride;
  F8 h[NV];
  typename X::RAW xr[NV];
  typename R::RAW rr[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * LANES + l) * 8;
    if (c < a.width) {
      xr[j] = X::template load<false, once<X, ONCE>>(x + c);
      if (a.res) rr[j] = R::template load<false, once<R, ONCE>>(res + c);
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * LANES + l) * 8;
    h[j] = F8{{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    if (c < a.width) {
      h[j] = X::wide(xr[j]);
      if (a.res) {
        const F8 f = R::wide(rr[j]);
        h[j].a += f.a;
        h[j].b += f.b;
      }
      const typename R::RAW n = R::narrow(h[j]);
      h[j] = R::wide(n);
      if (a.h) R::store(h_out + c, n);
      ss = dot4(h[j].b, h[j].b, dot4(h[j].a, h[j].a, ss));
    }
  }
  ss = row_sum<LANES>(ss, red);
  const float r = root(ss, 1.f / (float)a.width, a.eps);
  float most = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * LANES + l) * 8;
    if (c >= a.width) continue;
    const f32x4 w1 = *(const f32x4*)(a.w + c) + a.w_add, w2 = *(const f32x4*)(a.w + c + 4) + a.w_add;
    h[j].a = h[j].a * r * w1;
    h[j].b = h[j].b * r * w2;
    if (a.y) X::store((typename X::T*)a.y + row * a.y_stride + c, X::narrow(h[j]));
    if (a.y8 && a.group == 0) most = fmaxf(most, amax8(h[j]));
  }
  if (!a.y8) return;
  const float least = 0x1p-100f;
  float scale = 0.f;
  if (a.group == 0) {
    scale = fmaxf(row_max<LANES>(most, red + 4), least) / 448.f;
    if (l == 0) a.y_scale[row] = scale;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * LANES + l) * 8;
    if (c >= a.width) continue;  // sixteen lanes of a group together
    if (a.group) {
      scale = fmaxf(max_16(amax8(h[j])), least) / 448.f;
      if ((l & 15) == 0) a.y_scale[row * (a.width / 128) + c / 128] = scale;
    }
    *(u32x2*)(a.y8 + row * a.width + c) = to_e4m3(h[j], Divisor(scale));
  }
}

// Gradient.  Work-groups go over the rows in steps of the grid; a thread keeps
// dw of its columns in registers for all of its rows, so dw costs one partial
// sum of a row's width per work-group.  The weights wait in LDS: with them in
// registers and a wave to a row of 2,048 (32 columns to a lane, 238 registers, two
// waves to a SIMD) 10,240 rows took 38.6 us, so 35.3; reading past the caches 32.1.
// Threads of a work-group: 512, or a row's 1,024.
template <int LANES>
constexpr int kNormBwdThreads = LANES == 1024 ? 1024 : 512;

template <class X, class R, int LANES, int NV, bool ONCE>
__global__ __launch_bounds__(kNormBwdThreads<LANES>, 4) void k_stack_add_norm_bwd(const NormArgs a) {
  constexpr int kT = kNormBwdThreads<LANES>, G = kT / LANES;
  __shared__ float red[2][G][LANES < 256 ? 1 : LANES / 32];
  __shared__ f32x4 part[G > 1 ? 2 * kT : 1];
  const int l = threadIdx.x % LANES, sub = threadIdx.x / LANES;
  __shared__ f32x4 wl[2 * LANES * NV];
  F8 g[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) g[j] = F8{{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  for (int i = threadIdx.x; i < a.width / 4; i += kT) wl[i] = *(const f32x4*)(a.w + 4 * i) + a.w_add;
  __syncthreads();
  const auto weight = [&](int c) { return F8{wl[c / 4], wl[c / 4 + 1]}; };
  const float inv = 1.f / (float)a.width;
  int turn = 0;
  struct Raw {
    typename R::RAW h[NV], d[NV];
    typename X::RAW y[NV];
  };
  const auto fetch = [&](Raw& q, int64_t row) {
    const typename R::T* hp = (const typename R::T*)a.x + row * a.x_stride;
    const typename X::T* yp = (const typename X::T*)a.dy + row * a.dy_stride;
    const typename R::T* dp = (const typename R::T*)a.res + row * a.res_stride;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * LANES + l) * 8;
      if (row < a.rows && c < a.width) {
        q.h[j] = R::template load<false, once<R, ONCE>>(hp + c);
        q.y[j] = X::template load<false, once<X, ONCE>>(yp + c);
        if (a.res) q.d[j] = R::template load<false, once<R, ONCE>>(dp + c);
      }
    }
  };
  const auto put = [&](int64_t row, int c, const F8& d) {
    if (a.y) X::store((typename X::T*)a.y + row * a.y_stride + c, X::narrow(d));
    if (a.h) R::store((typename R::T*)a.h + row * a.h_stride + c, R::narrow(d));
  };
  // The next row is asked for before this one is summed, where a row takes a
  // work-group or half of one, so that few are under way, and it fits 24 registers:
  // us with / without, bf16, 1,174 x 8,184 20.9 / 22.3, 2,500 x 8,192 33.8 / 36.9, 1,200 x 16,384 36.6 / 40.3,
  // 5,120 x 4,096 33.0 / 34.0, over a stream in fp32 2,500 x 8,192 65.9 / 66.4; but 3,000 x 2,048 13.6 /
  // 13.1, and all in fp32 2,500 x 8,192 69.2 / 67.0.
  constexpr bool AHEAD = LANES * NV > 256 && sizeof(typename X::T) == 2 && sizeof(Raw) <= 96;
  const int64_t step = (int64_t)gridDim.x * G;
  Raw next;
  if (AHEAD) fetch(next, (int64_t)blockIdx.x * G + sub);
  for (int64_t first = (int64_t)blockIdx.x * G; first < a.rows; first += step, turn ^= 1) {
    const int64_t row = first + sub;
    int width = row < a.rows ? a.width : 0;  // no row: no columns
    Raw q;
    if (AHEAD) {
      q = next;
      fetch(next, row + step);
    } else {
      fetch(q, row);
    }
    float ss = 0.f, hx = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * LANES + l) * 8;
      if (c >= width) continue;
      const F8 h = R::wide(q.h[j]), y = X::wide(q.y[j]), w = weight(c);
      ss = dot4(h.b, h.b, dot4(h.a, h.a, ss));
      hx = dot4(y.b * w.b, h.b, dot4(y.a * w.a, h.a, hx));
    }
    row_sums<LANES>(ss, hx, red[turn][sub]);
    const float r = root(ss, inv, a.eps);
    const float m = hx * r * r * inv;
    if (r == 0.f) {  // n is 0 whatever h is, and nothing comes back through it
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * LANES + l) * 8;
        if (c >= width) continue;
        F8 d = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        if (a.res) d = R::wide(q.d[j]);
        put(row, c, d);
      }
      width = 0;  // done
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * LANES + l) * 8;
      if (c >= width) continue;
      const F8 h = R::wide(q.h[j]), y = X::wide(q.y[j]), w = weight(c);
      F8 d = {r * (y.a * w.a - h.a * m), r * (y.b * w.b - h.b * m)};
      g[j].a += y.a * (h.a * r);
      g[j].b += y.b * (h.b * r);
      if (a.res) {
        const F8 f = R::wide(q.d[j]);
        d.a += f.a;
        d.b += f.b;
      }
      put(row, c, d);
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * LANES + l) * 8;
    if constexpr (G > 1) {  // the work-group's rows, one after the other
      __syncthreads();
      part[threadIdx.x] = g[j].a;
      part[kT + threadIdx.x] = g[j].b;
      __syncthreads();
      if (sub == 0) {
#pragma unroll
        for (int i = 1; i < G; ++i) {
          g[j].a += part[i * LANES + l];
          g[j].b += part[kT + i * LANES + l];
        }
      }
    }
    if (sub == 0 && c < a.width) {
      float* to = a.partial + (int64_t)blockIdx.x * a.width + c;
      *(f32x4*)to = g[j].a;
      *(f32x4*)(to + 4) = g[j].b;
    }
  }
}

// dw = the partial sums added up: 32 columns per work-group, 32 runs of
// partials each, then the runs in order.
__global__ __launch_bounds__(1024) void k_stack_norm_dw(const float* partial, int n, int width, float* dw) {
  __shared__ float red[32][33];
  const int col = threadIdx.x & 31, run = threadIdx.x >> 5, at = blockIdx.x * 32 + col;
  float t = 0.f;
  if (at < width) {
#pragma unroll 8
    for (int i = run; i < n; i += 32) t += partial[(int64_t)i * width + at];
  }
  red[run][col] = t;
  __syncthreads();
  if (run == 0 && at < width) {
    for (int i = 1; i < 32; ++i) t += red[i][col];
    dw[at] = t;
  }
}

}  // namespace stack
