// What a stack needs around its layers, for gfx950: host side and the C ABI
// (gdn_stack.h).  The kernels live in stack_norm_kernels.hpp and
// stack_logits_kernels.hpp.
//
// Per call, on the caller's stream:
//   add_norm        k_stack_add_norm; its gradient k_stack_add_norm_bwd and
//                   k_stack_norm_dw
//   logprobs        k_stack_parts, k_stack_logprobs (rows of up to 2,048 columns:
//                   the latter alone); gradient k_stack_logprobs_bwd
//   distill         k_stack_parts, k_stack_distill (the same); gradient
//                   k_stack_distill_bwd
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <string>

#include "../../include/gdn_stack.h"
#include "stack_logits_kernels.hpp"
#include "stack_norm_kernels.hpp"

std::string& gdn_last_error_text();  // gdn_cpr.hip

namespace {

using namespace stack;

gdn_status fail(gdn_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  gdn_last_error_text() = buf;
  return st;
}

gdn_status done() {
  gdn_last_error_text().clear();
  return GDN_OK;
}

gdn_status launch_status(const char* fn) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(GDN_ERR_HIP, "%s: kernel launch failed: %s", fn, hipGetErrorString(e));
  return done();
}

size_t align_up(size_t x) { return (x + 255) & ~(size_t)255; }

#define CHECK_ALIGN(p, name, to)                                                                           \
  do {                                                                                                     \
    if ((uintptr_t)(p) % (to) != 0) return fail(GDN_ERR_INVALID_ARG, "%s: %s is not %d-byte aligned", fn, name, (int)(to)); \
  } while (0)

#define CHECK_PTR_TO(p, name, to)                                           \
  do {                                                                      \
    if (!(p)) return fail(GDN_ERR_INVALID_ARG, "%s: %s is NULL", fn, name); \
    CHECK_ALIGN(p, name, to);                                               \
  } while (0)

#define CHECK_PTR(p, name) CHECK_PTR_TO(p, name, 16)

#define CHECK(call)               \
  do {                            \
    const gdn_status r_ = (call); \
    if (r_ != GDN_OK) return r_;  \
  } while (0)

gdn_status check_dtype(const char* fn, const char* name, int32_t t) {
  if (t != GDN_DTYPE_F32 && t != GDN_DTYPE_BF16)
    return fail(GDN_ERR_UNSUPPORTED, "%s: %s must be GDN_DTYPE_F32 or GDN_DTYPE_BF16", fn, name);
  return GDN_OK;
}

gdn_status check_rows(const char* fn, int64_t rows) {
  if (rows < 0) return fail(GDN_ERR_INVALID_ARG, "%s: negative size", fn);
  if (rows > INT32_MAX / 2) return fail(GDN_ERR_UNSUPPORTED, "%s: too many rows", fn);
  return GDN_OK;
}

// A row stride as given, resolved: 0 is `row` elements.
gdn_status check_stride(const char* fn, const char* name, int64_t given, int64_t row, int unit, int64_t* out) {
  *out = given ? given : row;
  if (*out < row || *out % unit != 0 || *out > INT64_MAX / INT32_MAX) {
    if (unit > 1)
      return fail(GDN_ERR_INVALID_ARG, "%s: %s must be 0 or a multiple of %d of at least %lld", fn, name, unit, (long long)row);
    return fail(GDN_ERR_INVALID_ARG, "%s: %s must be 0 or at least %lld", fn, name, (long long)row);
  }
  return GDN_OK;
}

gdn_status check_workspace(const char* fn, void* ws, size_t given, size_t need) {
  if (!ws || given < need)
    return fail(GDN_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, need, ws ? given : (size_t)0);
  CHECK_ALIGN(ws, "workspace", 16);
  return GDN_OK;
}

// an output over an input has to lie exactly on it
gdn_status check_in_place(const char* fn, const void* out, int64_t out_stride, int32_t out_type, const void* in,
                          int64_t in_stride, int32_t in_type) {
  if (out && out == in && (out_stride != in_stride || out_type != in_type))
    return fail(GDN_ERR_INVALID_ARG, "%s: in place needs equal types and strides", fn);
  return GDN_OK;
}

// ---------------------------------------------------------------------------
// norm

// A launch counts its threads in 32 bits.
constexpr int64_t kMostThreads = (int64_t(1) << 32) - 4096;

gdn_status check_norm(const char* fn, const gdn_norm_shape* s, int64_t rows) {
  if (!s) return fail(GDN_ERR_INVALID_ARG, "%s: shape is NULL", fn);
  if (s->width < 8 || s->width > GDN_STACK_MAX_WIDTH || s->width % 8 != 0)
    return fail(GDN_ERR_UNSUPPORTED, "%s: width must be a multiple of 8 in [8, %d]", fn, GDN_STACK_MAX_WIDTH);
  CHECK(check_dtype(fn, "dtype", s->dtype));
  CHECK(check_dtype(fn, "residual_dtype", s->residual_dtype));
  if (s->residual_dtype != s->dtype && s->residual_dtype != GDN_DTYPE_F32)
    return fail(GDN_ERR_UNSUPPORTED, "%s: residual_dtype must be dtype or GDN_DTYPE_F32", fn);
  if (s->group != -1 && s->group != 0 && s->group != GDN_STACK_GROUP)
    return fail(GDN_ERR_UNSUPPORTED, "%s: group must be -1, 0 or %d", fn, GDN_STACK_GROUP);
  if (s->group > 0 && s->width % s->group != 0)
    return fail(GDN_ERR_UNSUPPORTED, "%s: group must divide width", fn);
  if (!(s->eps >= 0.f) || std::isinf(s->eps)) return fail(GDN_ERR_INVALID_ARG, "%s: eps must be finite and not negative", fn);
  CHECK(check_rows(fn, rows));
  if (rows * (s->width <= 128 ? 16 : s->width <= 2048 ? 64 : 256) > kMostThreads)
    return fail(GDN_ERR_UNSUPPORTED, "%s: too many rows", fn);
  return GDN_OK;
}

// Calls that move more than this read past the caches what is read for the last
// time (x, the residual, the gradients that come in, logits), us past / into them:
//   norm      10,240 x 2,048 (168 MB) 32.4 / 39.3   6,144 (101 MB) 17.7 / 21.8   4,096 (67 MB) 12.2 / 11.8
//   gradient                          32.0 / 36.5                  22.1 / 23.9                 17.0 / 15.7
//   parts     2,048 x 131,072 (537 MB), divergence 84.9 / 95.3; with entropy 4,096 156 / 177; fp32 1,024 87 / 92
// Of rows that end inside a part the last one is read through the caches, and so are rows
// of one part, whatever the call's size: past them, 60,000 x 900 51.2 / 52.2 in bf16 but 51.4 / 49.5 in fp32,
// 60,000 x 2,000 63.2 / 64.8 and 85.9 / 82.5, its divergence in fp32 94.7 / 82.5.
// Outputs of the norm stay in the caches, as a product reads them next: stored past
// them, 10,240 x 2,048 would take 26 us, but norm, product and norm 139 and not 123.
// Gradients of logits do not fit and go past them too, 2,048 x 131,072 170 / 184, fp32
// 513 x 50,001 (103 MB) 37.6 / 41.6, the divergence's 38.7 / 42.3; with the product that reads them, of width 1,024,
// 1,024 rows (268 MB) 768 / 783, 4,096 1,556 / 1,609, but 256 rows (67 MB) 459 / 457.
constexpr int64_t kOnceFrom = int64_t(96) << 20;

// Work-groups of the gradient's row pass, each with a partial dw: enough to fill
// the card, few enough that adding them up is short (us with 256 / 512 / 1,024 of them:
// 10,240 x 2,048 37.9 / 35.3 / 38.3, 5,120 x 4,096 39.1 / 37.3 / 39.5, 2,500 x 8,192 38.5 / 41.6 / 47.4,
// 1,200 x 16,384 42.5 / 48.6 / 60.4, all before rows were read ahead).
int norm_bwd_groups(const gdn_norm_shape& s, int64_t rows) {
  const int64_t per = s.width <= 128 ? 32 : s.width <= 1024 ? 8 : s.width <= 4096 ? 2 : 1;
  return (int)std::min<int64_t>(s.width <= 4096 ? 512 : 256, (rows + per - 1) / per);
}

template <class X, class R>
bool norm_reads_once(const NormArgs& a) {
  const int64_t bytes = sizeof(typename X::T) * ((a.y ? 1 : 0) + 1) +
                        sizeof(typename R::T) * ((a.res ? 1 : 0) + (a.h ? 1 : 0) + (a.dy ? 1 : 0));
  return a.rows * a.width * bytes >= kOnceFrom;
}

template <class X, class R, int LANES, int NV>
struct NormFn {
  static void forward(const NormArgs& a, hipStream_t st) {
    const int64_t per = kNormThreads / LANES;
    const dim3 grid((unsigned)((a.rows + per - 1) / per)), wg(kNormThreads);
    if (norm_reads_once<X, R>(a))
      hipLaunchKernelGGL((k_stack_add_norm<X, R, LANES, NV, true>), grid, wg, 0, st, a);
    else
      hipLaunchKernelGGL((k_stack_add_norm<X, R, LANES, NV, false>), grid, wg, 0, st, a);
  }
};

template <class X, class R, int LANES, int NV>
struct NormBwdFn {
  static void backward(const NormArgs& a, int groups, hipStream_t st) {
    if (norm_reads_once<X, R>(a))
      hipLaunchKernelGGL((k_stack_add_norm_bwd<X, R, LANES, NV, true>), dim3(groups), dim3(kNormBwdThreads<LANES>), 0, st, a);
    else
      hipLaunchKernelGGL((k_stack_add_norm_bwd<X, R, LANES, NV, false>), dim3(groups), dim3(kNormBwdThreads<LANES>), 0, st, a);
  }
};

#define GDN_STACK_NORM_BWD_WIDTH(X, R, width, call)           \
  do {                                                        \
    if ((width) <= 128) NormBwdFn<X, R, 16, 1>::call;            \
    else if ((width) <= 512) NormBwdFn<X, R, 64, 1>::call;       \
    else if ((width) <= 1024) NormBwdFn<X, R, 64, 2>::call;      \
    else if ((width) <= 2048) NormBwdFn<X, R, 256, 1>::call;     \
    else if ((width) <= 4096) NormBwdFn<X, R, 256, 2>::call;     \
    else if ((width) <= 8192) NormBwdFn<X, R, 1024, 1>::call;    \
    else NormBwdFn<X, R, 1024, 2>::call;                         \
  } while (0)

// A row's threads follow from its width alone, so that its bits do.
#define GDN_STACK_NORM_WIDTH(X, R, width, call)               \
  do {                                                        \
    if ((width) <= 128) NormFn<X, R, 16, 1>::call;            \
    else if ((width) <= 512) NormFn<X, R, 64, 1>::call;       \
    else if ((width) <= 1024) NormFn<X, R, 64, 2>::call;      \
    else if ((width) <= 2048) NormFn<X, R, 64, 4>::call;      \
    else if ((width) <= 4096) NormFn<X, R, 256, 2>::call;     \
    else if ((width) <= 8192) NormFn<X, R, 256, 4>::call;     \
    else NormFn<X, R, 256, 8>::call;                          \
  } while (0)

#define GDN_STACK_NORM(WIDTH, shape, call)                                                                  \
  do {                                                                                               \
    if ((shape).dtype == GDN_DTYPE_F32) WIDTH(F32, F32, (shape).width, call);         \
    else if ((shape).residual_dtype == GDN_DTYPE_F32) WIDTH(B16, F32, (shape).width, call); \
    else WIDTH(B16, B16, (shape).width, call);                                        \
  } while (0)

}  // namespace

extern "C" size_t gdn_stack_norm_workspace_size(const gdn_norm_shape* shape, int64_t num_rows) {
  if (check_norm("gdn_stack_norm_workspace_size", shape, num_rows) != GDN_OK) return 0;
  return align_up((size_t)norm_bwd_groups(*shape, num_rows) * shape->width * sizeof(float) + 1);
}

extern "C" gdn_status gdn_stack_add_norm(const gdn_norm_shape* shape, int64_t num_rows, const void* x,
                                         int64_t x_stride, const void* residual, int64_t residual_stride,
                                         const float* w, void* residual_out, int64_t residual_out_stride, void* y,
                                         int64_t y_stride, uint8_t* y8, float* y_scale, void* stream) {
  const char* fn = "gdn_stack_add_norm";
  CHECK(check_norm(fn, shape, num_rows));
  NormArgs a{};
  const int W = shape->width;
  CHECK(check_stride(fn, "x_stride", x_stride, W, 8, &a.x_stride));
  CHECK(check_stride(fn, "residual_stride", residual_stride, W, 8, &a.res_stride));
  CHECK(check_stride(fn, "residual_out_stride", residual_out_stride, W, 8, &a.h_stride));
  CHECK(check_stride(fn, "y_stride", y_stride, W, 8, &a.y_stride));
  CHECK_PTR(w, "w");
  if (num_rows == 0) return done();
  CHECK_PTR(x, "x");
  CHECK_ALIGN(residual, "residual", 16);
  CHECK_ALIGN(residual_out, "residual_out", 16);
  CHECK_ALIGN(y, "y", 16);
  CHECK_ALIGN(y8, "y8", 16);
  CHECK_ALIGN(y_scale, "y_scale", 16);
  if (!y && !y8) return fail(GDN_ERR_INVALID_ARG, "%s: y and y8 are both NULL", fn);
  if (!y8 != !y_scale) return fail(GDN_ERR_INVALID_ARG, "%s: y8 and y_scale go together", fn);
  if (y8 && shape->group < 0) return fail(GDN_ERR_INVALID_ARG, "%s: y8 needs a group", fn);
  if (residual_out && y == residual_out) return fail(GDN_ERR_INVALID_ARG, "%s: y is residual_out", fn);
  const int32_t dt = shape->dtype, rdt = shape->residual_dtype;
  CHECK(check_in_place(fn, residual_out, a.h_stride, rdt, x, a.x_stride, dt));
  CHECK(check_in_place(fn, residual_out, a.h_stride, rdt, residual, a.res_stride, rdt));
  CHECK(check_in_place(fn, y, a.y_stride, dt, x, a.x_stride, dt));
  CHECK(check_in_place(fn, y, a.y_stride, dt, residual, a.res_stride, rdt));
  a.x = x;
  a.res = residual;
  a.w = w;
  a.h = residual_out;
  a.y = y;
  a.y8 = y8;
  a.y_scale = y_scale;
  a.rows = num_rows;
  a.width = W;
  a.group = shape->group;
  a.eps = shape->eps;
  a.w_add = shape->zero_centered ? 1.f : 0.f;
  GDN_STACK_NORM(GDN_STACK_NORM_WIDTH, *shape, forward(a, (hipStream_t)stream));
  return launch_status(fn);
}

extern "C" gdn_status gdn_stack_add_norm_bwd(const gdn_norm_shape* shape, int64_t num_rows, const void* h,
                                             int64_t h_stride, const float* w, const void* dy, int64_t dy_stride,
                                             const void* d_residual_out, int64_t d_residual_out_stride, void* dx,
                                             int64_t dx_stride, void* d_residual, int64_t d_residual_stride,
                                             float* dw, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "gdn_stack_add_norm_bwd";
  CHECK(check_norm(fn, shape, num_rows));
  NormArgs a{};
  const int W = shape->width;
  CHECK(check_stride(fn, "h_stride", h_stride, W, 8, &a.x_stride));
  CHECK(check_stride(fn, "dy_stride", dy_stride, W, 8, &a.dy_stride));
  CHECK(check_stride(fn, "d_residual_out_stride", d_residual_out_stride, W, 8, &a.res_stride));
  CHECK(check_stride(fn, "dx_stride", dx_stride, W, 8, &a.y_stride));
  CHECK(check_stride(fn, "d_residual_stride", d_residual_stride, W, 8, &a.h_stride));
  CHECK_PTR(w, "w");
  CHECK_PTR(dw, "dw");
  if (num_rows > 0) {
    CHECK_PTR(h, "h");
    CHECK_PTR(dy, "dy");
    CHECK_ALIGN(d_residual_out, "d_residual_out", 16);
    CHECK_ALIGN(dx, "dx", 16);
    CHECK_ALIGN(d_residual, "d_residual", 16);
    if (!dx && !d_residual) return fail(GDN_ERR_INVALID_ARG, "%s: dx and d_residual are both NULL", fn);
    if (dx == d_residual) return fail(GDN_ERR_INVALID_ARG, "%s: dx is d_residual", fn);
  }
  const int32_t dt = shape->dtype, rdt = shape->residual_dtype;
  CHECK(check_in_place(fn, dx, a.y_stride, dt, h, a.x_stride, rdt));
  CHECK(check_in_place(fn, dx, a.y_stride, dt, dy, a.dy_stride, dt));
  CHECK(check_in_place(fn, dx, a.y_stride, dt, d_residual_out, a.res_stride, rdt));
  CHECK(check_in_place(fn, d_residual, a.h_stride, rdt, h, a.x_stride, rdt));
  CHECK(check_in_place(fn, d_residual, a.h_stride, rdt, dy, a.dy_stride, dt));
  CHECK(check_in_place(fn, d_residual, a.h_stride, rdt, d_residual_out, a.res_stride, rdt));
  CHECK(check_workspace(fn, workspace, workspace_bytes, gdn_stack_norm_workspace_size(shape, num_rows)));
  a.x = h;
  a.res = d_residual_out;
  a.dy = dy;
  a.w = w;
  a.h = d_residual;
  a.y = dx;
  a.rows = num_rows;
  a.width = W;
  a.eps = shape->eps;
  a.w_add = shape->zero_centered ? 1.f : 0.f;
  a.partial = (float*)workspace;
  const int groups = norm_bwd_groups(*shape, num_rows);
  hipStream_t st = (hipStream_t)stream;
  if (groups > 0) GDN_STACK_NORM(GDN_STACK_NORM_BWD_WIDTH, *shape, backward(a, groups, st));
  hipLaunchKernelGGL(k_stack_norm_dw, dim3((W + 31) / 32), dim3(1024), 0, st, a.partial, groups, W, dw);
  return launch_status(fn);
}

// ---------------------------------------------------------------------------
// logits

namespace {

gdn_status check_logits_shape(const char* fn, const gdn_logits_shape* s, int64_t rows) {
  if (!s) return fail(GDN_ERR_INVALID_ARG, "%s: shape is NULL", fn);
  if (s->vocab < 1 || s->vocab > GDN_STACK_MAX_VOCAB)
    return fail(GDN_ERR_UNSUPPORTED, "%s: vocab must be in [1, %d]", fn, GDN_STACK_MAX_VOCAB);
  CHECK(check_dtype(fn, "dtype", s->dtype));
  if (s->top < 0 || s->top > GDN_STACK_MAX_TEACHER)
    return fail(GDN_ERR_UNSUPPORTED, "%s: top must be in [0, %d]", fn, GDN_STACK_MAX_TEACHER);
  CHECK(check_rows(fn, rows));
  if (rows * ((s->vocab + kPart - 1) / kPart) > kMostThreads / 64) return fail(GDN_ERR_UNSUPPORTED, "%s: too many rows", fn);
  return GDN_OK;
}

gdn_status check_top(const char* fn, const gdn_logits_shape& s) {
  if (s.top > GDN_STACK_MAX_TOP || s.top > s.vocab)
    return fail(GDN_ERR_UNSUPPORTED, "%s: top must be at most %d and at most vocab", fn, GDN_STACK_MAX_TOP);
  return GDN_OK;
}

gdn_status check_entries(const char* fn, const gdn_logits_shape& s) {
  if (s.top < 1) return fail(GDN_ERR_UNSUPPORTED, "%s: top must be in [1, %d]", fn, GDN_STACK_MAX_TEACHER);
  return GDN_OK;
}

int element_size(const gdn_logits_shape& s) { return s.dtype == GDN_DTYPE_F32 ? 4 : 2; }

gdn_status check_logits(const char* fn, const gdn_logits_shape* s, int64_t rows, const void* logits, int64_t stride,
                        const float* scale, LogitsArgs* a) {
  CHECK(check_logits_shape(fn, s, rows));
  CHECK(check_stride(fn, "logits_stride", stride, s->vocab, 1, &a->stride));
  CHECK_ALIGN(logits, "logits", element_size(*s));
  CHECK_ALIGN(scale, "scale", 4);
  if (rows > 0 && !logits) return fail(GDN_ERR_INVALID_ARG, "%s: logits is NULL", fn);
  a->logits = logits;
  a->rows = rows;
  a->vocab = s->vocab;
  a->parts = (s->vocab + kPart - 1) / kPart;
  a->top = s->top;
  a->scale = scale;
  a->given_logprobs = s->teacher_logprobs != 0;
  return GDN_OK;
}

gdn_status check_gradient(const char* fn, const gdn_logits_shape& s, void* d_logits, int64_t stride, LogitsArgs* a) {
  CHECK(check_stride(fn, "d_logits_stride", stride, s.vocab, 1, &a->d_stride));
  CHECK_ALIGN(d_logits, "d_logits", element_size(s));
  if (a->rows > 0 && !d_logits) return fail(GDN_ERR_INVALID_ARG, "%s: d_logits is NULL", fn);
  CHECK(check_in_place(fn, d_logits, a->d_stride, 0, a->logits, a->stride, 0));
  a->d_logits = d_logits;
  return GDN_OK;
}

size_t record_bytes(const gdn_logits_shape& s, int64_t rows) {
  return align_up((size_t)rows * ((s.vocab + kPart - 1) / kPart) * sizeof(f32x4));
}

dim3 part_grid(const LogitsArgs& a) { return dim3((unsigned)((a.rows * a.parts + kWaves - 1) / kWaves)); }
dim3 row_grid(const LogitsArgs& a) { return dim3((unsigned)((a.rows + kWaves - 1) / kWaves)); }

template <class E>
bool reads_once(const LogitsArgs& a) {
  return a.rows * a.vocab * (int64_t)sizeof(typename E::T) >= kOnceFrom;
}

template <class E, bool ENTROPY, bool TOP>
void run_parts(const LogitsArgs& a, hipStream_t st) {
  if (reads_once<E>(a))
    hipLaunchKernelGGL((k_stack_parts<E, ENTROPY, TOP, true>), part_grid(a), dim3(64 * kWaves), 0, st, a);
  else
    hipLaunchKernelGGL((k_stack_parts<E, ENTROPY, TOP, false>), part_grid(a), dim3(64 * kWaves), 0, st, a);
}

template <class E, int MODE, RowForm FORM>
void run_rows(const LogitsArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((k_stack_logprobs<E, MODE, FORM>), row_grid(a), dim3(64 * kWaves), 0, st, a);
}

template <class E, int MODE>
void run_short(const LogitsArgs& a, hipStream_t st) {
  a.entropy ? run_rows<E, MODE, kMakeEntropy>(a, st) : run_rows<E, MODE, kMake>(a, st);
}

template <class E>
void run_logprobs(const LogitsArgs& a, hipStream_t st) {
  const int mode = top_mode(a.vocab, a.top);
  if (a.parts == 1) {  // up to 2,048 columns
    mode == kNoTop ? run_short<E, kNoTop>(a, st)
    : mode == kTopColumns ? run_short<E, kTopColumns>(a, st)
                          : run_short<E, kTopEights>(a, st);
    return;
  }
  if (mode == kTopGroups)
    a.entropy ? run_parts<E, true, true>(a, st) : run_parts<E, false, true>(a, st);
  else
    a.entropy ? run_parts<E, true, false>(a, st) : run_parts<E, false, false>(a, st);
  mode == kNoTop ? run_rows<E, kNoTop, kJoin>(a, st)
  : mode == kTopEights ? run_rows<E, kTopEights, kJoin>(a, st)
                       : run_rows<E, kTopGroups, kJoin>(a, st);
}

template <class E, bool ONCE>
void launch_logprobs_bwd(const LogitsArgs& a, hipStream_t st) {
  if (a.d_entropy)
    hipLaunchKernelGGL((k_stack_logprobs_bwd<E, true, ONCE>), part_grid(a), dim3(64 * kWaves), 0, st, a);
  else
    hipLaunchKernelGGL((k_stack_logprobs_bwd<E, false, ONCE>), part_grid(a), dim3(64 * kWaves), 0, st, a);
}

template <class E>
void run_logprobs_bwd(const LogitsArgs& a, hipStream_t st) {
  reads_once<E>(a) ? launch_logprobs_bwd<E, true>(a, st) : launch_logprobs_bwd<E, false>(a, st);
}

template <class E>
void run_distill(const LogitsArgs& a, hipStream_t st) {
  if (a.parts == 1) {
    hipLaunchKernelGGL((k_stack_distill<E, kMake>), row_grid(a), dim3(64 * kWaves), 0, st, a);
  } else {
    run_parts<E, false, false>(a, st);
    hipLaunchKernelGGL((k_stack_distill<E, kJoin>), row_grid(a), dim3(64 * kWaves), 0, st, a);
  }
}

template <class E>
void run_distill_bwd(const LogitsArgs& a, hipStream_t st) {
  if (reads_once<E>(a))
    hipLaunchKernelGGL((k_stack_distill_bwd<E, true>), part_grid(a), dim3(64 * kWaves), 0, st, a);
  else
    hipLaunchKernelGGL((k_stack_distill_bwd<E, false>), part_grid(a), dim3(64 * kWaves), 0, st, a);
}

#define GDN_STACK_LOGITS(shape, fn_, ...) \
  ((shape).dtype == GDN_DTYPE_F32 ? fn_<F32>(__VA_ARGS__) : fn_<B16>(__VA_ARGS__))

}  // namespace

extern "C" size_t gdn_stack_logits_workspace_size(const gdn_logits_shape* shape, int64_t num_rows) {
  if (check_logits_shape("gdn_stack_logits_workspace_size", shape, num_rows) != GDN_OK) return 0;
  const size_t rec = record_bytes(*shape, num_rows);
  return rec + (shape->top ? rec * (kGroups * sizeof(float) / sizeof(f32x4)) : 0) + 256;
}

extern "C" gdn_status gdn_stack_logprobs(const gdn_logits_shape* shape, int64_t num_rows, const void* logits,
                                         int64_t logits_stride, const int32_t* targets, const float* scale,
                                         float* logprobs, float* entropy, int32_t* top_ids, float* top_logprobs,
                                         float* stats, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "gdn_stack_logprobs";
  LogitsArgs a{};
  CHECK(check_logits(fn, shape, num_rows, logits, logits_stride, scale, &a));
  CHECK(check_top(fn, *shape));
  CHECK_ALIGN(targets, "targets", 4);
  CHECK_ALIGN(logprobs, "logprobs", 4);
  CHECK_ALIGN(entropy, "entropy", 4);
  CHECK_ALIGN(top_ids, "top_ids", 4);
  CHECK_ALIGN(top_logprobs, "top_logprobs", 4);
  CHECK_ALIGN(stats, "stats", 4);
  if (num_rows == 0) return done();
  if (!targets != !logprobs) return fail(GDN_ERR_INVALID_ARG, "%s: targets and logprobs go together", fn);
  if (shape->top && (!top_ids || !top_logprobs))
    return fail(GDN_ERR_INVALID_ARG, "%s: top_ids or top_logprobs is NULL", fn);
  if (!logprobs && !entropy && !shape->top && !stats) return fail(GDN_ERR_INVALID_ARG, "%s: no output is asked for", fn);
  CHECK(check_workspace(fn, workspace, workspace_bytes, gdn_stack_logits_workspace_size(shape, num_rows)));
  a.targets = targets;
  a.rec = (f32x4*)workspace;
  a.group_max = (float*)((char*)workspace + record_bytes(*shape, num_rows));
  a.logprobs = logprobs;
  a.entropy = entropy;
  a.top_ids = top_ids;
  a.top_logprobs = top_logprobs;
  a.stats = stats;
  GDN_STACK_LOGITS(*shape, run_logprobs, a, (hipStream_t)stream);
  return launch_status(fn);
}

extern "C" gdn_status gdn_stack_logprobs_bwd(const gdn_logits_shape* shape, int64_t num_rows, const void* logits,
                                             int64_t logits_stride, const int32_t* targets, const float* scale,
                                             const float* stats, const float* entropy, const float* d_logprobs,
                                             const float* d_entropy, void* d_logits, int64_t d_logits_stride,
                                             void* stream) {
  const char* fn = "gdn_stack_logprobs_bwd";
  LogitsArgs a{};
  CHECK(check_logits(fn, shape, num_rows, logits, logits_stride, scale, &a));
  CHECK(check_gradient(fn, *shape, d_logits, d_logits_stride, &a));
  CHECK_ALIGN(targets, "targets", 4);
  CHECK_ALIGN(entropy, "entropy", 4);
  CHECK_ALIGN(d_logprobs, "d_logprobs", 4);
  CHECK_ALIGN(d_entropy, "d_entropy", 4);
  if (num_rows == 0) return done();
  CHECK_PTR_TO(stats, "stats", 4);
  if (!d_logprobs && !d_entropy) return fail(GDN_ERR_INVALID_ARG, "%s: d_logprobs and d_entropy are both NULL", fn);
  if (d_logprobs && !targets) return fail(GDN_ERR_INVALID_ARG, "%s: d_logprobs needs targets", fn);
  if (d_entropy && !entropy) return fail(GDN_ERR_INVALID_ARG, "%s: d_entropy needs entropy", fn);
  a.targets = targets;
  a.in_stats = stats;
  a.in_entropy = entropy;
  a.d_logprobs = d_logprobs;
  a.d_entropy = d_entropy;
  GDN_STACK_LOGITS(*shape, run_logprobs_bwd, a, (hipStream_t)stream);
  return launch_status(fn);
}

extern "C" gdn_status gdn_stack_distill(const gdn_logits_shape* shape, int64_t num_rows, const void* logits,
                                        int64_t logits_stride, const int32_t* teacher_ids, const float* teacher_values,
                                        const float* scale, float* loss, float* stats, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  const char* fn = "gdn_stack_distill";
  LogitsArgs a{};
  CHECK(check_logits(fn, shape, num_rows, logits, logits_stride, scale, &a));
  CHECK(check_entries(fn, *shape));
  CHECK_ALIGN(stats, "stats", 16);
  if (num_rows == 0) return done();
  CHECK_PTR_TO(teacher_ids, "teacher_ids", 4);
  CHECK_PTR_TO(teacher_values, "teacher_values", 4);
  CHECK_PTR_TO(loss, "loss", 4);
  CHECK(check_workspace(fn, workspace, workspace_bytes, gdn_stack_logits_workspace_size(shape, num_rows)));
  a.ids = teacher_ids;
  a.values = teacher_values;
  a.rec = (f32x4*)workspace;
  a.loss = loss;
  a.stats = stats;
  GDN_STACK_LOGITS(*shape, run_distill, a, (hipStream_t)stream);
  return launch_status(fn);
}

extern "C" gdn_status gdn_stack_distill_bwd(const gdn_logits_shape* shape, int64_t num_rows, const void* logits,
                                            int64_t logits_stride, const int32_t* teacher_ids,
                                            const float* teacher_values, const float* scale, const float* stats,
                                            const float* d_loss, void* d_logits, int64_t d_logits_stride,
                                            void* stream) {
  const char* fn = "gdn_stack_distill_bwd";
  LogitsArgs a{};
  CHECK(check_logits(fn, shape, num_rows, logits, logits_stride, scale, &a));
  CHECK(check_entries(fn, *shape));
  CHECK(check_gradient(fn, *shape, d_logits, d_logits_stride, &a));
  if (num_rows == 0) return done();
  CHECK_PTR_TO(teacher_ids, "teacher_ids", 4);
  CHECK_PTR_TO(teacher_values, "teacher_values", 4);
  CHECK_PTR(stats, "stats");
  CHECK_PTR_TO(d_loss, "d_loss", 4);
  a.ids = teacher_ids;
  a.values = teacher_values;
  a.in_stats = stats;
  a.d_loss = d_loss;
  GDN_STACK_LOGITS(*shape, run_distill_bwd, a, (hipStream_t)stream);
  return launch_status(fn);
}
