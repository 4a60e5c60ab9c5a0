/*
 * gdn_stack.h -- C ABI of what a stack of Gated DeltaNet (gdn_cpr.h) and
 * attention layers (gdn_attn.h) needs between its layers and at its end, for
 * AMD Instinct MI355X (gfx950).
 *
 *   gdn_stack_add_norm    the residual's addition and the root-mean-square norm
 *                         in one pass, in the input type, in 8 bits with scales
 *                         or in both; with its gradient;
 *   gdn_stack_logprobs    log probabilities of given tokens, the entropy and the
 *                         top alternatives from a row of logits; with the
 *                         gradient of the first two;
 *   gdn_stack_distill     the divergence of the logits' distribution from a
 *                         teacher's top entries; with its gradient.
 *
 * A rollout's log probabilities and the trainer's are compared with each other
 * (English page, "Experimental Results"), so a row's results depend on the row
 * alone: every sum over a row runs in an order that its length fixes, however
 * many rows the call has and wherever they lie.  dw of the norm is a sum over
 * rows; its order depends on the number of rows and the width only.
 *
 * Conventions: those of gdn_cpr.h (device pointers; calls only enqueue on
 * `stream`; nothing is allocated; host-detectable errors return a status
 * before anything is enqueued; gdn_cpr_last_error describes the last one).
 * Pointers are 16-byte aligned; logits, their gradients and the arrays of
 * numbers to a row that go with them (all but distill's stats) need the
 * alignment of their elements only, so that they may be any rows of larger ones.
 * A stride is the distance in elements between a tensor's rows; 0 means that
 * they are contiguous.  Rows of the norm's tensors have strides that are
 * multiples of 8 and at least the width; those of logits any stride of at
 * least the vocabulary, and what lies between two rows is left as it is.
 * A launch's threads are counted in 32 bits: rows up to 2^24 - 16 of a width
 * past 2,048 (2^26 - 64 up to that, 2^28 - 256 up to 128), and of logits rows *
 * ceil(vocab / 2,048) up to 2^26 - 64.
 */
#ifndef GDN_STACK_H
#define GDN_STACK_H

#include "gdn_cpr.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_STACK_MAX_WIDTH 16384
#define GDN_STACK_GROUP 128
#define GDN_STACK_MAX_VOCAB (1 << 20)
#define GDN_STACK_MAX_TOP 64
#define GDN_STACK_MAX_TEACHER 256

/* The norm (host struct). */
typedef struct {
  int32_t width;          /* columns of a row: a multiple of 8, 8 .. GDN_STACK_MAX_WIDTH */
  int32_t dtype;          /* gdn_dtype of x, y and their gradients */
  int32_t residual_dtype; /* that of the residual stream: dtype, or fp32 */
  int32_t group;          /* columns to a scale of the 8-bit output: GDN_STACK_GROUP (which
                             then divides width), 0 for one scale to a row, -1 where there
                             is no such output */
  int32_t zero_centered;  /* the weights are stored as w - 1 */
  float eps;
} gdn_norm_shape;

/* Rows of logits (host struct). */
typedef struct {
  int32_t vocab;            /* columns of a row, 1 .. GDN_STACK_MAX_VOCAB */
  int32_t dtype;            /* gdn_dtype of the logits and their gradient */
  int32_t top;              /* logprobs: alternatives to a row, 0 .. GDN_STACK_MAX_TOP, at most
                               vocab; distill: the teacher's entries to a row, 1 ..
                               GDN_STACK_MAX_TEACHER */
  int32_t teacher_logprobs; /* distill: the teacher's values are log probabilities */
} gdn_logits_shape;

/*
 * h = x + residual, added in fp32 and rounded to the residual's type, or x in
 * that type where residual is NULL; with r = rsqrt(mean(h^2) + eps) of h as rounded (so
 * the norm of a stored h has the same bits), n = h r w.
 *   w             fp32 [width]
 *   residual_out  h; may be NULL, and may be residual or x (same type and
 *                 stride)
 *   y             n in dtype; may be x, or residual of that type (same stride)
 *   y8, y_scale   n in e4m3: the quotient n / s, in fp32, to the nearest code (half to
 *                 even), s = max(amax, 2^-100) / 448 over the group's |n|; y8 [rows,
 *                 width], y_scale fp32 [rows, width / group] ([rows, 1] for group
 *                 0), both contiguous
 * y or y8 may be NULL (y_scale with y8), not both.  Computed in fp32, rounded
 * once; the sum of h^2 is finite for |h| up to 2^63 / sqrt(width).  Past that,
 * and in a row that holds an infinity, r is 0: n is 0, and NaN in the place of
 * the infinity.  r is 0 too where eps is 0 and so is the mean (rows of
 * zeros; squares below 2^-149 are 0, and lose bits below 2^-126).  A NaN makes all of
 * its row NaN (y_scale aside).
 */
gdn_status gdn_stack_add_norm(const gdn_norm_shape* shape, int64_t num_rows, const void* x, int64_t x_stride,
                              const void* residual, int64_t residual_stride, const float* w, void* residual_out,
                              int64_t residual_out_stride, void* y, int64_t y_stride, uint8_t* y8, float* y_scale,
                              void* stream);

/*
 * Its gradient: from h (residual_out, in residual_dtype), dy (of y, or of
 * y8 s: the rounding counts as none) and d_residual_out (of residual_out as its
 * later readers give it; NULL for none),
 *   dh = d_residual_out + r (dn - h r^2 mean(dn h)),  dn = dy w,
 * the gradient of x and of residual alike: dx in dtype, d_residual in
 * residual_dtype, either may be NULL.  dw fp32 [width] (0 without rows).  Of a
 * row with r = 0, dh is d_residual_out and dw has nothing; one whose h holds a
 * NaN gives NaN everywhere.  dx may be dy, d_residual may be d_residual_out,
 * either may be h of its type (same strides).
 */
gdn_status gdn_stack_add_norm_bwd(const gdn_norm_shape* shape, int64_t num_rows, const void* h, int64_t h_stride,
                                  const float* w, const void* dy, int64_t dy_stride, const void* d_residual_out,
                                  int64_t d_residual_out_stride, void* dx, int64_t dx_stride, void* d_residual,
                                  int64_t d_residual_stride, float* dw, void* workspace, size_t workspace_bytes,
                                  void* stream);

/* Bytes of workspace of gdn_stack_add_norm_bwd (host only; 0 for an invalid
 * shape or size).  Two calls that may run at once need one each. */
size_t gdn_stack_norm_workspace_size(const gdn_norm_shape* shape, int64_t num_rows);

/*
 * With z = scale logits of a row, m its largest logit, L = log sum exp(scale
 * (logits - m)) and log q = scale (logits - m) - L:
 *   targets       int32 [rows], or NULL.  A row whose target is no index of
 *                 the vocabulary is left out: not read, and zeros in all
 *                 outputs (indices -1)
 *   scale         fp32 [rows], positive, at most 2^127: one over the row's
 *                 temperature; NULL for 1
 *   logprobs      [rows] log q of the target; NULL without targets
 *   entropy       [rows] -sum q log q; may be NULL
 *   top_ids, top_logprobs  [rows, top] the largest logits' indices, equal ones
 *                 by ascending index, and their log q; NULL for top 0
 *   stats         [rows, 2] m and L, which the gradient takes; may be NULL
 * All outputs fp32 (indices int32), contiguous.  Logits of -inf are masked:
 * q is 0.  A row of nothing else has log q = -inf, entropy 0 and stats (-inf,
 * 0).  A row that holds a NaN or +inf gives NaN; among the alternatives a (quiet)
 * NaN ranks as -inf.
 */
gdn_status gdn_stack_logprobs(const gdn_logits_shape* shape, int64_t num_rows, const void* logits,
                              int64_t logits_stride, const int32_t* targets, const float* scale, float* logprobs,
                              float* entropy, int32_t* top_ids, float* top_logprobs, float* stats, void* workspace,
                              size_t workspace_bytes, void* stream);

/*
 * The gradient of logprobs and entropy (from stats, and entropy where
 * d_entropy is given), with g = d_logprobs and f = d_entropy, fp32 [rows]:
 *   d_logits = scale (g ([v = target] - q) - f q (log q + entropy)).
 * d_logprobs or d_entropy may be NULL (0), not both; without targets
 * d_logprobs is NULL.  targets are those of the forward call, with d_entropy alone
 * too: they say which rows it left out.  Such rows, and rows of -inf only, get zeros.
 * d_logits may be logits (same stride).
 */
gdn_status gdn_stack_logprobs_bwd(const gdn_logits_shape* shape, int64_t num_rows, const void* logits,
                                  int64_t logits_stride, const int32_t* targets, const float* scale,
                                  const float* stats, const float* entropy, const float* d_logprobs,
                                  const float* d_entropy, void* d_logits, int64_t d_logits_stride, void* stream);

/*
 * loss = sum over a row's entries of p (log p - log q), q as above.
 *   teacher_ids     int32 [rows, top]; entries that are no index of the
 *                   vocabulary are not there.  One that comes twice counts twice
 *   teacher_values  fp32 [rows, top]: the teacher's logits, p = softmax(scale
 *                   values) over the row's entries; or with teacher_logprobs
 *                   its log probabilities, p = exp(values), which need not add
 *                   up to 1
 *   loss            [rows]; +inf where a q is 0 and its p is not
 *   stats           [rows, 4] m and L, then the largest of the values and log
 *                   sum exp(scale (values - largest)) (0 and 0 with
 *                   teacher_logprobs, and where no entry is there); may be NULL
 * A row without entries, or with p = 0 in all, has loss 0 and gradient 0.
 */
gdn_status gdn_stack_distill(const gdn_logits_shape* shape, int64_t num_rows, const void* logits,
                             int64_t logits_stride, const int32_t* teacher_ids, const float* teacher_values,
                             const float* scale, float* loss, float* stats, void* workspace, size_t workspace_bytes,
                             void* stream);

/*
 * Its gradient, d_loss fp32 [rows]:
 *   d_logits = d_loss scale (q sum p - sum of p over the entries of index v).
 * Rows of -inf only get zeros.  d_logits may be logits (same stride).
 */
gdn_status gdn_stack_distill_bwd(const gdn_logits_shape* shape, int64_t num_rows, const void* logits,
                                 int64_t logits_stride, const int32_t* teacher_ids, const float* teacher_values,
                                 const float* scale, const float* stats, const float* d_loss, void* d_logits,
                                 int64_t d_logits_stride, void* stream);

/* Bytes of workspace of gdn_stack_logprobs and gdn_stack_distill (host only; 0
 * for an invalid shape or size).  Two calls that may run at once need one
 * each. */
size_t gdn_stack_logits_workspace_size(const gdn_logits_shape* shape, int64_t num_rows);

#ifdef __cplusplus
}
#endif

#endif /* GDN_STACK_H */
