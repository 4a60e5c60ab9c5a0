// The attention layer for gfx950: host side and the C ABI (gdn_attn.h).
// The kernels live in attn_plan_kernels.hpp, attn_norm_rope_kernels.hpp,
// attn_cache_kernels.hpp and attn_kernels.hpp.
//
// Per call, on the caller's stream:
//   plan           k_attn_plan (and k_attn_plan_tokens for many tokens)
//   norm + rope    k_attn_norm_rope; its gradient k_attn_norm_rope_bwd and
//                  k_attn_norm_rope_dw
//   prefill        k_attn_append (tails, full blocks), then k_attn_prefill, or
//                  k_attn_rows and k_attn_join (takes_rows)
//   decode step    k_attn_rows (attention and append), k_attn_join
//   cache read     k_attn_cache_read
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <string>

#include "../../include/gdn_attn.h"
#include "attn_kernels.hpp"
#include "attn_norm_rope_kernels.hpp"
#include "attn_plan_kernels.hpp"

std::string& gdn_last_error_text();  // gdn_cpr.hip

namespace {

using namespace attn;

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
bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

#define CHECK_PTR(p, name)                                                                          \
  do {                                                                                              \
    if (!(p)) return fail(GDN_ERR_INVALID_ARG, "%s: %s is NULL", fn, name);                         \
    if (!aligned16(p)) return fail(GDN_ERR_INVALID_ARG, "%s: %s is not 16-byte aligned", fn, name); \
  } while (0)

#define CHECK_OPT_PTR(p, name)                                                                      \
  do {                                                                                              \
    if (!aligned16(p)) return fail(GDN_ERR_INVALID_ARG, "%s: %s is not 16-byte aligned", fn, name); \
  } while (0)

#define CHECK(call)                  \
  do {                               \
    const gdn_status r_ = (call);    \
    if (r_ != GDN_OK) return r_;     \
  } while (0)

int kv_heads(const gdn_attn_shape& s) { return s.num_kv_heads > 0 ? s.num_kv_heads : s.num_heads; }

constexpr int kMaxHeads = 1 << 15;

gdn_status check_shape(const char* fn, const gdn_attn_shape* s) {
  if (!s) return fail(GDN_ERR_INVALID_ARG, "%s: shape is NULL", fn);
  if (s->num_heads < 1 || s->num_heads > kMaxHeads)
    return fail(GDN_ERR_UNSUPPORTED, "%s: num_heads must be in [1, %d]", fn, kMaxHeads);
  if (s->num_kv_heads < 0 || s->num_kv_heads > s->num_heads ||
      (s->num_kv_heads > 0 && s->num_heads % s->num_kv_heads != 0))
    return fail(GDN_ERR_UNSUPPORTED, "%s: num_kv_heads must be 0 or divide num_heads", fn);
  if (s->head_dim != 64 && s->head_dim != 128 && s->head_dim != 256)
    return fail(GDN_ERR_UNSUPPORTED, "%s: head_dim must be 64, 128 or 256", fn);
  if (s->dtype != GDN_DTYPE_F32 && s->dtype != GDN_DTYPE_BF16)
    return fail(GDN_ERR_UNSUPPORTED, "%s: dtype must be GDN_DTYPE_F32 or GDN_DTYPE_BF16", fn);
  return GDN_OK;
}

gdn_status check_sizes(const char* fn, int64_t num_seqs, int64_t total_tokens) {
  if (num_seqs < 0 || total_tokens < 0) return fail(GDN_ERR_INVALID_ARG, "%s: negative size", fn);
  if (total_tokens > INT32_MAX / 2 || num_seqs > INT32_MAX / 2) return fail(GDN_ERR_UNSUPPORTED, "%s: too many tokens", fn);
  return GDN_OK;
}

// A token stride as given, resolved: 0 is `row` elements.
gdn_status check_stride(const char* fn, const char* name, int64_t given, int64_t row, int64_t* out) {
  *out = given ? given : row;
  if (*out < row || *out % 8 != 0 || *out > INT64_MAX / INT32_MAX)
    return fail(GDN_ERR_INVALID_ARG, "%s: %s must be 0 or a multiple of 8 of at least %lld", fn, name, (long long)row);
  return GDN_OK;
}

gdn_status check_pool(const char* fn, const gdn_attn_pool* p) {
  if (!p) return fail(GDN_ERR_INVALID_ARG, "%s: pool is NULL", fn);
  CHECK_PTR(p->block_table, "pool.block_table");
  CHECK_PTR(p->blocks_held, "pool.blocks_held");
  CHECK_PTR(p->free_blocks, "pool.free_blocks");
  CHECK_PTR(p->free_count, "pool.free_count");
  CHECK_PTR(p->seq_len, "pool.seq_len");
  if (p->num_slots < 1 || p->max_blocks < 1 || p->num_blocks < 1)
    return fail(GDN_ERR_INVALID_ARG, "%s: pool sizes must be positive", fn);
  return GDN_OK;
}

}  // namespace

// ---------------------------------------------------------------------------
// plan

extern "C" gdn_status gdn_attn_plan(const gdn_attn_pool* pool, int32_t num_seqs, int64_t total_tokens,
                                    const int32_t* cu_seqlens, int32_t advance, const gdn_attn_step* step,
                                    void* stream) {
  const char* fn = "gdn_attn_plan";
  CHECK(check_sizes(fn, num_seqs, total_tokens));
  CHECK(check_pool(fn, pool));
  if (!step) return fail(GDN_ERR_INVALID_ARG, "%s: step is NULL", fn);
  CHECK_PTR(cu_seqlens, "cu_seqlens");
  CHECK_PTR(step->status, "step.status");
  if (step->block_table != pool->block_table || step->max_blocks != pool->max_blocks || step->num_slots != pool->num_slots)
    return fail(GDN_ERR_INVALID_ARG, "%s: step.block_table, max_blocks and num_slots are not the pool's", fn);
  CHECK_OPT_PTR(step->slot_index, "step.slot_index");
  if (num_seqs > 0) CHECK_PTR(step->ctx_len, "step.ctx_len");
  if (total_tokens > 0) {
    CHECK_PTR(step->positions, "step.positions");
    CHECK_PTR(step->slot_map, "step.slot_map");
  }
  if (num_seqs == 0 && total_tokens > 0) return fail(GDN_ERR_INVALID_ARG, "%s: tokens without requests", fn);
  PlanArgs a{};
  a.table = pool->block_table;
  a.held = pool->blocks_held;
  a.free = pool->free_blocks;
  a.free_count = pool->free_count;
  a.seq_len = pool->seq_len;
  a.num_slots = pool->num_slots;
  a.max_blocks = pool->max_blocks;
  a.num_blocks = pool->num_blocks;
  a.N = num_seqs;
  a.T = (int)total_tokens;
  a.advance = advance != 0;
  a.tokens_here = total_tokens <= kTokensInPlan;
  a.cu = cu_seqlens;
  a.slot = step->slot_index;
  a.ctx_len = step->ctx_len;
  a.positions = step->positions;
  a.slot_map = step->slot_map;
  a.status = step->status;
  hipLaunchKernelGGL(k_attn_plan, dim3(1), dim3(kPlanThreads), 0, (hipStream_t)stream, a);
  if (!a.tokens_here)
    hipLaunchKernelGGL(k_attn_plan_tokens, dim3((a.T + 255) / 256), dim3(256), 0, (hipStream_t)stream, a);
  return launch_status(fn);
}

extern "C" gdn_status gdn_attn_release(const gdn_attn_pool* pool, int32_t num_seqs, const int32_t* slot_index,
                                       void* stream) {
  const char* fn = "gdn_attn_release";
  CHECK(check_sizes(fn, num_seqs, 0));
  CHECK(check_pool(fn, pool));
  CHECK_OPT_PTR(slot_index, "slot_index");
  if (num_seqs == 0) return done();
  ReleaseArgs a{};
  a.table = pool->block_table;
  a.held = pool->blocks_held;
  a.free = pool->free_blocks;
  a.free_count = pool->free_count;
  a.seq_len = pool->seq_len;
  a.num_slots = pool->num_slots;
  a.max_blocks = pool->max_blocks;
  a.num_blocks = pool->num_blocks;
  a.N = num_seqs;
  a.slot = slot_index;
  hipLaunchKernelGGL(k_attn_release, dim3(1), dim3(kPlanThreads), 0, (hipStream_t)stream, a);
  return launch_status(fn);
}

// ---------------------------------------------------------------------------
// norm and rotation

namespace {

// work-groups of the gradient's row pass, each with a partial dw: enough to
// fill the card (4 on each of 256 CUs), few enough that adding them up is short
// (20,000 tokens of 20 heads, d = 128: 68 us; with half as many 93, twice 78)
constexpr int kNormBwdGroups = 1024;

int norm_bwd_groups(const gdn_attn_shape& s, int64_t T) {
  const int64_t rows = T * s.num_heads, per = kNormThreads / (s.head_dim / 8);
  return (int)std::min<int64_t>(kNormBwdGroups, std::max<int64_t>(1, (rows + per - 1) / per));
}

gdn_status check_norm(const char* fn, const gdn_attn_shape* shape, const gdn_attn_rope* rope, int64_t T, const void* q,
                      const void* k, int64_t q_stride, int64_t k_stride, const float* w_q, const float* w_k,
                      const float* cos_sin, const int32_t* positions, NormRopeArgs* a) {
  CHECK(check_shape(fn, shape));
  CHECK(check_sizes(fn, 0, T));
  if (!rope) return fail(GDN_ERR_INVALID_ARG, "%s: rope is NULL", fn);
  const int d = shape->head_dim, H = shape->num_heads, Hk = kv_heads(*shape);
  if (T * H > INT32_MAX) return fail(GDN_ERR_UNSUPPORTED, "%s: too many rows", fn);
  if (rope->rotary_dim < 0 || rope->rotary_dim > d || rope->rotary_dim % 8 != 0)
    return fail(GDN_ERR_UNSUPPORTED, "%s: rotary_dim must be a multiple of 8 up to head_dim", fn);
  if (!(rope->eps >= 0.f) || std::isinf(rope->eps)) return fail(GDN_ERR_INVALID_ARG, "%s: eps must be finite and not negative", fn);
  CHECK_PTR(w_q, "w_q");
  CHECK_PTR(w_k, "w_k");
  CHECK(check_stride(fn, "q_stride", q_stride, (int64_t)H * d, &a->x_stride[0]));
  CHECK(check_stride(fn, "k_stride", k_stride, (int64_t)Hk * d, &a->x_stride[1]));
  if (T > 0) {
    CHECK_PTR(q, "q");
    CHECK_PTR(k, "k");
    if (rope->rotary_dim > 0) {
      if (rope->num_positions < 1) return fail(GDN_ERR_INVALID_ARG, "%s: num_positions must be positive", fn);
      CHECK_PTR(cos_sin, "cos_sin");
      CHECK_PTR(positions, "positions");
    }
  }
  a->x[0] = q;
  a->x[1] = k;
  a->w[0] = w_q;
  a->w[1] = w_k;
  a->heads[0] = H;
  a->heads[1] = Hk;
  a->rows[0] = T * H;
  a->rows[1] = T * Hk;
  a->cos_sin = cos_sin;
  a->positions = positions;
  a->rd = rope->rotary_dim;
  a->interleaved = rope->interleaved != 0;
  a->num_positions = rope->num_positions;
  a->eps = rope->eps;
  a->w_add = rope->zero_centered ? 1.f : 0.f;
  return GDN_OK;
}

// Outputs that the caches could not hold for long are stored past them: from
// 64 MB on (d = 128, forward and gradient in us, past / into the caches: 33 MB 16.4 / 15.3 and
// 26.6 / 25.4; 84 MB 37 / 43 and 59 / 61; 102 MB 40.6 / 41.5 and 61 / 68).  What reads them next is no
// slower for it (with the prefill of 5 x 2,048 behind it 207 us either way, of 4 x 1,700 with 28 MB 104 / 106).
template <class E, int D>
bool streams(const NormRopeArgs& a) {
  return (a.rows[0] + a.rows[1]) * (int64_t)(D * sizeof(typename E::T)) >= (int64_t(64) << 20);
}

template <class E, int D, int U, bool STREAM>
void launch_norm(NormRopeArgs& a, hipStream_t st) {
  const int64_t per = (int64_t)(kNormThreads / (D / 8)) * U;
  for (int i = 0; i < 2; ++i) a.groups[i] = (int)((a.rows[i] + per - 1) / per);
  hipLaunchKernelGGL((k_attn_norm_rope<E, D, U, STREAM>), dim3(a.groups[0] + a.groups[1]), dim3(kNormThreads), 0, st, a);
}

// Four rows per lane group once that still leaves 8 work-groups per CU (20
// heads, d = 128: 20,000 tokens 41.3 us with four, 43.5 with one; 6,400 tokens 15.9 and 15.2).
template <class E, int D>
void run_norm(NormRopeArgs& a, hipStream_t st) {
  const int64_t per = kNormThreads / (D / 8);
  if (streams<E, D>(a))
    launch_norm<E, D, 4, true>(a, st);
  else if (a.rows[0] + a.rows[1] >= per * 4 * 2048)
    launch_norm<E, D, 4, false>(a, st);
  else
    launch_norm<E, D, 1, false>(a, st);
}

template <class E, int D>
void run_norm_bwd(const NormRopeArgs& a, int groups, float* dw_q, float* dw_k, hipStream_t st) {
  if (streams<E, D>(a))
    hipLaunchKernelGGL((k_attn_norm_rope_bwd<E, D, true>), dim3(groups), dim3(kNormThreads), 0, st, a);
  else
    hipLaunchKernelGGL((k_attn_norm_rope_bwd<E, D, false>), dim3(groups), dim3(kNormThreads), 0, st, a);
  hipLaunchKernelGGL(k_attn_norm_rope_dw, dim3(2 * D / 32), dim3(1024), 0, st, a.partial, groups, D, dw_q, dw_k);
}

#define GDN_ATTN_DISPATCH(shape, fn_, ...)                                \
  do {                                                                    \
    const bool bf_ = (shape).dtype == GDN_DTYPE_BF16;                     \
    switch ((shape).head_dim) {                                           \
      case 64: bf_ ? fn_<ElemBf16, 64>(__VA_ARGS__) : fn_<ElemF32, 64>(__VA_ARGS__); break;    \
      case 128: bf_ ? fn_<ElemBf16, 128>(__VA_ARGS__) : fn_<ElemF32, 128>(__VA_ARGS__); break; \
      default: bf_ ? fn_<ElemBf16, 256>(__VA_ARGS__) : fn_<ElemF32, 256>(__VA_ARGS__); break;  \
    }                                                                     \
  } while (0)

}  // namespace

extern "C" gdn_status gdn_attn_qk_norm_rope(const gdn_attn_shape* shape, const gdn_attn_rope* rope,
                                            int64_t total_tokens, const void* q, const void* k, int64_t q_stride,
                                            int64_t k_stride, const float* w_q, const float* w_k,
                                            const float* cos_sin, const int32_t* positions, void* q_out, void* k_out,
                                            int64_t q_out_stride, int64_t k_out_stride, void* stream) {
  const char* fn = "gdn_attn_qk_norm_rope";
  NormRopeArgs a{};
  CHECK(check_norm(fn, shape, rope, total_tokens, q, k, q_stride, k_stride, w_q, w_k, cos_sin, positions, &a));
  const int64_t d = shape->head_dim;
  CHECK(check_stride(fn, "q_out_stride", q_out_stride, shape->num_heads * d, &a.out_stride[0]));
  CHECK(check_stride(fn, "k_out_stride", k_out_stride, kv_heads(*shape) * d, &a.out_stride[1]));
  if (total_tokens == 0) return done();
  CHECK_PTR(q_out, "q_out");
  CHECK_PTR(k_out, "k_out");
  a.out[0] = q_out;
  a.out[1] = k_out;
  for (int i = 0; i < 2; ++i)
    if (a.out[i] == a.x[i] && a.out_stride[i] != a.x_stride[i])
      return fail(GDN_ERR_INVALID_ARG, "%s: in place needs equal strides", fn);
  GDN_ATTN_DISPATCH(*shape, run_norm, a, (hipStream_t)stream);
  return launch_status(fn);
}

extern "C" gdn_status gdn_attn_qk_norm_rope_bwd(const gdn_attn_shape* shape, const gdn_attn_rope* rope,
                                                int64_t total_tokens, const void* q, const void* k, int64_t q_stride,
                                                int64_t k_stride, const float* w_q, const float* w_k,
                                                const float* cos_sin, const int32_t* positions, const void* d_q_out,
                                                const void* d_k_out, int64_t dqo_stride, int64_t dko_stride, void* dq,
                                                void* dk, int64_t dq_stride, int64_t dk_stride, float* dw_q,
                                                float* dw_k, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "gdn_attn_qk_norm_rope_bwd";
  NormRopeArgs a{};
  CHECK(check_norm(fn, shape, rope, total_tokens, q, k, q_stride, k_stride, w_q, w_k, cos_sin, positions, &a));
  const int64_t d = shape->head_dim;
  CHECK(check_stride(fn, "dqo_stride", dqo_stride, shape->num_heads * d, &a.dy_stride[0]));
  CHECK(check_stride(fn, "dko_stride", dko_stride, kv_heads(*shape) * d, &a.dy_stride[1]));
  CHECK(check_stride(fn, "dq_stride", dq_stride, shape->num_heads * d, &a.out_stride[0]));
  CHECK(check_stride(fn, "dk_stride", dk_stride, kv_heads(*shape) * d, &a.out_stride[1]));
  CHECK_PTR(dw_q, "dw_q");
  CHECK_PTR(dw_k, "dw_k");
  if (total_tokens > 0) {
    CHECK_PTR(d_q_out, "d_q_out");
    CHECK_PTR(d_k_out, "d_k_out");
    CHECK_PTR(dq, "dq");
    CHECK_PTR(dk, "dk");
  }
  a.dy[0] = d_q_out;
  a.dy[1] = d_k_out;
  a.out[0] = dq;
  a.out[1] = dk;
  for (int i = 0; i < 2; ++i)
    if ((a.out[i] == a.dy[i] && a.out_stride[i] != a.dy_stride[i]) || (a.out[i] == a.x[i] && a.out_stride[i] != a.x_stride[i]))
      return fail(GDN_ERR_INVALID_ARG, "%s: in place needs equal strides", fn);
  const size_t need = gdn_attn_workspace_size(shape, GDN_ATTN_OP_NORM_ROPE_BWD, total_tokens, 0, 0);
  if (!workspace || workspace_bytes < need)
    return fail(GDN_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                workspace ? workspace_bytes : (size_t)0);
  if (!aligned16(workspace)) return fail(GDN_ERR_INVALID_ARG, "%s: workspace is not 16-byte aligned", fn);
  a.partial = (float*)workspace;
  GDN_ATTN_DISPATCH(*shape, run_norm_bwd, a, norm_bwd_groups(*shape, total_tokens), dw_q, dw_k, (hipStream_t)stream);
  return launch_status(fn);
}

// ---------------------------------------------------------------------------
// attention

namespace {

// work items of the append: room for every block that the tokens can touch
int64_t touched_blocks(int32_t N, int64_t T) { return T / kBlock + 2 * (int64_t)N; }

// Records of k_attn_rows: `rec_bytes` of them behind `off`.
struct RowsLayout {
  size_t base, total_word, rec, rec_bytes, total;
};

RowsLayout rows_layout(size_t off, int32_t N, size_t rec_bytes) {
  RowsLayout L;
  L.base = off;
  off = align_up(off + sizeof(int32_t) * (size_t)N);
  L.total_word = off;
  off = align_up(off + sizeof(int32_t));
  L.rec = off;
  L.rec_bytes = align_up(rec_bytes) + 256;
  L.total = off + L.rec_bytes;
  return L;
}

// bytes of one partition's records: `rows` rows of each key/value head
size_t record_bytes(const gdn_attn_shape& s, int rows) {
  return (size_t)kv_heads(s) * rows * (s.head_dim + 2) * sizeof(float);
}

// A pool of num_blocks has num_blocks / 8 partitions, and one more per
// sequence, unless sequences share blocks.
int64_t pool_parts(int32_t N, int32_t num_blocks) { return (int64_t)num_blocks / kPartBlocks + (1 + kChunkCost) * (int64_t)N; }

// Decode: a chunk is up to 16 of a key/value head's query heads.
int decode_rows(const gdn_attn_shape& s) { return std::min(16, s.num_heads / kv_heads(s)); }

RowsLayout decode_layout(const gdn_attn_shape& s, int32_t N, int32_t num_blocks) {
  const int chunks = (s.num_heads / kv_heads(s) + 15) / 16;
  return rows_layout(0, N, (size_t)pool_parts(N, num_blocks) * chunks * record_bytes(s, decode_rows(s)));
}

// Prefill by k_attn_rows: rows of a chunk.  d = 256 has registers for one
// 16-row tile; with 64 rows, four tiles, the others spilled (16 x 37 new tokens
// after 5,000, 4 query heads to each of 8: 130 us instead of 116 at d = 64, 291 instead of 177 at 128).
int chunk_rows(const gdn_attn_shape& s, int64_t rows) { return s.head_dim == 256 || rows <= 16 ? 16 : 32; }

// Prefill takes k_attn_rows, which splits the keys and reads them once per
// chunk, if the batch has no more chunks than this, each sequence counted with the
// most rows of any, or a sequence one only; else k_attn_prefill, which splits rows
// only, 256 to a work-group.  Turns of 64 tokens (d = 256: 32) after 5,000, k_attn_rows /
// k_attn_prefill in us, by chunks:
//                                     256        512        640        768       1,024
//   d = 64,  4 query heads to each of 8   67 / 132   86 / 133  118 / 133  132 / 135  153 / 135
//   d = 128, the same                     85 / 178  137 / 178  175 / 177  193 / 181  241 / 181
//   d = 256, 8 to each of 2              108 / 215  210 / 215  264 / 215  302 / 217  393 / 220
// One bound for all: the two are even at about 780 chunks at d = 64, 650 at 128 and 530 at
// 256, so batches of 530 to 640 at d = 256 take the slower one (by up to 23 %).  How full the
// chunks and tiles are moves these by some per cent (37 tokens, 640 chunks: d = 64
// 116 / 129, d = 128 174 / 171).
constexpr int kMostChunks = 640;

bool takes_rows(const gdn_attn_shape& s, int32_t N, int64_t rows) {
  const int chunk = chunk_rows(s, rows);
  const int64_t chunks = (rows + chunk - 1) / chunk;
  return chunks <= 1 || N * (int64_t)kv_heads(s) * chunks <= kMostChunks;
}

// Its records, as far as this bound (beyond, chunks go to work-groups whole).
constexpr size_t kFewRecordBytes = size_t(512) << 20;

int tile_rows(const gdn_attn_shape& s) {
  return s.head_dim == 64 ? PrefillTile<64>::kRows : s.head_dim == 128 ? PrefillTile<128>::kRows : PrefillTile<256>::kRows;
}

// k_attn_prefill's row tiles of a key/value head: every sequence's last may be short, and one in excess
int64_t row_tiles(const gdn_attn_shape& s, int32_t N, int64_t T) { return T * (s.num_heads / kv_heads(s)) / tile_rows(s) + N; }

struct PrefillLayout {
  size_t old_k, old_v, bad, order, raw_k, raw_v;
  RowsLayout rows;
  size_t total;
};

PrefillLayout prefill_layout(const gdn_attn_shape& s, int32_t N, int64_t T, int32_t num_blocks) {
  const size_t block = (size_t)kv_heads(s) * kBlock * s.head_dim * sizeof(uint16_t);
  PrefillLayout L{};
  size_t off = 0;
  L.old_k = off;
  off = align_up(off + N * block);
  L.old_v = off;
  off = align_up(off + N * block);
  L.bad = off;
  off = align_up(off + (size_t)touched_blocks(N, T) * kv_heads(s) * sizeof(int32_t));
  L.order = off;
  off = align_up(off + sizeof(i32x2) * (size_t)row_tiles(s, N, T));
  const int64_t G = s.num_heads / kv_heads(s);
  if (N > 0 && takes_rows(s, N, (T * G + N - 1) / N)) {  // it may, if no sequence has many more than the others
    const int chunk = chunk_rows(s, 32);
    const int64_t most = std::max<int64_t>(1, kMostChunks / (N * (int64_t)kv_heads(s)));
    const size_t chunks = (size_t)std::min(most, (T * G + chunk - 1) / chunk);
    L.raw_k = off;
    off = align_up(off + (size_t)touched_blocks(N, T) * block);
    L.raw_v = off;
    off = align_up(off + (size_t)touched_blocks(N, T) * block);
    L.rows = rows_layout(off, N, std::min(kFewRecordBytes, (size_t)pool_parts(N, num_blocks) * chunks * record_bytes(s, chunk)));
    off = L.rows.total;
  }
  L.total = off;
  return L;
}

gdn_status check_step(const char* fn, const gdn_attn_step* step, const gdn_attn_cache* cache) {
  if (!step) return fail(GDN_ERR_INVALID_ARG, "%s: step is NULL", fn);
  if (!cache) return fail(GDN_ERR_INVALID_ARG, "%s: cache is NULL", fn);
  CHECK_PTR(step->block_table, "step.block_table");
  CHECK_OPT_PTR(step->slot_index, "step.slot_index");
  CHECK_PTR(cache->k8, "cache.k8");
  CHECK_PTR(cache->v8, "cache.v8");
  CHECK_PTR(cache->k_scale, "cache.k_scale");
  CHECK_PTR(cache->v_scale, "cache.v_scale");
  CHECK_PTR(cache->tail_k, "cache.tail_k");
  CHECK_PTR(cache->tail_v, "cache.tail_v");
  if (step->max_blocks < 1 || step->num_slots < 1 || cache->num_blocks < 1 || cache->num_slots < 1)
    return fail(GDN_ERR_INVALID_ARG, "%s: step and cache sizes must be positive", fn);
  if (step->num_slots != cache->num_slots)
    return fail(GDN_ERR_INVALID_ARG, "%s: the step's table has %d rows, the cache %d", fn, step->num_slots, cache->num_slots);
  return GDN_OK;
}

void fill_cache(StepArgs& s, const gdn_attn_shape& shape, int32_t N, int64_t T, const gdn_attn_step& step,
                const gdn_attn_cache& cache) {
  s.ctx_len = step.ctx_len;
  s.table = step.block_table;
  s.slot = step.slot_index;
  s.max_blocks = step.max_blocks;
  s.N = N;
  s.T = (int)T;
  s.H = shape.num_heads;
  s.Hk = kv_heads(shape);
  s.G = s.H / s.Hk;
  s.cache.k8 = cache.k8;
  s.cache.v8 = cache.v8;
  s.cache.k_scale = cache.k_scale;
  s.cache.v_scale = cache.v_scale;
  s.cache.tail_k = (uint16_t*)cache.tail_k;
  s.cache.tail_v = (uint16_t*)cache.tail_v;
  s.cache.num_blocks = cache.num_blocks;
  s.cache.num_slots = cache.num_slots;
}

// Checks shared by prefill and decode; fills everything but cu, the old tails and records.
gdn_status check_attention(const char* fn, const gdn_attn_shape* shape, int32_t N, int64_t T, const void* q,
                           const void* k, const void* v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                           const gdn_attn_step* step, const gdn_attn_cache* cache, float scale, void* o, StepArgs* a) {
  CHECK(check_shape(fn, shape));
  if (shape->dtype != GDN_DTYPE_BF16) return fail(GDN_ERR_UNSUPPORTED, "%s: attention takes bf16", fn);
  CHECK(check_sizes(fn, N, T));
  if (T * shape->num_heads > INT32_MAX) return fail(GDN_ERR_UNSUPPORTED, "%s: too many rows", fn);
  CHECK(check_step(fn, step, cache));
  if (!(scale > 0.f) || std::isinf(scale)) return fail(GDN_ERR_INVALID_ARG, "%s: scale must be positive and finite", fn);
  if (N == 0 && T > 0) return fail(GDN_ERR_INVALID_ARG, "%s: tokens without sequences", fn);
  const int64_t d = shape->head_dim;
  CHECK(check_stride(fn, "q_stride", q_stride, shape->num_heads * d, &a->q_stride));
  CHECK(check_stride(fn, "k_stride", k_stride, kv_heads(*shape) * d, &a->k_stride));
  CHECK(check_stride(fn, "v_stride", v_stride, kv_heads(*shape) * d, &a->v_stride));
  if (N > 0) CHECK_PTR(step->ctx_len, "step.ctx_len");
  if (T > 0) {
    CHECK_PTR(q, "q");
    CHECK_PTR(k, "k");
    CHECK_PTR(v, "v");
    CHECK_PTR(o, "o");
  }
  a->q = (const uint16_t*)q;
  a->k = (const uint16_t*)k;
  a->v = (const uint16_t*)v;
  a->o = (uint16_t*)o;
  a->c = scale * 1.44269504088896340736f;
  fill_cache(*a, *shape, N, T, *step, *cache);
  return GDN_OK;
}

gdn_status check_workspace(const char* fn, const void* workspace, size_t bytes, size_t need) {
  if (!workspace || bytes < need)
    return fail(GDN_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, need, workspace ? bytes : (size_t)0);
  if (!aligned16(workspace)) return fail(GDN_ERR_INVALID_ARG, "%s: workspace is not 16-byte aligned", fn);
  return GDN_OK;
}

void place_records(RowsArgs& a, const RowsLayout& L, char* ws, const gdn_attn_shape& s, int chunk, int rows) {
  a.base = (int32_t*)(ws + L.base);
  a.total = (int32_t*)(ws + L.total_word);
  a.chunk_rows = chunk;
  a.rec_rows = rows;
  // 256 bytes for aligning the second array
  a.max_parts = (int)std::min<size_t>((L.rec_bytes - 256) / record_bytes(s, rows), INT32_MAX / 2);
  a.rec_ml = (float*)(ws + L.rec);
  a.rec_o = a.rec_ml + align_up((size_t)a.max_parts * a.s.Hk * rows * 2 * sizeof(float)) / sizeof(float);
}

template <int D, int RT, bool MULTI, bool STREAM>
gdn_status run_rows(const RowsArgs& a, int chunks, hipStream_t st, const char* fn) {
  const int W = std::max(1, std::min(256 * kRowsPerCu<D, MULTI> / a.s.Hk, a.max_parts));  // 256 CUs
  hipLaunchKernelGGL((k_attn_rows<D, RT, MULTI, STREAM>), dim3(W, a.s.Hk), dim3(256), 0, st, a);
  hipLaunchKernelGGL(k_attn_join<D>, dim3(a.s.N, a.s.Hk, (chunks * a.rec_rows + 3) / 4), dim3(256), 0, st, a, W);
  return launch_status(fn);
}

template <int D>
gdn_status run_decode(const RowsArgs& a, int chunks, hipStream_t st, const char* fn) {
  return chunks == 1 ? run_rows<D, 1, false, true>(a, chunks, st, fn) : run_rows<D, 1, false, false>(a, chunks, st, fn);
}

template <int D>
gdn_status run_prefill(const StepArgs& a, int64_t tiles, hipStream_t st, const char* fn) {
  typedef PrefillTile<D> P;
  hipLaunchKernelGGL((k_attn_append<D, false>), dim3((unsigned)touched_blocks(a.N, a.T) + 1, a.Hk), dim3(kAppendThreads<D>), 0, st, a);
  hipLaunchKernelGGL(k_attn_prefill<D>, dim3((unsigned)(tiles * a.Hk)), dim3(P::kThreads), 0, st, a);
  return launch_status(fn);
}

template <int D>
gdn_status run_few(const RowsArgs& a, int chunks, hipStream_t st, const char* fn) {
  hipLaunchKernelGGL((k_attn_append<D, true>), dim3((unsigned)touched_blocks(a.s.N, a.s.T), a.s.Hk), dim3(kAppendThreads<D>), 0, st, a.s);
  if constexpr (D == 256) {
    return chunks == 1 ? run_rows<D, 1, true, true>(a, chunks, st, fn) : run_rows<D, 1, true, false>(a, chunks, st, fn);
  } else {
    if (a.chunk_rows == 16) return run_rows<D, 1, true, true>(a, chunks, st, fn);  // one chunk, or it would be 32
    return chunks == 1 ? run_rows<D, 2, true, true>(a, chunks, st, fn) : run_rows<D, 2, true, false>(a, chunks, st, fn);
  }
}

}  // namespace

extern "C" gdn_status gdn_attn_prefill(const gdn_attn_shape* shape, int32_t num_seqs, int64_t total_tokens,
                                       int32_t max_new, const void* q, const void* k, const void* v, int64_t q_stride,
                                       int64_t k_stride, int64_t v_stride, const int32_t* cu_seqlens,
                                       const gdn_attn_step* step, const gdn_attn_cache* cache, float scale, void* o,
                                       void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "gdn_attn_prefill";
  StepArgs a{};
  CHECK(check_attention(fn, shape, num_seqs, total_tokens, q, k, v, q_stride, k_stride, v_stride, step, cache, scale, o, &a));
  if (max_new < 0) return fail(GDN_ERR_INVALID_ARG, "%s: max_new is negative", fn);
  CHECK_PTR(cu_seqlens, "cu_seqlens");
  if (total_tokens == 0) return done();
  const PrefillLayout L = prefill_layout(*shape, num_seqs, total_tokens, cache->num_blocks);
  CHECK(check_workspace(fn, workspace, workspace_bytes, L.total));
  char* ws = (char*)workspace;
  a.cu = cu_seqlens;
  a.old_k = (uint16_t*)(ws + L.old_k);
  a.old_v = (uint16_t*)(ws + L.old_v);
  a.bad = (int32_t*)(ws + L.bad);
  const int64_t most = (int64_t)(max_new > 0 ? std::min<int64_t>(max_new, total_tokens) : total_tokens) * a.G;
  if (L.rows.rec_bytes > 0 && takes_rows(*shape, num_seqs, most)) {
    RowsArgs ra{};
    a.raw_k = (uint16_t*)(ws + L.raw_k);
    a.raw_v = (uint16_t*)(ws + L.raw_v);
    ra.s = a;
    const int chunk = chunk_rows(*shape, most), chunks = (int)((most + chunk - 1) / chunk);
    place_records(ra, L.rows, ws, *shape, chunk, chunk);
    switch (shape->head_dim) {
      case 64: return run_few<64>(ra, chunks, (hipStream_t)stream, fn);
      case 128: return run_few<128>(ra, chunks, (hipStream_t)stream, fn);
      default: return run_few<256>(ra, chunks, (hipStream_t)stream, fn);
    }
  }
  a.order = (i32x2*)(ws + L.order);
  a.tile_rows = tile_rows(*shape);
  const int64_t tiles = row_tiles(*shape, num_seqs, total_tokens);
  switch (shape->head_dim) {
    case 64: return run_prefill<64>(a, tiles, (hipStream_t)stream, fn);
    case 128: return run_prefill<128>(a, tiles, (hipStream_t)stream, fn);
    default: return run_prefill<256>(a, tiles, (hipStream_t)stream, fn);
  }
}

extern "C" gdn_status gdn_attn_decode_step(const gdn_attn_shape* shape, int32_t num_seqs, const void* q, const void* k,
                                           const void* v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                           const gdn_attn_step* step, const gdn_attn_cache* cache, float scale,
                                           void* o, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "gdn_attn_decode_step";
  RowsArgs a{};
  CHECK(check_attention(fn, shape, num_seqs, num_seqs, q, k, v, q_stride, k_stride, v_stride, step, cache, scale, o, &a.s));
  if (num_seqs == 0) return done();
  const RowsLayout L = decode_layout(*shape, num_seqs, cache->num_blocks);
  CHECK(check_workspace(fn, workspace, workspace_bytes, L.total));
  place_records(a, L, (char*)workspace, *shape, 16, decode_rows(*shape));
  const int chunks = (a.s.G + 15) / 16;
  switch (shape->head_dim) {
    case 64: return run_decode<64>(a, chunks, (hipStream_t)stream, fn);
    case 128: return run_decode<128>(a, chunks, (hipStream_t)stream, fn);
    default: return run_decode<256>(a, chunks, (hipStream_t)stream, fn);
  }
}

extern "C" gdn_status gdn_attn_cache_read(const gdn_attn_shape* shape, int32_t num_seqs, int64_t total_tokens,
                                          const int32_t* cu_seqlens, const gdn_attn_step* step,
                                          const gdn_attn_cache* cache, void* k_out, void* v_out, void* stream) {
  const char* fn = "gdn_attn_cache_read";
  CHECK(check_shape(fn, shape));
  if (shape->dtype != GDN_DTYPE_BF16) return fail(GDN_ERR_UNSUPPORTED, "%s: attention takes bf16", fn);
  CHECK(check_sizes(fn, num_seqs, total_tokens));
  CHECK(check_step(fn, step, cache));
  CHECK_PTR(cu_seqlens, "cu_seqlens");
  if (total_tokens == 0) return done();
  if (num_seqs == 0) return fail(GDN_ERR_INVALID_ARG, "%s: tokens without sequences", fn);
  CHECK_PTR(k_out, "k_out");
  CHECK_PTR(v_out, "v_out");
  StepArgs a{};
  fill_cache(a, *shape, num_seqs, total_tokens, *step, *cache);
  a.cu = cu_seqlens;
  const dim3 grid((unsigned)touched_blocks(a.N, a.T), a.Hk);
  switch (shape->head_dim) {
    case 64:
      hipLaunchKernelGGL(k_attn_cache_read<64>, grid, dim3(256), 0, (hipStream_t)stream, a, (uint16_t*)k_out, (uint16_t*)v_out);
      break;
    case 128:
      hipLaunchKernelGGL(k_attn_cache_read<128>, grid, dim3(256), 0, (hipStream_t)stream, a, (uint16_t*)k_out, (uint16_t*)v_out);
      break;
    default:
      hipLaunchKernelGGL(k_attn_cache_read<256>, grid, dim3(256), 0, (hipStream_t)stream, a, (uint16_t*)k_out, (uint16_t*)v_out);
  }
  return launch_status(fn);
}

extern "C" size_t gdn_attn_workspace_size(const gdn_attn_shape* shape, int32_t op, int64_t total_tokens,
                                          int32_t num_seqs, int32_t num_blocks) {
  const std::string before = gdn_last_error_text();
  const bool ok = check_shape("gdn_attn_workspace_size", shape) == GDN_OK &&
                  check_sizes("gdn_attn_workspace_size", num_seqs, total_tokens) == GDN_OK && num_blocks >= 0;
  gdn_last_error_text() = before;  // a size query is no call
  if (!ok) return 0;
  if (op == GDN_ATTN_OP_PREFILL) return prefill_layout(*shape, num_seqs, total_tokens, num_blocks).total;
  if (op == GDN_ATTN_OP_DECODE) return decode_layout(*shape, num_seqs, num_blocks).total;
  if (op == GDN_ATTN_OP_NORM_ROPE_BWD)
    return align_up((size_t)norm_bwd_groups(*shape, total_tokens) * 2 * shape->head_dim * sizeof(float));
  return 0;
}
