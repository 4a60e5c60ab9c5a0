/*
 * gdn_attn.h -- C ABI of the softmax-attention layer that hybrid models place
 * between Gated DeltaNet layers (gdn_cpr.h), for AMD Instinct MI355X (gfx950).
 *
 * Four things, in the order a step uses them:
 *   gdn_attn_plan            block tables and slot maps from request lengths
 *                            (once per step, shared by every layer);
 *   gdn_attn_qk_norm_rope    RMS norm of every head's q and k and the position
 *                            rotation in one pass, with its gradient;
 *   gdn_attn_prefill,        causal attention over a paged cache held in 8
 *   gdn_attn_decode_step     bits, for any number of new tokens per sequence
 *                            and for one each, appending them to the cache;
 *   gdn_attn_cache_read      the cached keys and values, written out.
 *
 * The cache's rule.  A sequence's tokens are cut into blocks of
 * GDN_ATTN_BLOCK = 64 by position.  A block is quantised once, when its last
 * token arrives: e4m3 (4 exponent bits, 3 of fraction, no infinities) with
 * one scale per (block, key/value head) for K and one for V.  Until then its
 * tokens stay in the input type, in the tail.  The query at position p reads
 *   - its own block, positions 64 floor(p / 64) .. p, in the input type, and
 *   - every earlier block in 8 bits.
 * So what a query reads depends on its position only, not on how the tokens
 * arrived (one prompt, several segments, one at a time), as the chunk
 * boundaries of the Gated DeltaNet layer do not; and the arithmetic is
 * ordered by position too (partitions of 512 keys folded left to right, 64
 * keys at a time inside them), so outputs are bit-identical between prefill
 * and decode and between a sequence run alone and packed with others.
 *
 * Scales are powers of two, 2^e with the least e >= -100 for which the
 * block's largest finite magnitude is at most 448 * 2^e.  Dividing by such a
 * scale is exact, so an element is rounded once, and its cached value is a
 * bf16 number.  e4m3 keeps its relative precision over 15 binades, so a
 * power of two instead of amax / 448 gives up at most one binade at the
 * bottom.  A finite magnitude past 240 * 2^120 (3.2e38; bf16 ends at 3.4e38)
 * is cached as that, since the next e4m3 value, 256, would be 2^128.  A NaN
 * or infinity is cached as NaN.
 *
 * Conventions: those of gdn_cpr.h (device pointers, 16-byte aligned; calls
 * only enqueue on `stream`; nothing is allocated; host-detectable errors
 * return a status before anything is enqueued; gdn_cpr_last_error describes
 * the last one).  Beyond these:
 *   - T tokens are packed, cu_seqlens int32 [N + 1] over them.
 *   - A token stride is the distance in elements between a tensor's tokens;
 *     the heads of a token are contiguous.  0 means heads * head_dim.  It is
 *     a multiple of 8 and at least heads * head_dim, so q, k and v may be read
 *     in place out of a projection that makes them in one row.
 *   - Device data (lengths, tables, positions) is the caller's to get right;
 *     the kernels keep their accesses inside the arrays where it is not:
 *     cu_seqlens are held to 0 .. T (the plan counts blocks by the lengths as
 *     they are, and holds what it writes per token), block ids to the pool,
 *     positions to the rotation table; a block that the table does not have
 *     is not written; an entry with more full blocks than max_blocks counts
 *     as refused.  Tokens outside [cu_seqlens[0], cu_seqlens[N]) belong to no
 *     sequence; nothing is read or written for them.
 */
#ifndef GDN_ATTN_H
#define GDN_ATTN_H

#include "gdn_cpr.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_ATTN_BLOCK 64

typedef enum { GDN_ATTN_OP_PREFILL = 0, GDN_ATTN_OP_DECODE = 1, GDN_ATTN_OP_NORM_ROPE_BWD = 2 } gdn_attn_op;

/* Layer shape (host struct). */
typedef struct {
  int32_t num_heads;    /* H: query heads */
  int32_t num_kv_heads; /* Hk: key/value heads; divides H, and query head h
                           reads key/value head h / (H / Hk).  0 means H */
  int32_t head_dim;     /* 64, 128 or 256 */
  int32_t dtype;        /* gdn_dtype of q, k, v, o, the tails and gradients;
                           attention takes GDN_DTYPE_BF16, norm and rotation
                           either */
} gdn_attn_shape;

/*
 * The block pool that all layers share (host struct of device arrays).
 *   block_table [num_slots, max_blocks] int32  the pool blocks of a cache row,
 *               in order of position; unused entries are -1
 *   blocks_held [num_slots] int32              how many of them are in use
 *   free_blocks [num_blocks] int32             a stack of free block ids
 *   free_count  [1] int32                      its height
 *   seq_len     [num_slots] int32              tokens in the cache, per row
 * A new pool has blocks_held = seq_len = 0, block_table = -1 and every id
 * once on the stack.
 */
typedef struct {
  int32_t* block_table;
  int32_t* blocks_held;
  int32_t* free_blocks;
  int32_t* free_count;
  int32_t* seq_len;
  int32_t num_slots;
  int32_t max_blocks;
  int32_t num_blocks;
} gdn_attn_pool;

/*
 * What a step's plan gives every layer (host struct of device arrays).
 *   ctx_len     [N] int32   tokens in the cache before the step; -1: the
 *               request was refused or its row is -1
 *   positions   [T] int32   every new token's position in its sequence
 *   slot_map    [T] int64   every new token's place in the pool, block *
 *               GDN_ATTN_BLOCK + offset; -1 in a request that has ctx_len -1
 *   status      [1] int32   requests refused for want of blocks
 *   block_table, max_blocks, num_slots   the pool's (the plan refuses others)
 *   slot_index  [N] int32 cache row of every batch entry, or NULL for row i.
 *               Rows are distinct within a call; -1 marks an entry that is
 *               only there to fill the batch.
 */
typedef struct {
  int32_t* ctx_len;
  int32_t* positions;
  int64_t* slot_map;
  int32_t* status;
  const int32_t* block_table;
  const int32_t* slot_index;
  int32_t max_blocks;
  int32_t num_slots;
} gdn_attn_step;

/*
 * One layer's cache (host struct of device arrays).
 *   k8      [num_blocks, Hk, d / 64, 64, 64] e4m3: half-open groups of 64
 *           dims, in each the block's 64 tokens, in each 64 dims
 *   v8      [num_blocks, Hk, d, 64] e4m3: per dim the block's 64 tokens
 *   k_scale, v_scale  [num_blocks, Hk] fp32 powers of two
 *   tail_k  [num_slots, Hk, 64, d], tail_v [num_slots, Hk, d, 64], input type:
 *           the tokens of the block that the row's last token is in (row or
 *           column position mod 64; the others are left as they were)
 */
typedef struct {
  uint8_t* k8;
  uint8_t* v8;
  float* k_scale;
  float* v_scale;
  void* tail_k;
  void* tail_v;
  int32_t num_blocks;
  int32_t num_slots;
} gdn_attn_cache;

/* Norm and rotation (host struct). */
typedef struct {
  int32_t rotary_dim;    /* leading dims of every head that are rotated; a
                            multiple of 8 up to head_dim, 0 for none */
  int32_t interleaved;   /* pairs (2i, 2i + 1) instead of (i, i + rotary_dim / 2) */
  int32_t zero_centered; /* the weights are stored as w - 1 */
  int32_t num_positions; /* rows of cos_sin */
  float eps;
} gdn_attn_rope;

/*
 * Block tables and slot maps for N requests with cu_seqlens[i + 1] -
 * cu_seqlens[i] new tokens each, on top of pool->seq_len.  A request that
 * needs more blocks than its row holds takes them off the top of the free
 * stack, in batch order; all it needs or none.  Request i is refused when it
 * needs blocks and the needs of requests 0 .. i together exceed what was
 * free, or its row of the table is too narrow.  A refused request keeps its
 * row as it was and has ctx_len -1.  Running the plan again with the same
 * lengths takes nothing more.
 *   advance  1: seq_len of every request that goes on grows by its new
 *            tokens (the usual case: the next step's plan continues from
 *            them).  0: seq_len is left to the caller.
 */
gdn_status gdn_attn_plan(const gdn_attn_pool* pool, int32_t num_seqs, int64_t total_tokens,
                         const int32_t* cu_seqlens, int32_t advance, const gdn_attn_step* step,
                         void* stream);

/*
 * Requests leave: the blocks of the N rows slot_index[i] (NULL: row i) go
 * back on the free stack, last request and last block first, so that a plan
 * right after gives them out in the same order; the rows are emptied (table
 * -1, blocks_held 0, seq_len 0).  Entries that are -1 are skipped, and so is
 * a row's second entry (which of the two counts is not defined).
 */
gdn_status gdn_attn_release(const gdn_attn_pool* pool, int32_t num_seqs, const int32_t* slot_index,
                            void* stream);

/* Bytes of workspace (host only; 0 for an invalid shape or op, or where the
 * op needs none).  num_blocks is the cache's; norm_rope_bwd reads only the
 * shape and total_tokens.  Decode has a record for every 512 tokens that the
 * pool can hold, 6 % of one layer's cache with 16 query heads to a key head;
 * one workspace serves all layers. */
size_t gdn_attn_workspace_size(const gdn_attn_shape* shape, int32_t op, int64_t total_tokens,
                               int32_t num_seqs, int32_t num_blocks);

/*
 * q, k -> q_out, k_out: with x a head's d values, r = rsqrt(mean(x^2) + eps)
 * and n = x r w (w_q or w_k, fp32 [d]), the pair (n1, n2) at position p
 * becomes (n1 c - n2 s, n2 c + n1 s); dims past rotary_dim stay n.
 *   cos_sin    [num_positions, rotary_dim] fp32: per position the rotary_dim
 *              / 2 cosines, then the sines
 *   positions  [T] int32 (the plan's); one outside the table gives NaN in
 *              the rotated dims
 *   q_out, k_out may be q and k themselves (same strides).
 * Everything is computed in fp32 and rounded once.  Unused with rotary_dim
 * 0: cos_sin and positions may be NULL.
 */
gdn_status gdn_attn_qk_norm_rope(const gdn_attn_shape* shape, const gdn_attn_rope* rope, int64_t total_tokens,
                                 const void* q, const void* k, int64_t q_stride, int64_t k_stride,
                                 const float* w_q, const float* w_k, const float* cos_sin,
                                 const int32_t* positions, void* q_out, void* k_out, int64_t q_out_stride,
                                 int64_t k_out_stride, void* stream);

/*
 * Its gradient: from d_q_out, d_k_out (of q_out, k_out) and the forward's
 * q, k, the gradients dq, dk (input type) and dw_q, dw_k (fp32 [d], over all
 * tokens and heads; 0 when there are none).  With dn the gradient rotated
 * back and xh = x r: dw = sum dn xh, dx = r (dn w - xh mean(dn w xh)).
 * The sums run in a fixed order that depends on the sizes only.
 * dq, dk may be d_q_out, d_k_out themselves (same strides).
 */
gdn_status gdn_attn_qk_norm_rope_bwd(const gdn_attn_shape* shape, const gdn_attn_rope* rope, int64_t total_tokens,
                                     const void* q, const void* k, int64_t q_stride, int64_t k_stride,
                                     const float* w_q, const float* w_k, const float* cos_sin,
                                     const int32_t* positions, const void* d_q_out, const void* d_k_out,
                                     int64_t dqo_stride, int64_t dko_stride, void* dq, void* dk,
                                     int64_t dq_stride, int64_t dk_stride, float* dw_q, float* dw_k,
                                     void* workspace, size_t workspace_bytes, void* stream);

/*
 * Attention of every sequence's new tokens over its cache and themselves
 * (causal), appending them: o = softmax(scale q k^T) v by the cache's rule.
 *   q [T, H, d], k, v [T, Hk, d]  with token strides; o [T, H, d] contiguous
 *   step      the plan's; every request's blocks up to its last token are in
 *             its table.  Tokens of an entry with ctx_len -1, or with a
 *             slot_index that is no row of the cache (whatever its ctx_len),
 *             get o = 0 and leave the cache alone.
 *   max_new   an upper bound of any sequence's new tokens (0: T); it chooses
 *             between kernels and changes no bits
 *   scale     positive and finite
 * Sums are fp32, of p v with p up to 2^8: where a weighted sum of |v| passes
 * 2^119 or so, o may be infinite though the exact mean is not.
 */
gdn_status gdn_attn_prefill(const gdn_attn_shape* shape, int32_t num_seqs, int64_t total_tokens, int32_t max_new,
                            const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                            int64_t v_stride, const int32_t* cu_seqlens, const gdn_attn_step* step,
                            const gdn_attn_cache* cache, float scale, void* o, void* workspace,
                            size_t workspace_bytes, void* stream);

/* The same with one new token for each of N sequences (T = N). */
gdn_status gdn_attn_decode_step(const gdn_attn_shape* shape, int32_t num_seqs, const void* q, const void* k,
                                const void* v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                const gdn_attn_step* step, const gdn_attn_cache* cache, float scale, void* o,
                                void* workspace, size_t workspace_bytes, void* stream);

/*
 * The cached keys and values of N rows, in the input type: k_out, v_out
 * [T, Hk, d] contiguous hold, packed by cu_seqlens, positions 0 .. of every
 * row; row i has cu_seqlens[i + 1] - cu_seqlens[i] tokens cached.  Full
 * blocks come out of their 8 bits, the open one out of the tail.
 * Rows -1 give zeros.  slot_index, block_table as in gdn_attn_step.
 */
gdn_status gdn_attn_cache_read(const gdn_attn_shape* shape, int32_t num_seqs, int64_t total_tokens,
                               const int32_t* cu_seqlens, const gdn_attn_step* step, const gdn_attn_cache* cache,
                               void* k_out, void* v_out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_ATTN_H */
