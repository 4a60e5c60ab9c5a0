// Block tables and slot maps from request lengths, and their release.
//
// The plan is two prefix sums over the requests (blocks needed, blocks taken)
// and a flat pass over the blocks and the tokens that they describe.  Its
// bytes are few (12 per token, 24 per request), so what bounds it is latency:
// one work-group does the sums, in registers and LDS, and up to
// kTokensInPlan tokens as well; more tokens go to a second launch of as many
// work-groups as they fill, because one CU writes only a few bytes per cycle
// (64 requests, a call: 4,096 tokens 7.1 us in one launch, 8.4 in two; 16,000 tokens 14.8 and
// 8.6).
#pragma once

#include "attn_device.hpp"

namespace attn {

struct PlanArgs {
  int32_t *table, *held, *free, *free_count, *seq_len;
  int num_slots, max_blocks, num_blocks;
  int N, T, advance, tokens_here;
  const int32_t *cu, *slot;
  int32_t *ctx_len, *positions, *status;
  int64_t* slot_map;
};

constexpr int kPlanThreads = 1024;
constexpr int kTokensInPlan = 4096;

// Inclusive prefix sum over the work-group's threads; *total gets the sum.
// Adds saturate at INT32_MAX (associative for what is not negative).
__device__ __forceinline__ int sat_add(int a, int b) {
  const uint32_t s = (uint32_t)a + (uint32_t)b;
  return s > 0x7fffffffu ? 0x7fffffff : (int)s;
}

__device__ __forceinline__ int block_scan(int x, int* wave_sums, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(x, o);
    if (lane >= o) x = sat_add(x, y);
  }
  __syncthreads();  // the sums of the scan before have been read
  if (lane == 63) wave_sums[wave] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 64; ++w) {
    const int s = wave_sums[w];
    if (w < wave) before = sat_add(before, s);
    all = sat_add(all, s);
  }
  *total = all;
  return sat_add(before, x);
}

// the first index of the inclusive prefix sums s[0 .. n) above j
__device__ __forceinline__ int first_above(const int* s, int n, int j) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (s[mid] > j)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

__device__ __forceinline__ void write_token(const PlanArgs& a, int t, int pos, int row, bool on) {
  a.positions[t] = pos;
  int64_t place = -1;
  const int col = pos >> 6;
  if (on && col >= 0 && col < a.max_blocks) {
    const int id = a.table[(size_t)row * a.max_blocks + col];
    if (id >= 0) place = (int64_t)id * kBlock + (pos & (kBlock - 1));
  }
  a.slot_map[t] = place;
}

__global__ __launch_bounds__(kPlanThreads) void k_attn_plan(const PlanArgs a) {
  __shared__ int s_take[kPlanThreads], s_held[kPlanThreads], s_row[kPlanThreads], s_ctx[kPlanThreads];
  __shared__ int s_cu[kPlanThreads + 1], s_sums[kPlanThreads / 64], s_refused;
  const int tid = threadIdx.x;
  const int there = min(max(*a.free_count, 0), a.num_blocks);
  int needed = 0, taken = 0;
  if (tid == 0) s_refused = 0;
  for (int base = 0; base < a.N; base += kPlanThreads) {
    const int i = base + tid, n = min(kPlanThreads, a.N - base);
    int row = -1, ctx = 0, held = 0, len = 0, want = 0, need = 0;
    bool fine = false;
    if (i < a.N) {
      const int c0 = a.cu[i], c1 = a.cu[i + 1];
      s_cu[tid] = c0;
      if (tid == n - 1) s_cu[n] = c1;
      len = c1 - c0;
      row = row_of(a.slot, i, a.num_slots);
      if (row >= 0) {
        ctx = a.seq_len[row];
        held = a.held[row];
        fine = len >= 0 && ctx >= 0 && held >= 0 && held <= a.max_blocks && ctx <= 0x7fffffff - kBlock - len;
        if (fine) {
          want = (ctx + len + kBlock - 1) >> 6;
          need = max(want - held, 0);
        }
      }
    }
    int chunk_need, chunk_take;
    const int upto = sat_add(needed, block_scan(need, s_sums, &chunk_need));
    const bool ok = fine && (need == 0 || (upto <= there && want <= a.max_blocks));
    const int take = ok ? need : 0;
    s_take[tid] = block_scan(take, s_sums, &chunk_take);
    s_held[tid] = held;
    s_row[tid] = row;
    s_ctx[tid] = ok ? ctx : -1 - max(ctx, 0);  // below 0: not going on
    if (i < a.N) {
      a.ctx_len[i] = ok ? ctx : -1;
      if (take) a.held[row] = held + take;
      if (ok && a.advance) a.seq_len[row] = ctx + len;
      if (row >= 0 && !ok) atomicAdd(&s_refused, 1);
    }
    __syncthreads();
    // the blocks taken, off the top of the stack in request order
    for (int j = tid; j < chunk_take; j += kPlanThreads) {
      const int r = first_above(s_take, n, j);
      const int col = s_held[r] + j - (r ? s_take[r - 1] : 0);
      a.table[(size_t)s_row[r] * a.max_blocks + col] = a.free[there - 1 - taken - j];
    }
    if (a.tokens_here) {
      __syncthreads();
      for (int t = max(s_cu[0], 0) + tid; t < min(s_cu[n], a.T); t += kPlanThreads) {
        const int r = seq_of(s_cu, n, t);
        const bool on = s_ctx[r] >= 0;
        const int from = on ? s_ctx[r] : -1 - s_ctx[r];
        write_token(a, t, from + t - s_cu[r], s_row[r], on);
      }
    }
    needed = sat_add(needed, chunk_need);
    taken += chunk_take;
    __syncthreads();  // the LDS arrays are written again for the next requests
  }
  if (tid == 0) {
    if (taken) *a.free_count = there - taken;
    *a.status = s_refused;
  }
}

// Tokens of a large plan: a thread each.  Those outside every request are left alone, as above.
__global__ __launch_bounds__(256) void k_attn_plan_tokens(const PlanArgs a) {
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t >= a.T || t < a.cu[0] || t >= a.cu[a.N]) return;
  const int i = seq_of(a.cu, a.N, t);
  const int row = row_of(a.slot, i, a.num_slots);
  const int ctx = a.ctx_len[i];
  const bool on = ctx >= 0;
  const int from = on ? ctx : row >= 0 ? max(a.seq_len[row], 0) : 0;
  write_token(a, t, from + t - a.cu[i], row, on);
}

struct ReleaseArgs {
  int32_t *table, *held, *free, *free_count, *seq_len;
  int num_slots, max_blocks, num_blocks, N;
  const int32_t* slot;
};

__global__ __launch_bounds__(kPlanThreads) void k_attn_release(const ReleaseArgs a) {
  __shared__ int s_upto[kPlanThreads], s_row[kPlanThreads], s_sums[kPlanThreads / 64];
  const int tid = threadIdx.x;
  int top = min(max(*a.free_count, 0), a.num_blocks);
  for (int base = 0; base < a.N; base += kPlanThreads) {
    const int n = min(kPlanThreads, a.N - base), i = a.N - 1 - base - tid;  // from the last request on
    int row = -1, held = 0, total;
    if (tid < n) {
      row = row_of(a.slot, i, a.num_slots);
      // exchanged, so that a row named twice gives its blocks back once
      if (row >= 0) held = min(max(atomicExch(&a.held[row], 0), 0), a.max_blocks);
    }
    s_upto[tid] = block_scan(held, s_sums, &total);
    s_row[tid] = row;
    if (row >= 0) a.seq_len[row] = 0;
    __syncthreads();
    for (int j = tid; j < total; j += kPlanThreads) {
      const int r = first_above(s_upto, n, j);
      int32_t* e = a.table + (size_t)s_row[r] * a.max_blocks + (s_upto[r] - 1 - j);  // its last block first
      if (top + j < a.num_blocks) a.free[top + j] = *e;
      *e = -1;
    }
    top = min(sat_add(top, total), a.num_blocks);
    __syncthreads();
  }
  if (tid == 0) *a.free_count = top;
}

}  // namespace attn
