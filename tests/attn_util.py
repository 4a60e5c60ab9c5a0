"""Helpers of the attention layer's tests: seeded inputs and the layer's calls."""

from __future__ import annotations

import numpy as np
import torch

import bitwise_invariant_gated_amd as gdn

DEV = "cuda"


def bf16(rng, *shape, std=1.0):
    """Random bf16 values, as a CPU tensor."""
    return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).bfloat16()


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Layer:
    """A pool, one layer's cache and the calls on them, for sequences whose
    whole q, k, v are given: seqs[i] = (q, k, v) CPU bf16 tensors."""

    def __init__(self, h, hk, d, seqs, slots=None, extra_blocks=7, garbage=True, scale=None):
        self.shape = gdn.AttnShape(h, hk, d)
        self.seqs, self.scale = seqs, scale
        n = len(seqs)
        self.slots = list(range(n)) if slots is None else slots
        num_slots = max(self.slots + [0]) + 2
        width = max([-(-s[0].shape[0] // 64) for s in seqs] + [1]) + 1
        blocks = sum(-(-s[0].shape[0] // 64) for s in seqs) + extra_blocks
        self.pool = gdn.alloc_attn_pool(num_slots, width, blocks, DEV)
        self.cache = gdn.alloc_attn_cache(self.shape, blocks, num_slots, DEV)
        if garbage:  # nothing of what was there before may be read
            for t in (self.cache.k8, self.cache.v8):
                t.fill_(0x7f)
            for t in (self.cache.tail_k, self.cache.tail_v, self.cache.k_scale, self.cache.v_scale):
                t.fill_(float("nan"))
        self.done = [0] * n
        self.slot_index = torch.tensor(self.slots, dtype=torch.int32, device=DEV)

    def pack(self, take):
        """Device q, k, v and cu_seqlens of the next take[i] tokens of every sequence."""
        part = [[s[j][a:a + m] for s, a, m in zip(self.seqs, self.done, take)] for j in range(3)]
        cu = torch.tensor(np.concatenate([[0], np.cumsum(take)]), dtype=torch.int32, device=DEV)
        return [torch.cat(p).to(DEV).contiguous() for p in part], cu

    def plan(self, take, cu):
        plan = gdn.alloc_attn_plan(self.pool, len(take), sum(take), self.slot_index)
        gdn.gdn_attn_plan(self.pool, cu, plan)
        assert int(plan.status) == 0
        assert plan.ctx_len.tolist() == self.done
        return plan

    def prefill(self, take, max_new=0, o=None):
        """The next take[i] tokens of every sequence; list of their outputs."""
        (q, k, v), cu = self.pack(take)
        plan = self.plan(take, cu)
        o = torch.full_like(q, float("nan"))
        ws = gdn.alloc_attn_workspace(self.shape, gdn.GDN_ATTN_OP_PREFILL, sum(take), len(take),
                                      self.cache.k8.shape[0], DEV)
        gdn.gdn_attn_prefill(self.shape, q, k, v, cu, plan, self.cache, o, ws, scale=self.scale, max_new=max_new)
        self.done = [a + m for a, m in zip(self.done, take)]
        return list(torch.split(o, list(take)))

    def decode(self):
        take = [1] * len(self.seqs)
        (q, k, v), cu = self.pack(take)
        plan = self.plan(take, cu)
        o = torch.full_like(q, float("nan"))
        ws = gdn.alloc_attn_workspace(self.shape, gdn.GDN_ATTN_OP_DECODE, len(take), len(take),
                                      self.cache.k8.shape[0], DEV)
        gdn.gdn_attn_decode_step(self.shape, q, k, v, plan, self.cache, o, ws, scale=self.scale)
        self.done = [a + 1 for a in self.done]
        return list(torch.split(o, take))

    def read(self):
        """Cached keys and values of every sequence."""
        cu = torch.tensor(np.concatenate([[0], np.cumsum(self.done)]), dtype=torch.int32, device=DEV)
        plan = gdn.alloc_attn_plan(self.pool, len(self.done), 0, self.slot_index)
        k, v = gdn.gdn_attn_cache_read(self.shape, cu, sum(self.done), plan, self.cache)
        return list(torch.split(k, self.done)), list(torch.split(v, self.done))


def random_seqs(seed, lens, h, hk, d, q_std=1.5):
    rng = np.random.default_rng(seed)
    return [(bf16(rng, L, h, d, std=q_std), bf16(rng, L, hk, d), bf16(rng, L, hk, d)) for L in lens]


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


def tolerance(v) -> float:
    """Largest |o - exact|: p is rounded to bf16 (8 bits: 2^-8 of it at most, so
    2^-8 max|v| in the weighted mean) and so is o (2^-8 |o| <= 2^-8 max|v|);
    scores, exp2 and the fp32 sums add a few 2^-20 of max|v|, covered by the 5%."""
    return 1.05 * 2.0 ** -7 * float(np.abs(v[np.isfinite(v)]).max())


# long contexts of the tests on marked_seqs: heads, key/value heads, head dim, tokens
LONG = [(8, 2, 128, [9000, 2, 5200]), (2, 1, 128, [70000]), (2, 1, 64, [33087, 9000]), (4, 2, 256, [20000, 300])]
SHARED = (1, 1, 64, 20050)


def marked_seqs(seed, lens, h, hk, d):
    """Sequences in which every block shows in the output: V is zero but in dim
    (block mod d), where it is positive and of a size of its own, and the scores are
    even enough that no block's share of its dim is small.  The scales of K and V
    change from block to block."""
    rng = np.random.default_rng(seed)
    out = []
    for n in lens:
        block = np.arange(n) // 64
        k = rng.standard_normal((n, hk, d)) * 2.0 ** (block % 3 - 1)[:, None, None]
        v = np.zeros((n, hk, d))
        v[np.arange(n), :, block % d] = rng.uniform(0.5, 1.0, (n, hk)) * 2.0 ** (block % d % 5)[:, None]
        to = lambda x: torch.from_numpy(x.astype(np.float32)).bfloat16()  # noqa: E731
        out.append((bf16(rng, n, h, d, std=0.5), to(k), to(v)))
    return out


def error_bound(o, spread):
    """Largest |result - o|, element by element; spread: the same mean of |v|.  p is
    rounded to bf16, by 2^-8 = u of itself at most, in numerator and denominator alike:
    |sum p (1 + e) v / sum p (1 + e) - o| <= u / (1 - u) (spread + |o|).  The output's
    rounding: u of it.  Scores (d products in fp32, |terms| of some tens at most), exp2
    and the sums in fp32 change p by less than 2^-10."""
    u = 2.0 ** -8
    return (u / (1 - u) * (1 + u) + 2.0 ** -10) * (spread + np.abs(o)) + u * np.abs(o)


def expect_within(q, k, v, scale, first=0):
    """The oracle's o of the positions from `first` on, and error_bound."""
    from oracle import attention as ref

    q, k, v = (f64(x) for x in (q, k, v))
    o = ref.attention(q[first:], k, v, scale, first)
    spread = o if (v >= 0).all() else ref.attention(q[first:], k, np.abs(v), scale, first)
    return o, error_bound(o, spread)
