"""Generation with a small hybrid stack: Gated DeltaNet layers and, every fourth,
softmax attention over the 8-bit paged cache.

    python examples/hybrid_generate.py

Random weights.  The prompts are prefilled in one packed batch, then tokens are
generated step by step: one block plan per step serves every attention layer.
At the end the prompts with what was generated are prefilled again, and the
hidden states of all generated positions are compared bit for bit.  The
projections are library products; they run on tiles of a fixed number of rows,
so that a row's bits do not depend on the batch it is in.
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bitwise_invariant_gated_amd as gdn  # noqa: E402

TILE = 64  # rows of a projection


def project(x, w):
    """x w, `TILE` rows at a time."""
    y = torch.empty((x.shape[0], w.shape[1]), dtype=x.dtype, device=x.device)
    for r in range(0, x.shape[0], TILE):
        part = x[r:r + TILE]
        n = part.shape[0]
        if n < TILE:
            part = torch.cat([part, part.new_zeros(TILE - n, x.shape[1])])
        y[r:r + n] = torch.mm(part, w)[:n]
    return y


def rms(x):
    return torch.nn.functional.rms_norm(x.float(), x.shape[-1:], eps=1e-6).to(x.dtype)


class DeltaNetLayer:
    def __init__(self, width, heads, d, rand):
        self.shape = gdn.LayerShape(heads, d, d, 64, torch.bfloat16)
        self.w_in, self.w_out = rand(width, heads * (3 * d + 2)), rand(heads * d, width)

    def begin(self, seqs, pool, dev):
        h, d = self.shape.num_heads, self.shape.head_dim_k
        self.cache = gdn.alloc_cache(self.shape, seqs, dev)
        self.h0 = torch.zeros((seqs, h, d, d), device=dev)

    def __call__(self, x, cu, plan, positions, decode):
        h, d, t = self.shape.num_heads, self.shape.head_dim_k, x.shape[0]
        q, k, v, g, b = project(x, self.w_in).split([h * d, h * d, h * d, h, h], -1)
        q, k = (torch.nn.functional.normalize(y.reshape(t, h, d).float(), dim=-1).bfloat16() for y in (q, k))
        v, g, b = v.reshape(t, h, d).contiguous(), -torch.nn.functional.softplus(g.float()), torch.sigmoid(b.float())
        g, b = g.bfloat16().contiguous(), b.bfloat16().contiguous()
        o = torch.empty_like(q)
        n = cu.numel() - 1
        if decode:
            ws = gdn.alloc_workspace(self.shape, n, 0, gdn.GDN_OP_DECODE, x.device)
            gdn.gdn_cpr_decode_step(self.shape, q, k, v, g, b, self.cache, o, ws)
        else:
            ws = gdn.alloc_workspace(self.shape, n, t, gdn.GDN_OP_PREFILL, x.device)
            gdn.gdn_cpr_prefill(self.shape, q, k, v, g, b, cu, self.h0, self.cache, o, ws)
        return project(o.reshape(t, -1), self.w_out)


class AttentionLayer:
    def __init__(self, width, heads, kv_heads, d, rand, dev, max_len):
        self.shape, self.rope = gdn.AttnShape(heads, kv_heads, d), gdn.AttnRope(d // 2)
        self.w_in, self.w_out = rand(width, (heads + 2 * kv_heads) * d), rand(heads * d, width)
        self.w_q, self.w_k = torch.ones(d, device=dev), torch.ones(d, device=dev)
        angle = torch.arange(max_len, device=dev)[:, None] * 1e4 ** (-torch.arange(d // 4, device=dev) / (d // 4))
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).contiguous()

    def begin(self, seqs, pool, dev):
        self.cache = gdn.alloc_attn_cache(self.shape, pool.free_blocks.numel(), seqs, dev)

    def __call__(self, x, cu, plan, positions, decode):
        s, t, n = self.shape, x.shape[0], cu.numel() - 1
        heads = project(x, self.w_in).view(t, -1, s.head_dim)  # q, k and v of a token side by side
        q, k, v = heads.split([s.num_heads, s.kv_heads, s.kv_heads], 1)
        gdn.gdn_attn_qk_norm_rope(s, self.rope, q, k, self.w_q, self.w_k, self.cos_sin, plan.positions, q, k)
        o = torch.empty((t, s.num_heads, s.head_dim), dtype=x.dtype, device=x.device)
        blocks = self.cache.k_scale.shape[0]
        if decode:
            ws = gdn.alloc_attn_workspace(s, gdn.GDN_ATTN_OP_DECODE, t, n, blocks, x.device)
            gdn.gdn_attn_decode_step(s, q, k, v, plan, self.cache, o, ws)
        else:
            ws = gdn.alloc_attn_workspace(s, gdn.GDN_ATTN_OP_PREFILL, t, n, blocks, x.device)
            gdn.gdn_attn_prefill(s, q, k, v, cu, plan, self.cache, o, ws)
        return project(o.reshape(t, -1), self.w_out)


class Model:
    def __init__(self, vocab=512, width=256, layers=8, heads=4, d=64, attn_heads=4, kv_heads=2, attn_d=128, seed=0,
                 max_len=4096, dev="cuda"):
        gen = torch.Generator(dev).manual_seed(seed)

        def rand(*shape):
            return (torch.randn(shape, generator=gen, device=dev) * shape[0] ** -0.5).bfloat16()

        self.dev, self.embed, self.head = dev, rand(vocab, width) * vocab ** 0.5, rand(width, vocab)
        self.layers = [AttentionLayer(width, attn_heads, kv_heads, attn_d, rand, dev, max_len) if i % 4 == 3
                       else DeltaNetLayer(width, heads, d, rand) for i in range(layers)]

    def begin(self, seqs, max_len):
        """Empty states and caches for `seqs` requests of up to max_len tokens."""
        width = -(-max_len // gdn.GDN_ATTN_BLOCK)
        self.pool = gdn.alloc_attn_pool(seqs, width, seqs * width, self.dev)
        for layer in self.layers:
            layer.begin(seqs, self.pool, self.dev)

    def step(self, tokens, lens, decode=False):
        """Hidden states of the given new tokens, lens[i] of request i, packed."""
        cu = torch.tensor([0] + list(lens), device=self.dev).cumsum(0).to(torch.int32)
        plan = gdn.alloc_attn_plan(self.pool, len(lens), tokens.numel())
        gdn.gdn_attn_plan(self.pool, cu, plan)
        x = self.embed[tokens]
        for layer in self.layers:
            x = x + layer(rms(x), cu, plan, plan.positions, decode)
        return x

    def next_tokens(self, hidden):
        return project(rms(hidden), self.head).argmax(-1)


def generate(model, prompts, steps):
    """(tokens [steps + 1, N], hidden states [steps, N, width] of all but the last) after the prompts."""
    lens = [p.numel() for p in prompts]
    model.begin(len(prompts), max(lens) + steps + 1)
    hidden = model.step(torch.cat(prompts), lens)
    last = torch.tensor(lens, device=model.dev).cumsum(0) - 1
    tokens, states = [model.next_tokens(hidden[last])], []
    for _ in range(steps):
        states.append(model.step(tokens[-1], [1] * len(prompts), decode=True))
        tokens.append(model.next_tokens(states[-1]))
    return torch.stack(tokens), torch.stack(states)


def main(lens=(5, 64, 200, 1), steps=70, **kw):
    model = Model(**kw)
    gen = torch.Generator(model.dev).manual_seed(1)
    prompts = [torch.randint(0, model.embed.shape[0], (n,), generator=gen, device=model.dev) for n in lens]
    tokens, states = generate(model, prompts, steps)
    assert torch.isfinite(states).all()
    # all of it again, as one prefill
    whole = [torch.cat([p, tokens[:steps, i]]) for i, p in enumerate(prompts)]
    total = [w.numel() for w in whole]
    model.begin(len(whole), max(total))
    again = torch.split(model.step(torch.cat(whole), total), total)
    for i, n in enumerate(lens):
        same = torch.equal(again[i][n:].view(torch.int16), states[:, i].contiguous().view(torch.int16))
        assert same, f"request {i}: prefill and decode differ"
    print(f"{len(lens)} requests, {steps} steps: decode == prefill bit for bit; first tokens {tokens[:4, 0].tolist()}")
    return tokens


if __name__ == "__main__":
    main()
