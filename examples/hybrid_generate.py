"""Generation with a small hybrid stack: Gated DeltaNet layers and, every fourth,
softmax attention over the 8-bit paged cache.

    python examples/hybrid_generate.py

Random weights.  The prompts are prefilled in one packed batch, then tokens are
generated step by step: one block plan per step serves every attention layer,
one call between two layers adds to the residual stream and norms it, and one
call after the last gives the best tokens with their log probabilities.
At the end the prompts with what was generated are prefilled again, as a trainer
would: the hidden states of all generated positions and the log probabilities of
their tokens are compared bit for bit, and the divergence of the trainer's
distributions from the alternatives that generation noted is exactly 0.  The
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


def same_bits(a, b):
    view = torch.int16 if a.element_size() == 2 else torch.int32
    return torch.equal(a.contiguous().view(view), b.contiguous().view(view))


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
        self.norm, self.weights = gdn.NormShape(width), torch.ones((layers + 1, width), device=dev)
        self.layers = [AttentionLayer(width, attn_heads, kv_heads, attn_d, rand, dev, max_len) if i % 4 == 3
                       else DeltaNetLayer(width, heads, d, rand) for i in range(layers)]

    def begin(self, seqs, max_len):
        """Empty states and caches for `seqs` requests of up to max_len tokens."""
        width = -(-max_len // gdn.GDN_ATTN_BLOCK)
        self.pool = gdn.alloc_attn_pool(seqs, width, seqs * width, self.dev)
        for layer in self.layers:
            layer.begin(seqs, self.pool, self.dev)

    def step(self, tokens, lens, decode=False):
        """The residual stream after the last layer and its norm for the given new tokens, lens[i] of
        request i, packed."""
        cu = torch.tensor([0] + list(lens), device=self.dev).cumsum(0).to(torch.int32)
        plan = gdn.alloc_attn_plan(self.pool, len(lens), tokens.numel())
        gdn.gdn_attn_plan(self.pool, cu, plan)
        x = self.embed[tokens]
        y = torch.empty_like(x)
        gdn.gdn_stack_add_norm(self.norm, x, None, self.weights[0], None, y)
        for layer, w in zip(self.layers, self.weights[1:]):
            gdn.gdn_stack_add_norm(self.norm, layer(y, cu, plan, plan.positions, decode), x, w, x, y)
        return x, y

    def score(self, y, targets=None, top=0):
        """(logits, log probabilities of the targets, entropy, ids and log probabilities of the best
        tokens, statistics) of every row."""
        logits = project(y, self.head)
        t, dev = logits.shape[0], self.dev
        shape = gdn.LogitsShape(self.head.shape[1], top=top)
        logprobs = None if targets is None else torch.empty(t, device=dev)
        entropy, stats = torch.empty(t, device=dev), torch.empty((t, 2), device=dev)
        ids, best = torch.empty((t, top), dtype=torch.int32, device=dev), torch.empty((t, top), device=dev)
        gdn.gdn_stack_logprobs(shape, logits, targets, logprobs, entropy, ids if top else None, best if top else None, stats,
                               gdn.alloc_logits_workspace(shape, t, dev))
        return logits, logprobs, entropy, ids, best, stats

    def head_gradients(self, x, y, targets, g):
        """Gradients of sum g log p(targets) with respect to the stream x, the last norm's weights and
        the head, from step's outputs."""
        logits, _, entropy, _, _, stats = self.score(y, targets)
        gdn.gdn_stack_logprobs_bwd(gdn.LogitsShape(logits.shape[1]), logits, targets, stats, entropy, g, None, logits)
        dx, dw = torch.empty_like(x), torch.empty_like(self.weights[-1])
        gdn.gdn_stack_add_norm_bwd(self.norm, x, self.weights[-1], logits @ self.head.t(), None, dx, None, dw,
                                   gdn.alloc_norm_workspace(self.norm, x.shape[0], self.dev))
        return dx, dw, y.t() @ logits


def generate(model, prompts, steps, top=8):
    """After the prompts: tokens [steps + 1, N], the stream [steps, N, width] at all but the last, and
    of every token the ids and log probabilities of the best, its own first."""
    lens = [p.numel() for p in prompts]
    model.begin(len(prompts), max(lens) + steps + 1)
    last = torch.tensor(lens, device=model.dev).cumsum(0) - 1
    y, states, ids, best = model.step(torch.cat(prompts), lens)[1][last], [], [], []
    for i in range(steps + 1):
        _, _, _, k, lp, _ = model.score(y, top=top)
        ids.append(k)
        best.append(lp)
        if i < steps:
            x, y = model.step(k[:, 0].long(), [1] * len(prompts), decode=True)
            states.append(x)
    ids = torch.stack(ids)
    return ids[:, :, 0].long(), torch.stack(states), ids, torch.stack(best)


def main(lens=(5, 64, 200, 1), steps=70, **kw):
    model = Model(**kw)
    gen = torch.Generator(model.dev).manual_seed(1)
    prompts = [torch.randint(0, model.embed.shape[0], (n,), generator=gen, device=model.dev) for n in lens]
    tokens, states, ids, best = generate(model, prompts, steps)
    assert torch.isfinite(states).all() and torch.isfinite(best).all()
    # all of it again, as one prefill
    whole = [torch.cat([p, tokens[:steps, i]]) for i, p in enumerate(prompts)]
    total = [w.numel() for w in whole]
    model.begin(len(whole), max(total))
    x, y = model.step(torch.cat(whole), total)
    for i, (n, hidden, normed) in enumerate(zip(lens, torch.split(x, total), torch.split(y, total))):
        assert same_bits(hidden[n:], states[:, i]), f"request {i}: prefill and decode differ"
        # position n - 1 + j gives token j
        logits, logprobs, _, _, _, _ = model.score(normed[n - 1:], tokens[:, i].to(torch.int32).contiguous())
        assert same_bits(logprobs, best[:, i, 0]), f"request {i}: log probabilities differ"
        shape = gdn.LogitsShape(logits.shape[1], top=ids.shape[2], teacher_logprobs=True)
        loss = torch.empty_like(logprobs)
        gdn.gdn_stack_distill(shape, logits, ids[:, i].contiguous(), best[:, i].contiguous(), loss, None,
                              gdn.alloc_logits_workspace(shape, loss.numel(), model.dev))
        assert (loss == 0).all(), f"request {i}: divergence {loss.max()}"
    print(f"{len(lens)} requests, {steps} steps: decode == prefill bit for bit, states, log probabilities and {ids.shape[2]} "
          f"alternatives; first tokens {tokens[:4, 0].tolist()}")
    return tokens


if __name__ == "__main__":
    main()
