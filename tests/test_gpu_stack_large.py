"""GPU tests of calls that move more than the caches hold: what is read and written past them has
the bits of the same rows in small calls, in place too."""

import pytest
import torch

import bitwise_invariant_gated_amd as gdn
from gpu_util import note
from stack_util import DEV, NORM, add_norm, add_norm_bwd, distill, distill_bwd, logprobs, logprobs_bwd, same_bits

pytestmark = pytest.mark.gpu

B, F = torch.bfloat16, torch.float32
MB = 1 << 20


def randn(*shape, dtype=F, seed=0):
    g = torch.Generator(DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


@pytest.mark.parametrize("w", [128, 1000, 2048, 4096, 8200, 16384])
@pytest.mark.parametrize("types", [(B, B), (B, F), (F, F)])
def test_norm(w, types):
    dt, rdt = types
    t = 130 * MB // (4 * w) + 3  # at least 96 MB in every type
    note(f"large add_norm {t} x {w} {types}")
    s = gdn.NormShape(w, dt, rdt, 0)
    x, res, dy, dr, wt = randn(t, w, dtype=dt), randn(t, w, dtype=rdt, seed=1), randn(t, w, dtype=dt, seed=2), randn(t, w, dtype=rdt, seed=3), randn(w, seed=4)
    h, y, y8, sc = add_norm(s, x, res, wt)
    dx, dd, dw = add_norm_bwd(s, h, wt, dy, dr, both=True)
    for a in (0, t // 2, t - 5):
        one = slice(a, a + 5)
        assert all(same_bits(p, q[one]) for p, q in zip(add_norm(s, x[one].clone(), res[one].clone(), wt), (h, y, y8, sc)))
        got = add_norm_bwd(s, h[one].clone(), wt, dy[one].clone(), dr[one].clone(), both=True)
        assert same_bits(got[0], dx[one]) and same_bits(got[1], dd[one])
    # dw, of as many rows: each row's share is off by 4 NORM of itself at most, as is their sum
    n = h.double() * torch.rsqrt(h.double().square().mean(-1, keepdim=True) + s.eps)
    share = dy.double() * n
    assert ((dw.double() - share.sum(0)).abs() <= 4 * NORM * share.abs().sum(0)).all()
    only = torch.full_like(dx, float("nan"))
    gdn.gdn_stack_add_norm_bwd(s, h, wt, dy, dr, only, None, dw, gdn.alloc_norm_workspace(s, t, DEV))
    assert same_bits(only, dx)
    gdn.gdn_stack_add_norm_bwd(s, h, wt, dy, dr, dy, h, dw, gdn.alloc_norm_workspace(s, t, DEV))
    assert same_bits(dy, dx) and same_bits(h, dd)
    gdn.gdn_stack_add_norm(s, x, res, wt, res, x)
    assert same_bits(x, y)


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("v", [900, 5000, 50001, 131072])
def test_logits(v, dtype):
    t = 110 * MB // (2 * v) + 3
    note(f"large logits {t} x {v} {dtype}")
    x = randn(t, v, dtype=dtype)
    x *= 3
    x[::3, v // 2:] = -float("inf")
    g = torch.Generator(DEV).manual_seed(5)
    target = torch.randint(-v // 8, v // 2, (t,), generator=g, device=DEV).to(torch.int32)
    scale, up = 0.5 + torch.rand(t, generator=g, device=DEV), randn(t, seed=6)
    few = torch.randint(0, v, (t, 9), generator=g, device=DEV).to(torch.int32)
    values = randn(t, 9, seed=7)
    s = gdn.LogitsShape(v, dtype, 9)
    o = logprobs(s, x, target, scale)
    lean = logprobs(s, x, target, scale, entropy=False)
    bare = logprobs(gdn.LogitsShape(v, dtype), x, target, scale, entropy=False)
    for n in ("logprobs", "stats", "top_ids", "top_logprobs"):
        assert same_bits(getattr(lean, n), getattr(o, n))
    assert same_bits(bare.logprobs, o.logprobs) and same_bits(bare.stats, o.stats)
    loss, stats = distill(s, x, few, values, scale)
    d1, d2 = logprobs_bwd(s, x, target, o, up, up, scale), distill_bwd(s, x, few, values, stats, up, scale)
    lone = logprobs_bwd(s, x, target, o, up, None, scale)
    for a in (0, t // 2, t - 4):
        one = slice(a, a + 4)
        xs, ts, cs, us = x[one].clone(), target[one].clone(), scale[one].clone(), up[one].clone()
        p = logprobs(s, xs, ts, cs)
        for n in ("logprobs", "entropy", "stats", "top_ids", "top_logprobs"):
            assert same_bits(getattr(p, n), getattr(o, n)[one])
        ls, st = distill(s, xs, few[one].clone(), values[one].clone(), cs)
        assert same_bits(ls, loss[one]) and same_bits(st, stats[one])
        assert same_bits(logprobs_bwd(s, xs, ts, p, us, us, cs), d1[one])
        assert same_bits(logprobs_bwd(s, xs, ts, p, us, None, cs), lone[one])
        assert same_bits(distill_bwd(s, xs, few[one].clone(), values[one].clone(), st, us, cs), d2[one])
    y = x.clone()
    assert same_bits(distill_bwd(s, y, few, values, stats, up, scale, out=y), d2)
    assert same_bits(logprobs_bwd(s, x, target, o, up, up, scale, out=x), d1)
