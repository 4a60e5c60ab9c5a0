"""GPU tests of the norm with the rotation and its gradient on outputs of 64 MB and more,
which are stored past the caches."""

import numpy as np
import pytest
import torch

from gpu_util import note
from oracle import attention as ref

from attn_util import f64
from test_gpu_attn_norm_rope import EPS, SLACK, Case, rounding

pytestmark = pytest.mark.gpu

# tokens, heads, key heads, dim, rotated dims, adjacent pairs, type
CASES = [(12001, 16, 16, 128, 128, False, torch.bfloat16), (5003, 24, 8, 128, 64, True, torch.float32),
         (20011, 24, 8, 64, 32, False, torch.bfloat16), (9007, 15, 15, 64, 64, True, torch.float32),
         (8009, 14, 7, 256, 64, False, torch.bfloat16), (4001, 16, 2, 256, 256, False, torch.float32)]


def sample(t):
    return sorted({0, 1, t // 3, t // 2, t - 2, t - 1, *range(7, t, t // 40)})


def at(case, tokens):
    """The case's oracle arguments for some tokens only."""
    def args(i):
        return (f64(case.x[i][tokens]), f64(case.w[i]) + case.zc, case.cos[tokens], case.sin[tokens], EPS, case.inter)
    return args


def make(case):
    c = Case(*case, seed=sum(case[:5]))
    assert sum(x.numel() * x.element_size() for x in c.x) >= 64 << 20
    return c


@pytest.mark.parametrize("case", CASES)
def test_forward(case):
    note(f"norm_rope large {case}")
    c = make(case)
    got, rows = c.forward(), sample(case[0])
    for i in range(2):
        want = ref.norm_rope(*at(c, rows)(i))
        assert np.abs(f64(got[i][rows]) - want).max() <= (rounding(c.dtype) + SLACK) * np.abs(want).max()
        assert not got[i].isnan().any()
    # the other kernel variants give every row the same bits
    for lo, hi in ((0, 1), (17, 300), (c.t - 2000, c.t)):
        a = Case(1, *case[1:], zero_centered=c.zc)
        a.t, a.x, a.w, a.pos = hi - lo, [x[lo:hi].clone() for x in c.x], c.w, c.pos[lo:hi].clone()
        a.cs = c.cs
        assert all(torch.equal(x, y[lo:hi]) for x, y in zip(a.forward(), got))


@pytest.mark.parametrize("case", CASES)
def test_backward(case):
    note(f"norm_rope_bwd large {case}")
    c = make(case)
    dx, dw = c.backward()
    rows = sample(case[0])
    cos, sin = (torch.from_numpy(x).cuda()[:, None, :] for x in (c.cos, c.sin))
    for i in range(2):
        want, _, _, size = ref.norm_rope_backward(*at(c, rows)(i), f64(c.dy[i][rows]))
        assert np.abs(f64(dx[i][rows]) - want).max() <= rounding(c.dtype) * np.abs(want).max() + SLACK * 2 * size
        assert not dx[i].isnan().any()
        # dw over all tokens, in 64 bits
        x, dy = c.x[i].double(), c.dy[i].double()
        a, b = (dy[..., :c.rd:2], dy[..., 1:c.rd:2]) if c.inter else dy[..., :c.rd].chunk(2, -1)
        a, b = a * cos + b * sin, b * cos - a * sin
        turned = torch.stack([a, b], -1).flatten(-2) if c.inter else torch.cat([a, b], -1)
        terms = torch.cat([turned, dy[..., c.rd:]], -1) * x * (x.pow(2).mean(-1, keepdim=True) + EPS).rsqrt()
        # a few 2^-24 of every term, added in fp32 along runs of at most some hundred
        assert ((dw[i].double() - terms.sum((0, 1))).abs() <= 2.0 ** -17 * terms.abs().sum((0, 1))).all()
    again = c.backward()
    assert all(torch.equal(p, q) for p, q in zip(dx + dw, again[0] + again[1]))
