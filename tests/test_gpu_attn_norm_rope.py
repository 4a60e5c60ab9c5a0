"""GPU tests of the per-head norm with the rotation and its gradient against the fp64 oracle."""

import numpy as np
import pytest
import torch

import bitwise_invariant_gated_amd as gdn
from gpu_util import note
from oracle import attention as ref

from attn_util import f64

pytestmark = pytest.mark.gpu

DEV = "cuda"
EPS = 1e-5


def table(n, rd):
    ang = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, rd, 2) / rd)[None, :]
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


class Case:
    def __init__(self, t, h, hk, d, rd, inter, dtype, zero_centered=False, seed=0, n_pos=500):
        rng = np.random.default_rng(seed)
        self.t, self.h, self.hk, self.d, self.rd, self.inter = t, h, hk, d, rd, inter
        self.dtype, self.zc = dtype, zero_centered
        self.shape = gdn.AttnShape(h, hk, d, dtype)
        self.rope = gdn.AttnRope(rd, inter, EPS, zero_centered)
        dev = lambda a, dt=dtype: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DEV).to(dt)  # noqa: E731
        self.x = [dev(rng.standard_normal((t, n, d)) * 1.7) for n in (h, hk)]
        self.dy = [dev(rng.standard_normal((t, n, d))) for n in (h, hk)]
        self.w = [dev(1 + 0.3 * rng.standard_normal(d) - zero_centered, torch.float32) for _ in range(2)]
        self.cs = torch.from_numpy(table(n_pos, rd)).to(DEV) if rd else None
        self.pos = torch.from_numpy(rng.integers(0, n_pos, t).astype(np.int32)).to(DEV)
        cs = f64(self.cs)[f64(self.pos).astype(int)] if rd else np.zeros((t, 0))
        self.cos, self.sin = cs[:, : rd // 2], cs[:, rd // 2:]

    def ref_args(self, i):
        return f64(self.x[i]), f64(self.w[i]) + self.zc, self.cos, self.sin, EPS, self.inter

    def forward(self, x=None, out=None):
        x = x or self.x
        out = out or [torch.full_like(v, float("nan")).contiguous() for v in self.x]
        gdn.gdn_attn_qk_norm_rope(self.shape, self.rope, *x, *self.w, self.cs, self.pos, *out)
        return out

    def backward(self, dy=None, dx=None):
        dy = dy or self.dy
        dx = dx or [torch.full_like(v, float("nan")) for v in self.x]
        dw = [torch.full((self.d,), float("nan"), device=DEV) for _ in range(2)]
        ws = gdn.alloc_attn_workspace(self.shape, gdn.GDN_ATTN_OP_NORM_ROPE_BWD, self.t, device=DEV)
        gdn.gdn_attn_qk_norm_rope_bwd(self.shape, self.rope, *self.x, *self.w, self.cs, self.pos, *dy, *dx, *dw, ws)
        return dx, dw


CASES = [(1, 1, 1, 64, 64, False), (1, 16, 2, 256, 64, False), (7, 3, 1, 128, 128, False), (33, 5, 5, 64, 16, True),
         (130, 4, 2, 256, 256, True), (65, 12, 4, 128, 8, False), (40, 2, 1, 64, 24, False), (9, 4, 4, 128, 0, False),
         (2100, 6, 2, 64, 32, False), (700, 20, 4, 128, 128, False)]


def rounding(dtype):
    """The output's own rounding, of its magnitude: half a unit in the last of
    bf16's 8 bits, or of fp32's 24."""
    return torch.finfo(dtype).eps / 2


# fp32 steps before the output's rounding: mean of squares (about d / 16 + 5
# roundings, halved by the root), root, reciprocal, two products and the
# rotation, each at most 2^-24 of the pair's magnitude
SLACK = 2.0 ** -20


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("zc", [False, True])
def test_forward(case, dtype, zc):
    note(f"norm_rope {case} {dtype} zc={zc}")
    c = Case(*case, dtype, zero_centered=zc, seed=sum(case[:5]))
    for i, got in enumerate(c.forward()):
        want = ref.norm_rope(*c.ref_args(i))
        most = np.abs(want).max()
        assert np.abs(f64(got) - want).max() <= (rounding(dtype) + SLACK) * most


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_backward(case, dtype):
    note(f"norm_rope_bwd {case} {dtype}")
    c = Case(*case, dtype, seed=1 + sum(case[:5]))
    dx, dw = c.backward()
    for i in range(2):
        want, want_w, terms, size = ref.norm_rope_backward(*c.ref_args(i), f64(c.dy[i]))
        assert np.abs(f64(dx[i]) - want).max() <= rounding(dtype) * np.abs(want).max() + SLACK * 2 * size
        # the terms carry a few 2^-24 each and are added in fp32 along runs of at most some hundred
        assert (np.abs(f64(dw[i]) - want_w) <= 2.0 ** -17 * terms + 1e-30).all()


def test_backward_against_differences():
    """dx and dw against central differences of the oracle's forward in fp64."""
    note("norm_rope_bwd differences")
    c = Case(5, 2, 1, 64, 32, False, torch.float32, seed=3)
    dx, dw = c.backward()
    rng = np.random.default_rng(4)
    for i in range(2):
        x, w, *rest = c.ref_args(i)
        dy = f64(c.dy[i])
        loss = lambda x_, w_: float((ref.norm_rope(x_, w_, *rest) * dy).sum())  # noqa: E731
        for _ in range(40):
            at = tuple(int(rng.integers(0, n)) for n in x.shape)
            e = np.zeros_like(x)
            e[at] = 1e-5
            fd = (loss(x + e, w) - loss(x - e, w)) / 2e-5
            assert abs(float(dx[i][at]) - fd) <= 1e-5 * max(1.0, np.abs(f64(dx[i])).max())
        for j in range(0, 64, 7):
            e = np.zeros_like(w)
            e[j] = 1e-5
            fd = (loss(x, w + e) - loss(x, w - e)) / 2e-5
            assert abs(float(dw[i][j]) - fd) <= 1e-5 * max(1.0, np.abs(f64(dw[i])).max())


def test_in_place_and_views_give_the_same_bits():
    note("norm_rope in place and strided")
    c = Case(50, 4, 2, 128, 64, False, torch.bfloat16, seed=5)
    want = c.forward()
    rows = torch.cat([c.x[0].flatten(1), c.x[1].flatten(1), torch.zeros(50, 256, device=DEV, dtype=torch.bfloat16)], 1)
    q, k = rows[:, :512].view(50, 4, 128), rows[:, 512:768].view(50, 2, 128)
    got = c.forward(x=[q, k])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    c.forward(x=[q, k], out=[q, k])
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and not rows[:, 768:].any()
    dx, dw = c.backward()
    dy = [t.clone() for t in c.dy]
    dx2, dw2 = c.backward(dy=dy, dx=dy)
    assert all(torch.equal(a, b) for a, b in zip(dx + dw, dx2 + dw2))


def test_rows_alone_equal_rows_in_a_batch():
    """A token's row does not depend on the batch around it (the two launch shapes too)."""
    note("norm_rope alone")
    c = Case(9000, 16, 4, 128, 128, False, torch.bfloat16, seed=6)
    want = c.forward()
    for t in (0, 777, 8999):
        a = Case(1, 16, 4, 128, 128, False, torch.bfloat16)
        a.x, a.w, a.cs, a.pos = [x[t:t + 1] for x in c.x], c.w, c.cs, c.pos[t:t + 1].clone()
        for got, w in zip(a.forward(), want):
            assert torch.equal(got[0], w[t])


def test_gradient_is_the_same_every_time():
    note("norm_rope_bwd repeat")
    c = Case(3000, 8, 2, 64, 64, False, torch.bfloat16, seed=7)
    a = c.backward()
    for _ in range(3):
        b = c.backward()
        assert all(torch.equal(x, y) for x, y in zip(a[0] + a[1], b[0] + b[1]))


def test_no_tokens():
    note("norm_rope no tokens")
    c = Case(0, 4, 2, 64, 32, False, torch.bfloat16)
    c.forward()
    _, dw = c.backward()
    assert all(torch.count_nonzero(w) == 0 and not w.isnan().any() for w in dw)


def test_position_outside_the_table_gives_nan_in_the_rotated_dims():
    note("norm_rope position outside")
    c = Case(3, 2, 1, 64, 32, False, torch.float32, seed=8)
    want = c.forward()
    c.pos[1] = 500
    c.pos[2] = -1
    got = c.forward()
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1:, :, 32:], w[1:, :, 32:]) and g[1:, :, :32].isnan().all()


def test_rows_of_zeros_and_of_no_numbers():
    note("norm_rope zeros and nan")
    c = Case(4, 2, 2, 128, 128, False, torch.float32, seed=9)
    clean = c.forward()
    c.x[0][1] = 0
    c.x[0][2, 1, 7] = float("inf")
    got = c.forward()
    assert torch.equal(got[0][0], clean[0][0]) and torch.equal(got[1], clean[1]) and torch.equal(got[0][2, 0], clean[0][2, 0])
    assert torch.count_nonzero(got[0][1]) == 0
    assert got[0][2, 1].isnan().any()
