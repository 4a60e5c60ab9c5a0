"""GPU tests of the residual norm, its 8-bit output and its gradient against the fp64 oracle."""

import numpy as np
import pytest
import torch

import bitwise_invariant_gated_amd as gdn
from gpu_util import note
from oracle import stack as ref
from stack_util import DEV, F8, NORM, add_norm, add_norm_bwd, dev, f64, half, new, same_bits

pytestmark = pytest.mark.gpu

EPS = 1e-5
B, F = torch.bfloat16, torch.float32
TYPES = [(B, B), (B, F), (F, F)]
# every number of threads and vectors to a row, at, before and behind their borders
WIDTHS = [8, 104, 128, 136, 512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 16384]


class Case:
    def __init__(self, t, w, types, zc=False, seed=0, wide=False):
        rng = np.random.default_rng(seed + t + w)
        self.t, self.width, (self.dt, self.rdt), self.zc = t, w, types, zc
        self.x = dev(rng.standard_normal((t, w)), self.dt)
        self.res = dev(rng.standard_normal((t, w)) * 3, self.rdt)
        self.dy = dev(rng.standard_normal((t, w)), self.dt)
        self.d_res = dev(rng.standard_normal((t, w)), self.rdt)
        self.w = dev(1 + 0.3 * rng.standard_normal(w) - zc)

    def shape(self, group=-1):
        return gdn.NormShape(self.width, self.dt, self.rdt, group, EPS, self.zc)

    def weights(self):
        return f64(self.w) + self.zc


@pytest.mark.parametrize("w", WIDTHS)
@pytest.mark.parametrize("types", TYPES)
def test_forward(w, types):
    for t in (1, 7, 33):
        note(f"add_norm {t} x {w} {types}")
        c = Case(t, w, types, zc=w % 16 == 8)
        h, y, _, _ = add_norm(c.shape(), c.x, c.res, c.w)
        assert same_bits(h, (c.x.float() + c.res.float()).to(c.rdt))
        want = ref.add_norm(f64(h), c.weights(), EPS)
        assert (np.abs(f64(y) - want) <= (half(c.dt) + NORM) * np.abs(want) + 1e-30).all()
        # without the residual, and without its output
        h, y, _, _ = add_norm(c.shape(), c.x, None, c.w)
        assert same_bits(h, c.x.to(c.rdt))
        want = ref.add_norm(f64(h), c.weights(), EPS)
        assert (np.abs(f64(y) - want) <= (half(c.dt) + NORM) * np.abs(want) + 1e-30).all()
        assert same_bits(add_norm(c.shape(), c.x, None, c.w, h=False)[1], y)


@pytest.mark.parametrize("w", [8, 128, 512, 1000, 1024, 2048, 4096, 5000, 16384])
@pytest.mark.parametrize("types", TYPES)
def test_eight_bits(w, types):
    for group in (0, 128) if w % 128 == 0 else (0,):
        note(f"add_norm 8 bits {w} {types} group {group}")
        c = Case(19, w, types, seed=5)
        c.res[3] *= 1e-30  # values far apart
        c.x[3] *= 1e-30
        c.x[4], c.res[4] = 0, 0
        h, y, y8, sc = add_norm(c.shape(group), c.x, c.res, c.w)
        assert same_bits(y, add_norm(c.shape(), c.x, c.res, c.w)[1])
        alone = add_norm(c.shape(group), c.x, c.res, c.w, y=False, h=False)
        assert same_bits(alone[2], y8) and same_bits(alone[3], sc)
        n = group or w
        want = ref.add_norm(f64(h), c.weights(), EPS).reshape(19, -1, n)
        scale = np.maximum(np.abs(want).max(-1), 2.0 ** -100) / 448
        assert (np.abs(f64(sc) - scale) <= 2 * NORM * scale).all()
        got = f64(y8.view(F8)).reshape(want.shape) * f64(sc)[..., None]
        # half a step of e4m3: 2^-4 of the value, or of its least steps of 2^-9 scales
        bound = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * scale[..., None])
        assert (np.abs(got - want) <= bound * (1 + 4 * NORM) + 4 * NORM * np.abs(want)).all()
        assert (np.abs(f64(y8.view(F8))).reshape(want.shape).max(-1)[[0, 5]] == 448).all()
        assert (y8[4] & 127 == 0).all() and torch.allclose(sc[4], torch.tensor(2.0 ** -100 / 448, device=DEV))


@pytest.mark.parametrize("w", WIDTHS)
@pytest.mark.parametrize("types", TYPES)
def test_backward(w, types):
    for t, res in ((1, True), (6, False), (40, True)):
        note(f"add_norm_bwd {t} x {w} {types} res={res}")
        c = Case(t, w, types, zc=w % 16 == 0, seed=3)
        h = (c.x.float() + c.res.float()).to(c.rdt)
        dx, dd, dw = add_norm_bwd(c.shape(), h, c.w, c.dy, c.d_res if res else None, both=res)
        hf, dy, wt = f64(h), f64(c.dy), c.weights()
        dr = f64(c.d_res) if res else np.zeros_like(hf)
        dh, want_w = ref.add_norm_backward(hf, wt, EPS, dy, dr)
        r = 1 / np.sqrt(np.mean(hf * hf, -1, keepdims=True) + EPS)
        dn = dy * wt
        size = np.abs(dr) + r * np.abs(dn) + r ** 3 * np.abs(hf) * np.mean(np.abs(dn * hf), -1, keepdims=True)
        assert (np.abs(f64(dx) - dh) <= half(c.dt) * np.abs(dh) + 2 * NORM * size).all()
        if dd is not None:
            assert (np.abs(f64(dd) - dh) <= half(c.rdt) * np.abs(dh) + 2 * NORM * size).all()
        assert (np.abs(f64(dw) - want_w) <= 4 * NORM * np.sum(np.abs(dy * hf * r), 0) + 1e-30).all()


@pytest.mark.parametrize("t,w,types", [(5000, 64, (B, B)), (2500, 2048, (B, F)), (1100, 4104, (F, F)), (700, 8192, (B, B))])
def test_many_rows(t, w, types):
    """More rows than the gradient has work-groups for; dw over all of them."""
    note(f"add_norm many {t} x {w} {types}")
    c = Case(t, w, types, seed=9)
    h, y, _, _ = add_norm(c.shape(), c.x, c.res, c.w)
    want = ref.add_norm(f64(h), c.weights(), EPS)
    assert (np.abs(f64(y) - want) <= (half(c.dt) + NORM) * np.abs(want) + 1e-30).all()
    dx, _, dw = add_norm_bwd(c.shape(), h, c.w, c.dy, None)
    hf, dy = f64(h), f64(c.dy)
    r = 1 / np.sqrt(np.mean(hf * hf, -1, keepdims=True) + EPS)
    dh, want_w = ref.add_norm_backward(hf, c.weights(), EPS, dy, np.zeros_like(hf))
    size = r * np.abs(dy * c.weights()) + r ** 3 * np.abs(hf) * np.mean(np.abs(dy * c.weights() * hf), -1, keepdims=True)
    assert (np.abs(f64(dx) - dh) <= half(c.dt) * np.abs(dh) + 2 * NORM * size).all()
    assert (np.abs(f64(dw) - want_w) <= 4 * NORM * np.sum(np.abs(dy * hf * r), 0)).all()
    assert all(same_bits(a, b) for a, b in zip(add_norm_bwd(c.shape(), h, c.w, c.dy, None), (dx, None, dw)))


@pytest.mark.parametrize("w", [64, 512, 2048, 4096])
def test_gradient_is_the_differences(w):
    """d sum(y dy + h dr) / dx by central differences of the fp32 kernel itself, along random directions."""
    note(f"add_norm differences {w}")
    rng = np.random.default_rng(w)
    c = Case(3, w, (F, F), seed=11)
    h, _, _, _ = add_norm(c.shape(), c.x, c.res, c.w)
    dx, _, dw = add_norm_bwd(c.shape(), h, c.w, c.dy, c.d_res)
    for _ in range(3):
        v, u = rng.standard_normal((3, w)), rng.standard_normal(w)
        got = []
        for e in (2.0 ** -7, -2.0 ** -7):
            hh, y, _, _ = add_norm(c.shape(), c.x + e * dev(v), c.res, c.w + e * dev(u))
            got.append((f64(y) * f64(c.dy)).sum() + (f64(hh) * f64(c.d_res)).sum())
        slope = (got[0] - got[1]) * 2.0 ** 6
        want = (f64(dx) * v).sum() + (f64(dw) * u).sum()
        # values of about 1 in 3 w places, each to 2^-22, over a step of 2^-6, and the third derivative's 2^-14
        size = np.sqrt((f64(c.dy) ** 2).sum() + (f64(c.d_res) ** 2).sum())
        assert abs(slope - want) <= size * (2.0 ** -22 * 2 ** 6 * 8 + 2.0 ** -14 * 8)


def test_strides_and_in_place():
    note("add_norm strides")
    for types in TYPES:
        c = Case(21, 520, types, seed=2)
        s = c.shape(0)
        h, y, y8, sc = add_norm(s, c.x, c.res, c.w)
        dx, dd, dw = add_norm_bwd(s, h, c.w, c.dy, c.d_res, both=True)

        def inside(t, pad=24):
            wide = torch.full((21, 520 + pad), 7.0, dtype=t.dtype, device=DEV)
            wide[:, 8:528] = t
            return wide, wide[:, 8:528]

        (_, x2), (_, r2), (hw, h2), (yw, y2) = inside(c.x), inside(c.res, 40), inside(h * 0), inside(y * 0, 32)
        gdn.gdn_stack_add_norm(s, x2, r2, c.w, h2, y2, y8.fill_(1), sc)
        assert same_bits(h2, h) and same_bits(y2, y)
        for wide in (hw, yw):
            assert (wide[:, :8] == 7).all() and (wide[:, 528:] == 7).all()
        # the residual stream updated in place, y over x
        x3, r3 = c.x.clone(), c.res.clone()
        gdn.gdn_stack_add_norm(s, x3, r3, c.w, r3, x3)
        assert same_bits(r3, h) and same_bits(x3, y)
        # gradients over what they come from
        g, d = c.dy.clone(), c.d_res.clone()
        ws = gdn.alloc_norm_workspace(s, 21, DEV)
        gdn.gdn_stack_add_norm_bwd(s, h, c.w, g, d, g, d, dw.fill_(0), ws)
        assert same_bits(g, dx) and same_bits(d, dd)
        _, h4 = inside(h)
        gw, g4 = inside(c.dy, 48)
        gdn.gdn_stack_add_norm_bwd(s, h4, c.w, g4, inside(c.d_res)[1], g4, h4, dw, ws)
        assert same_bits(g4, dx) and same_bits(h4, dd) and (gw[:, 528:] == 7).all()


def test_a_row_does_not_depend_on_the_others():
    note("add_norm rows alone")
    for w in (64, 136, 1000, 2048, 4096, 6000):
        c = Case(300, w, (B, B), seed=1)
        h, y, y8, sc = add_norm(c.shape(0), c.x, c.res, c.w)
        dx, _, _ = add_norm_bwd(c.shape(), h, c.w, c.dy, c.d_res)
        for i in (0, 5, 299):
            one = slice(i, i + 1)
            got = add_norm(c.shape(0), c.x[one].clone(), c.res[one].clone(), c.w)
            assert all(same_bits(a, b[one]) for a, b in zip(got, (h, y, y8, sc)))
            assert same_bits(add_norm_bwd(c.shape(), h[one].clone(), c.w, c.dy[one].clone(), c.d_res[one].clone())[0], dx[one])
        # the norm of the stored stream has the same bits
        assert same_bits(add_norm(c.shape(), h, None, c.w)[1], y)


def test_no_rows_and_special_values():
    note("add_norm no rows")
    c = Case(4, 256, (B, B))
    s = c.shape(128)
    e = torch.empty(0, 256, dtype=B, device=DEV)
    gdn.gdn_stack_add_norm(s, e, e, c.w, e, e)
    dw = new(256)
    gdn.gdn_stack_add_norm_bwd(s, e, c.w, e, None, e, None, dw, gdn.alloc_norm_workspace(s, 0, DEV))
    assert (dw == 0).all()
    note("add_norm special values")
    c.x[0, 5], c.x[1, 7], c.x[2] = float("nan"), float("inf"), 0
    c.res[2] = 0
    h, y, y8, sc = add_norm(s, c.x, c.res, c.w)
    assert torch.isnan(y[0]).all() and (y8[0] & 127 == 127).all()
    assert torch.isnan(y[1, 7]) and (y[1, :7] == 0).all() and (y[1, 8:] == 0).all()
    assert (y[2] == 0).all() and (y8[2] & 127 == 0).all() and torch.isfinite(sc).all()
    good = Case(4, 256, (B, B))
    assert same_bits(y[3], add_norm(s, good.x, good.res, good.w)[1][3])
