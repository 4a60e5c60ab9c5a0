"""GPU tests of the norm at rows whose sum of squares is 0 while eps is too, and of its gradient there."""

import numpy as np
import pytest
import torch

import bitwise_invariant_gated_amd as gdn
from gpu_util import note
from oracle import stack as ref
from stack_util import NORM, add_norm, add_norm_bwd, dev, f64, half

pytestmark = pytest.mark.gpu

B, F = torch.bfloat16, torch.float32
TYPES = [(B, B), (B, F), (F, F)]
# every number of threads to a row
WIDTHS = [104, 512, 1024, 2048, 4096, 8192, 16384]
GOOD = [0, 2, 5, 7]


def inputs(w, types, seed=0):
    rng = np.random.default_rng(seed + w)
    dt, rdt = types
    return (dev(rng.standard_normal((8, w)), rdt), dev(1 + 0.3 * rng.standard_normal(w)), dev(rng.standard_normal((8, w)), dt),
            dev(rng.standard_normal((8, w)), rdt))


@pytest.mark.parametrize("w", WIDTHS)
@pytest.mark.parametrize("types", TYPES)
def test_rows_of_zeros_without_eps(w, types):
    """0 / 0 counts as 0: such rows give zeros, and their gradient is d_residual_out."""
    note(f"add_norm zeros {w} {types}")
    h, wt, dy, d_res = inputs(w, types, seed=1)
    group = 128 if w % 128 == 0 else 0
    s = gdn.NormShape(w, *types, group, 0.0)
    bad = [1, 3, 4, 6]
    h[bad] = 0
    h[4, ::2] = -0.0
    _, y, y8, scale = add_norm(s, h.to(s.dtype), None, wt)
    stream = h.to(s.dtype).to(s.residual_dtype)
    assert (y[bad] == 0).all() and (y8[bad] & 127 == 0).all() and torch.isfinite(scale).all()
    want = ref.add_norm(f64(stream)[GOOD], f64(wt), 0.0)
    assert (np.abs(f64(y)[GOOD] - want) <= (half(s.dtype) + NORM) * np.abs(want) + 1e-30).all()
    dx, dd, dw = add_norm_bwd(s, h, wt, dy, d_res, both=True)
    assert torch.equal(dd[bad], d_res[bad]) and torch.equal(dx[bad], d_res[bad].to(s.dtype))
    hf, g = f64(h)[GOOD], f64(dy)[GOOD]
    dh, want_w = ref.add_norm_backward(hf, f64(wt), 0.0, g, f64(d_res)[GOOD])
    r = 1 / np.sqrt(np.mean(hf * hf, -1, keepdims=True))
    dn = g * f64(wt)
    size = np.abs(f64(d_res)[GOOD]) + r * np.abs(dn) + r ** 3 * np.abs(hf) * np.mean(np.abs(dn * hf), -1, keepdims=True)
    assert (np.abs(f64(dd)[GOOD] - dh) <= half(s.residual_dtype) * np.abs(dh) + 2 * NORM * size).all()
    assert (np.abs(f64(dw) - want_w) <= 4 * NORM * np.sum(np.abs(g * hf * r), 0) + 1e-30).all()
