"""GPU tests of the norm's gradient at rows whose sum of squares passes fp32's range."""

import numpy as np
import pytest
import torch

import bitwise_invariant_gated_amd as gdn
from gpu_util import note
from stack_util import add_norm_bwd, dev, same_bits

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
def test_gradient_where_the_squares_pass_the_range(w, types):
    """r is 0 there, so dh is d_residual_out alone, and dw has nothing from such rows."""
    note(f"add_norm_bwd limits {w} {types}")
    h, wt, dy, d_res = inputs(w, types)
    s = gdn.NormShape(w, *types)
    sane = add_norm_bwd(s, h[GOOD].clone(), wt, dy[GOOD].clone(), d_res[GOOD].clone(), both=True)
    quiet, still = dy.clone(), h.clone()
    h[1, 3], h[3, w - 1], h[3, 0] = float("inf"), -float("inf"), float("inf")
    h[4], h[6, 5] = 3e38, -2e38
    bad = [i for i in range(8) if i not in GOOD]
    quiet[bad] = 0
    for d in (d_res, None):
        dx, dd, dw = add_norm_bwd(s, h, wt, dy, d, both=True)
        want = d_res[bad] if d is not None else torch.zeros_like(d_res[bad])
        assert torch.equal(dd[bad], want) and torch.equal(dx[bad], want.to(s.dtype))
        if d is not None:
            assert same_bits(dx[GOOD], sane[0]) and same_bits(dd[GOOD], sane[1])
        assert torch.equal(dw, add_norm_bwd(s, still, wt, quiet, d)[2])
    # a NaN is still one
    h[1, 3] = float("nan")
    dx, _, dw = add_norm_bwd(s, h, wt, dy, None)
    assert torch.isnan(dx[1]).all() and torch.isnan(dw).all() and torch.isfinite(dx[[0, 2, 3, 4]]).all()
