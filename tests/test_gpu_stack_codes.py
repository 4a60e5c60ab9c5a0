"""GPU tests of the norm's 8-bit codes: each is the quotient n / s, formed in fp32, to the nearest code."""

import numpy as np
import pytest
import torch

import bitwise_invariant_gated_amd as gdn
from gpu_util import note
from stack_util import F8, add_norm, dev, same_bits

pytestmark = pytest.mark.gpu

F = torch.float32


def codes(y, scale):
    """From the fp32 norm and its scales as stored; numpy's quotient is rounded once."""
    y, scale = y.cpu().numpy(), scale.cpu().numpy()
    q = y.reshape(*scale.shape, -1) / scale[..., None]
    return torch.from_numpy(q.reshape(y.shape)).to(F8).view(torch.uint8)


def borders(w, rng):
    """Weights in units of their largest / 448 that lie on the borders between two codes, or up to two
    steps of fp32 beside them."""
    step = 2.0 ** rng.integers(-9, 6, w)
    at = np.where(step == 2.0 ** -9, rng.integers(0, 8, w), rng.integers(8, 15, w))
    x = (np.minimum((at + 0.5) * step, 432) * rng.choice([-1, 1], w)).astype(np.float32)
    return (x.view(np.int32) + rng.integers(-2, 3, w, dtype=np.int32)).view(np.float32)


@pytest.mark.parametrize("w,group", [(128, 128), (1000, 0), (2048, 128), (4096, 0), (8192, 128), (16384, 0)])
def test_codes_beside_the_borders(w, group):
    note(f"codes {w} group {group}")
    rng = np.random.default_rng(w)
    weights = borders(w, rng).astype(np.float64)
    weights[::group or w] = 448
    s = gdn.NormShape(w, F, F, group, 1e-6)
    # rows of one magnitude: n is the weights but for a rounding, so the scale is that of their largest
    x = dev(np.exp(rng.standard_normal((3, 1))) * np.ones((3, w)))
    for unit in np.exp(rng.standard_normal(40)):
        _, y, y8, scale = add_norm(s, x, None, dev(weights * unit))
        assert same_bits(y8.cpu(), codes(y, scale))


@pytest.mark.parametrize("group", [0, 128])
def test_codes_of_many_values(group):
    note(f"codes 4,000 x 1,024 group {group}")
    rng = np.random.default_rng(7)
    x, res = dev(rng.standard_normal((4000, 1024))), dev(4 * rng.standard_normal((4000, 1024)))
    _, y, y8, scale = add_norm(gdn.NormShape(1024, F, F, group), x, res, dev(1 + 0.2 * rng.standard_normal(1024)))
    assert same_bits(y8.cpu(), codes(y, scale))


@pytest.mark.parametrize("w,group", [(512, 128), (1000, 0), (4096, 0)])
def test_codes_at_the_ends_of_the_range(w, group):
    """Values up to fp32's largest and past it (the scale is infinite then, and finite values give 0),
    down to those that the least scale leaves nothing of."""
    note(f"codes ends {w} group {group}")
    rng = np.random.default_rng(w)
    for top in (3e38, 1e39, 1e-25, 2.0 ** -100, 1e-33, 1e-38):
        weights = np.clip(rng.standard_normal(w) * top, -3.4e38, 3.4e38)
        x = dev(rng.choice([-1, 1], (5, w)) * np.exp(0.1 * rng.standard_normal((5, w))))
        _, y, y8, scale = add_norm(gdn.NormShape(w, F, F, group, 0.0), x, None, dev(weights))
        with np.errstate(all="ignore"):
            want = codes(y, scale)
        got = y8.cpu()
        nan = want & 127 == 127
        assert torch.equal(got & 127 == 127, nan) and torch.equal(got[~nan], want[~nan])
        assert top < 1e38 or bool(nan.any()) or torch.isfinite(y).all()
