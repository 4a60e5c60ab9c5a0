"""GPU tests of the entropy's gradient at masked columns where d_entropy, the scale or their product is large
(a loss's scale, a temperature near 0): the probability is 0, and so is the gradient."""

import numpy as np
import pytest
import torch

import bitwise_invariant_gated_amd as gdn
from gpu_util import note
from stack_util import dev, logprobs, logprobs_bwd
from test_gpu_stack_logits import check_backward, make

pytestmark = pytest.mark.gpu

B, F = torch.bfloat16, torch.float32


@pytest.mark.parametrize("v", [50, 2048, 5000])
@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("up", [2.0 ** 27, 2.0 ** 31, 2.0 ** 60])
def test_large_gradients_at_masked_columns(v, dtype, up):
    note(f"logprobs_bwd masked {v} {dtype} d_entropy {up}")
    x, target, _ = make(6, v, dtype, seed=3, masked=True)
    x[1, v // 2:] = torch.finfo(dtype).min
    target = torch.where(dev(np.arange(6)) == 1, 0, target).to(torch.int32)
    scale = dev(np.array([1.0, 2, 0.5, 2, 1, 1.5]))  # no probability below fp32's normal range but those of 0
    g, f = dev(np.linspace(-1, 1, 6)), dev(np.array([1, -1, 1, -1, 0.5, -0.5]) * up)
    s = gdn.LogitsShape(v, dtype)
    o = logprobs(s, x, target, scale)
    for gg in (g, None):
        d = logprobs_bwd(s, x, target, o, gg, f, scale)
        assert torch.isfinite(d).all()
        check_backward(s, x, target if gg is not None else None, scale, gg, f, d)


@pytest.mark.parametrize("v", [50, 5000])
@pytest.mark.parametrize("dtype", [B, F])
def test_large_scales_at_masked_columns(v, dtype):
    """One token left of two that are far apart, at temperatures down to 1e-30."""
    note(f"logprobs_bwd masked {v} {dtype} large scales")
    x = torch.full((4, v), -float("inf"), dtype=dtype, device="cuda")
    x[:, 3], x[:, v - 1] = 1, 3
    target = dev(np.full(4, v - 1), torch.int32)
    scale, one = dev(np.array([1e3, 1e9, 1e20, 1e30])), dev(np.ones(4))
    s = gdn.LogitsShape(v, dtype)
    o = logprobs(s, x, target, scale)
    assert (o.logprobs == 0).all() and (o.entropy == 0).all()
    assert (logprobs_bwd(s, x, target, o, one, one, scale) == 0).all()
