"""CPU pin of the oracle's cache at the top of bf16's range."""

import numpy as np
import pytest
import torch

from oracle import attention as ref

TOP = torch.finfo(torch.bfloat16).max


@pytest.mark.parametrize("most", [TOP, 3.3e38, 248 * 2.0 ** 120, 240 * 2.0 ** 120])
def test_finite_values_stay_bf16_numbers(most):
    """Blocks whose scale is 2^120: the type's own rounding, but never past 240 * 2^120."""
    most = float(torch.tensor(most).bfloat16())
    x = torch.cat([torch.linspace(-1, 1, 63), torch.tensor([1.0])]).double() * most
    x = x.float().bfloat16().double().reshape(64, 1, 1).numpy()
    got = ref.cached(x)
    s = 2.0 ** 120
    want = (torch.from_numpy(x / s).float().to(torch.float8_e4m3fn).double().clamp(-240, 240) * s).numpy()
    assert np.array_equal(got, want)
    assert np.array_equal(torch.from_numpy(got).bfloat16().double().numpy(), got) and np.isfinite(got).all()
    got = ref.cached(np.where(np.arange(64)[:, None, None] == 5, np.inf, x))
    assert np.isnan(got[5]).all() and np.array_equal(np.delete(got, 5, 0), np.delete(want, 5, 0))
