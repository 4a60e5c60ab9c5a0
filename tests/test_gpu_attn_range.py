"""GPU tests of the 8-bit cache at the top of bf16's range: what is finite stays
finite, and does not reach rows that do not see it."""

import numpy as np
import pytest
import torch

from gpu_util import note
from oracle import attention as ref

from attn_util import Layer, f64, random_seqs, same_bits

pytestmark = pytest.mark.gpu

TOP = torch.finfo(torch.bfloat16).max
CTX, NEW, AT = 30, 170, 70  # the call fills blocks 0, 1 and 2; the value's token is in block 1


@pytest.mark.parametrize("h,hk,d", [(7, 7, 64), (16, 4, 128), (8, 2, 256)])
@pytest.mark.parametrize("value", [TOP, -TOP, 248 * 2.0 ** 120, 240 * 2.0 ** 120, 224 * 2.0 ** 120])
def test_largest_values(h, hk, d, value):
    """One V of the largest magnitudes, at a key of score 0: rows before it have the
    bits that they have without it, in both prefill kernels, and decode agrees with them."""
    note(f"attn largest values h={h} hk={hk} d={d} value={value}")
    seqs = random_seqs(51, [CTX + NEW] * 8, h, hk, d)
    for _, k, v in seqs:
        k[AT] = 0
        v[AT] = 1.0
    clean = [tuple(x.clone() for x in s) for s in seqs]
    for _, _, v in seqs:
        v[AT, :, 3] = value
    got = []
    for most, which in ((0, seqs), (NEW, seqs), (0, clean)):
        L = Layer(h, hk, d, which)
        L.prefill([CTX] * 8)
        got.append((L.prefill([NEW] * 8, max_new=most), L))
    (a, La), (b, _), (c, _) = got
    D = Layer(h, hk, d, seqs)
    D.prefill([CTX + NEW - 80] * 8)
    dec = [D.decode() for _ in range(80)]
    kept, vals = La.read()
    for i, (q, k, v) in enumerate(seqs):
        assert same_bits(a[i], b[i]), i
        assert same_bits(a[i][:AT - CTX], c[i][:AT - CTX]), i
        assert same_bits(a[i][-80:], torch.cat([s[i] for s in dec])), i
        assert torch.isfinite(a[i].float()).all() and torch.isfinite(vals[i].float()).all()
        assert np.array_equal(f64(vals[i]), ref.cached(f64(v)))
        want = ref.attention(f64(q[CTX:]), f64(k), f64(v), d ** -0.5, CTX)
        # of the value's own dim: p and o are rounded to bf16, 2^-8 of them each, numerator and denominator
        assert np.abs(f64(a[i][:, :, 3]) - want[:, :, 3]).max() <= 1.05 * 2.0 ** -7 * abs(value)
