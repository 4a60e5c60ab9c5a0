"""CPU check of the long-context tests' own power: with their inputs and their bound, a
block or a partition that is left out, taken twice or scaled wrongly is seen."""

import numpy as np
import pytest

from oracle import attention as ref

from attn_util import error_bound, f64, marked_seqs
from attn_util import LONG, SHARED


def shares(q, k, v, scale):
    """Per head: numerators [blocks, d] and denominators [blocks] of the last position."""
    kc, vc = ref.cached(k), ref.cached(v)
    n, hk, d = k.shape
    lo = (n - 1) // 64 * 64
    kc[lo:], vc[lo:] = k[lo:], v[lo:]  # its own block, in the input type
    grp, out = q.shape[1] // hk, []
    edges = np.arange(0, n, 64)
    for h in range(q.shape[1]):
        s = kc[:, h // grp] @ q[-1, h] * scale
        w = np.exp(s - s.max())
        out.append((np.add.reduceat(w[:, None] * vc[:, h // grp], edges, 0), np.add.reduceat(w, edges)))
    return out


@pytest.mark.parametrize("h,hk,d,n", [(h, hk, d, n) for h, hk, d, lens in LONG for n in lens if n > 1000] + [SHARED])
def test_a_wrong_block_or_partition_is_seen(h, hk, d, n):
    q, k, v = (f64(x) for x in marked_seqs(71, [n], h, hk, d)[0])
    heads = shares(q, k, v, d ** -0.5)
    blocks = -(-n // 64)
    o = [num.sum(0) / den.sum() for num, den in heads]
    want = ref.attention(q[-1:], k, v, d ** -0.5, n - 1)
    assert np.abs(np.stack(o) - want[0]).max() < 1e-9
    for first, last in [(b, b + 1) for b in range(blocks)] + [(b, min(b + 8, blocks)) for b in range(0, blocks, 8)]:
        part = [(num[first:last].sum(0), den[first:last].sum()) for num, den in heads]
        for what, dn, dd in (("left out", -1, -1), ("twice", 1, 1), ("V twice as large", 1, 0), ("V half", -0.5, 0)):
            seen = 0.0
            for (num, den), (pn, pd), right in zip(heads, part, o):
                wrong = (num.sum(0) + dn * pn) / (den.sum() + dd * pd)
                # a result within the bound of the wrong value, and within that of the right one?
                room = error_bound(right, right) + error_bound(wrong, wrong)
                seen = max(seen, (np.abs(wrong - right) / np.maximum(room, 1e-300)).max())
            assert seen > 1, (what, first, last, seen)
