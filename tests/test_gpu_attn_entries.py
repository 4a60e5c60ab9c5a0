"""GPU tests of batch entries that no request stands behind, in steps that a caller
fills by hand: they give zeros and leave the caches of the others alone."""

import pytest
import torch

import bitwise_invariant_gated_amd as gdn
from gpu_util import note

from attn_util import DEV, Layer, random_seqs, same_bits

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device=DEV)


def contents(L):
    """Every byte of a layer's cache."""
    c = L.cache
    return [t.clone().view(torch.uint8) for t in (c.k8, c.v8, c.k_scale, c.v_scale, c.tail_k, c.tail_v)]


def call(L, q, k, v, cu, plan, how):
    """One step by the decode call, or by either kernel of the prefill."""
    o = torch.full((q.shape[0], L.shape.num_heads, L.shape.head_dim), float("nan"), dtype=q.dtype, device=DEV)
    n = plan.ctx_len.numel()
    op = gdn.GDN_ATTN_OP_DECODE if how == "decode" else gdn.GDN_ATTN_OP_PREFILL
    ws = gdn.alloc_attn_workspace(L.shape, op, q.shape[0], n, L.cache.k8.shape[0], DEV)
    if how == "decode":
        gdn.gdn_attn_decode_step(L.shape, q, k, v, plan, L.cache, o, ws)
    else:
        gdn.gdn_attn_prefill(L.shape, q, k, v, cu, plan, L.cache, o, ws, max_new=how)
    return o


# decode; prefill with few rows a sequence; prefill that counts with all tokens in one sequence
@pytest.mark.parametrize("how,new", [("decode", 1), (2, 2), (0, 70)])
@pytest.mark.parametrize("row", [-1, 99])
@pytest.mark.parametrize("h,hk,d", [(7, 7, 64), (16, 4, 128), (8, 2, 256)])
def test_no_cache_row_beside_a_context(h, hk, d, row, how, new):
    """slot_index names no row, ctx_len says 127 tokens (the block fills): zeros, row 0 untouched."""
    note(f"attn no row h={h} hk={hk} d={d} row={row} how={how}")
    n, ctx = 8, 127
    seqs = random_seqs(61, [ctx + new] * n, h, hk, d)

    def step(rows):
        L = Layer(h, hk, d, seqs)
        L.prefill([ctx] * n)
        (q, k, v), cu = L.pack([new] * n)
        plan = L.plan([new] * n, cu)
        hand = gdn.AttnPlan(plan.ctx_len, plan.positions, plan.slot_map, plan.status, plan.block_table,
                            torch.tensor(rows, **I32))
        before = contents(L)
        return call(L, q, k, v, cu, hand, how).view(n, new, h, d), before, contents(L), L

    want, _, full, _ = step(list(range(n)))
    got, before, after, L = step([row] + list(range(1, n)))
    assert torch.count_nonzero(got[0]) == 0 and not got[0].isnan().any()
    assert all(same_bits(got[i], want[i]) for i in range(1, n))
    mine = L.pool.block_table[0, :4].long()  # row 0's blocks
    mine = mine[mine >= 0]
    for x in range(4):
        assert torch.equal(after[x][mine], before[x][mine])
        rest = torch.ones(len(after[x]), dtype=torch.bool, device=DEV)
        rest[mine] = False
        assert torch.equal(after[x][rest], full[x][rest])
    for x in (4, 5):
        assert torch.equal(after[x][0], before[x][0]) and torch.equal(after[x][1:], full[x][1:])
