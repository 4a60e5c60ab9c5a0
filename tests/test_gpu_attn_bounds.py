"""GPU tests of long contexts in which every block shows (marked_seqs), against the fp64
oracle element by element, within a bound that no lost, repeated or wrongly scaled block
keeps (test_attn_bounds.py)."""

import numpy as np
import pytest
import torch

import bitwise_invariant_gated_amd as gdn
from gpu_util import note

from attn_util import DEV, LONG, SHARED, Layer, bf16, expect_within, f64, marked_seqs, random_seqs, same_bits

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device=DEV)


def within(got, q, k, v, scale, first=0):
    want, room = expect_within(q, k, v, scale, first)
    return (np.abs(f64(got) - want) <= room).all()


@pytest.mark.parametrize("h,hk,d,lens", LONG)
def test_decode_after_long_contexts(h, hk, d, lens):
    """Partitions of one row on many work-groups (up to 137 of them, so the join goes on past 64 records)."""
    note(f"attn long decode h={h} hk={hk} d={d} {lens}")
    seqs = marked_seqs(71, lens, h, hk, d)
    L = Layer(h, hk, d, seqs)
    L.prefill([n - 1 for n in lens])
    got = L.decode()
    full = Layer(h, hk, d, seqs).prefill(lens)
    for i, seq in enumerate(seqs):
        assert same_bits(got[i], full[i][-1:]), i
        assert within(got[i], *seq, d ** -0.5, lens[i] - 1), i


@pytest.mark.parametrize("h,hk,d", [(4, 2, 128), (4, 1, 64), (4, 2, 256)])
@pytest.mark.parametrize("how", [70, 0])
def test_new_tokens_after_long_contexts(h, hk, d, how):
    """Turns of 70 and 7 tokens, six of each, by either prefill kernel: all rows have the same
    bits in both, the last of each sequence is near the oracle."""
    lens, new = [9000, 5200] * 6, [70, 7] * 6
    note(f"attn long turns h={h} hk={hk} d={d} max_new={how}")
    seqs = marked_seqs(72, lens, h, hk, d)
    out = []
    for most in (how, 70 - how):
        L = Layer(h, hk, d, seqs)
        L.prefill([n - m for n, m in zip(lens, new)])
        out.append(L.prefill(new, max_new=most))
    for i, seq in enumerate(seqs):
        assert same_bits(out[0][i], out[1][i]), i
        if i < 2:
            assert within(out[0][i][-1:], *seq, d ** -0.5, lens[i] - 1), i


@pytest.mark.parametrize("how,new", [("decode", 1), (40, 40)])
def test_rows_over_shared_blocks(how, new):
    """64 rows over the same blocks have more units than there is room for records: whole
    chunks go to work-groups, and every row is near the oracle."""
    h, hk, d, n = SHARED
    rows, ctx = 64, n - new
    note(f"attn shared blocks, marked, {how}")
    base = marked_seqs(71, [n], h, hk, d)[0]
    one = Layer(h, hk, d, [base], extra_blocks=rows)
    one.prefill([ctx])
    table = one.pool.block_table[:1].repeat(rows, 1).contiguous()
    table[:, ctx // 64] = one.pool.free_blocks[:rows]  # the block that the call fills is every row's own
    tails = [t[:1].repeat(rows, 1, 1, 1).contiguous() for t in (one.cache.tail_k, one.cache.tail_v)]
    cache = gdn.AttnCache(one.cache.k8, one.cache.v8, one.cache.k_scale, one.cache.v_scale, *tails)
    rng = np.random.default_rng(73)
    q = bf16(rng, rows, new, h, d, std=0.5)
    k, v = (x[ctx:].repeat(rows, 1, 1).to(DEV).contiguous() for x in base[1:])
    plan = gdn.AttnPlan(torch.full((rows,), ctx, **I32), torch.zeros(rows * new, **I32),
                        torch.zeros(rows * new, dtype=torch.int64, device=DEV), torch.zeros(1, **I32), table)
    qd = q.view(rows * new, h, d).to(DEV)
    o = torch.full_like(qd, float("nan"))
    op = gdn.GDN_ATTN_OP_DECODE if how == "decode" else gdn.GDN_ATTN_OP_PREFILL
    ws = gdn.alloc_attn_workspace(one.shape, op, rows * new, rows, cache.k8.shape[0], DEV)
    if how == "decode":
        gdn.gdn_attn_decode_step(one.shape, qd, k, v, plan, cache, o, ws)
    else:
        gdn.gdn_attn_prefill(one.shape, qd, k, v, torch.arange(0, rows * new + 1, new, **I32), plan, cache, o, ws, max_new=new)
    o = o.view(rows, new, h, d)
    for i in (0, 1, 31, 62, 63):
        whole = torch.cat([base[0][:ctx], q[i]])
        assert within(o[i][-1:], whole, *base[1:], d ** -0.5, n - 1), i


@pytest.mark.parametrize("h,hk,d", [(20, 1, 128), (24, 1, 256), (34, 2, 128), (40, 1, 64)])
def test_more_than_sixteen_query_heads_to_a_key_head(h, hk, d):
    """A decode step in several chunks per key/value head, one of them short."""
    lens = [1300, 700, 65, 2]
    note(f"attn wide groups h={h} hk={hk} d={d}")
    seqs = marked_seqs(74, lens, h, hk, d)
    L = Layer(h, hk, d, seqs)
    L.prefill([n - 1 for n in lens])
    got = L.decode()
    full = Layer(h, hk, d, seqs).prefill(lens)
    for i, seq in enumerate(seqs):
        assert same_bits(got[i], full[i][-1:]), i
        assert within(got[i], *seq, d ** -0.5, lens[i] - 1), i


@pytest.mark.parametrize("h,hk,d", [(4, 2, 64), (3, 1, 128), (2, 2, 256)])
def test_random_values_within_the_bound(h, hk, d):
    """Signed random values: the bound per element, of every row of prompts that end beside blocks."""
    lens = [1, 64, 65, 200, 63, 640]
    note(f"attn bound h={h} hk={hk} d={d}")
    seqs = random_seqs(75, lens, h, hk, d)
    for seq, o in zip(seqs, Layer(h, hk, d, seqs).prefill(lens)):
        assert within(o, *seq, d ** -0.5)
