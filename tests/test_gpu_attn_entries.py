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


def window(t, pad=128, fill=float("nan")):
    """A copy of t inside a larger array whose rows before and behind it hold `fill`: (view, whole)."""
    whole = torch.full((t.shape[0] + 2 * pad, *t.shape[1:]), fill, dtype=t.dtype, device=DEV)
    whole[pad:-pad] = t
    return whole[pad:-pad], whole


def around(whole, pad=128):
    return torch.cat([whole[:pad], whole[-pad:]])


# how the batch's first and last limits are wrong: before the tokens, and past them
@pytest.mark.parametrize("first,past", [(-5, 36), (-100, 100), (0, 1), (-1, 0)])
@pytest.mark.parametrize("how", [50, 0])
@pytest.mark.parametrize("h,hk,d", [(7, 7, 64), (16, 4, 128), (8, 2, 256)])
def test_limits_outside_the_tokens(h, hk, d, how, first, past):
    """cu_seqlens that begins before token 0 and ends behind token T: the call does what it
    does for limits held to 0 and T, and touches nothing around its arrays."""
    note(f"attn limits h={h} hk={hk} d={d} how={how} {first} {past}")
    lens = [40, 50, 13, 24] * 4
    n = len(lens)
    seqs = random_seqs(62, [70 + n for n in lens], h, hk, d)

    def step(wrong):
        L = Layer(h, hk, d, seqs)
        L.prefill([70] * n)
        (q, k, v), cu = L.pack(lens)
        plan = L.plan(lens, cu)
        if wrong:
            cu = cu.clone()
            cu[0] += first
            cu[-1] += past
        (q, qw), (k, kw), (v, vw) = window(q), window(k), window(v)
        o, ow = window(torch.full_like(q, float("nan")))
        ws = gdn.alloc_attn_workspace(L.shape, gdn.GDN_ATTN_OP_PREFILL, sum(lens), n, L.cache.k8.shape[0], DEV)
        gdn.gdn_attn_prefill(L.shape, q, k, v, cu, plan, L.cache, o, ws, max_new=how)
        assert around(ow).isnan().all()
        return o, contents(L), L, cu

    want, full, _, _ = step(False)
    got, after, L, cu = step(True)
    assert same_bits(got, want) and all(torch.equal(a, b) for a, b in zip(after, full))
    # the read-out of the new tokens' number of tokens, by the same wrong limits
    out = [window(torch.full((sum(lens), hk, d), float("nan"), dtype=torch.bfloat16, device=DEV)) for _ in range(4)]
    plan = gdn.alloc_attn_plan(L.pool, n, 0, L.slot_index)
    right = cu.clone()
    right[0], right[-1] = 0, sum(lens)
    for limits, (k, v) in ((cu, out[:2]), (right, out[2:])):
        gdn.gdn_attn_cache_read(L.shape, limits, sum(lens), plan, L.cache, k[0], v[0])
    for a, b in zip(out[:2], out[2:]):
        assert around(a[1]).isnan().all() and torch.equal(a[0].view(torch.int16), b[0].view(torch.int16))


def test_limits_that_leave_tokens_out():
    """Tokens before the first limit and behind the last belong to nobody: nothing of theirs is written."""
    h, hk, d, lens = 8, 2, 128, [40, 50, 70] * 4
    note("attn limits inside")
    seqs = random_seqs(63, lens, h, hk, d)
    for how in (70, 0):
        L = Layer(h, hk, d, seqs)
        want = torch.cat(L.prefill(lens))
        L = Layer(h, hk, d, seqs)
        (q, k, v), cu = L.pack(lens)
        (_, q), (_, k), (_, v) = window(q), window(k), window(v)
        cu += 128
        plan = gdn.alloc_attn_plan(L.pool, len(lens), q.shape[0], L.slot_index)
        plan.positions.fill_(-7)
        plan.slot_map.fill_(-7)
        gdn.gdn_attn_plan(L.pool, cu, plan)
        assert (around(plan.positions) == -7).all() and (around(plan.slot_map) == -7).all()
        assert plan.positions[128:-128].tolist() == [p for n in lens for p in range(n)]
        o = torch.full_like(q, float("nan"))
        ws = gdn.alloc_attn_workspace(L.shape, gdn.GDN_ATTN_OP_PREFILL, q.shape[0], len(lens), L.cache.k8.shape[0], DEV)
        gdn.gdn_attn_prefill(L.shape, q, k, v, cu, plan, L.cache, o, ws, max_new=how)
        assert same_bits(o[128:-128], want) and around(o).isnan().all()


@pytest.mark.parametrize("lens", [[40, 50, 13, 24], [1500, 2, 3000, 700]])  # tokens in the plan's launch, or in a second
@pytest.mark.parametrize("first,past", [(-5, 36), (-100, 100), (3, -4)])
def test_plan_with_limits_outside_the_tokens(lens, first, past):
    note(f"plan limits {lens} {first} {past}")
    pool = gdn.alloc_attn_pool(4, 60, 200, DEV)
    t = sum(lens)
    pos, pos_all = window(torch.full((t,), -7, **I32), fill=-7)
    place, place_all = window(torch.full((t,), -7, dtype=torch.int64, device=DEV), fill=-7)
    plan = gdn.AttnPlan(torch.empty(4, **I32), pos, place, torch.empty(1, **I32), pool.block_table)
    cu = torch.tensor([sum(lens[:i]) for i in range(5)], **I32)
    cu[0] += first
    cu[-1] += past
    gdn.gdn_attn_plan(pool, cu, plan)
    assert int(plan.status) == 0 and plan.ctx_len.tolist() == [0] * 4
    assert (around(pos_all) == -7).all() and (around(place_all) == -7).all()
    lo, hi = max(first, 0), t + min(past, 0)
    seq = torch.bucketize(torch.arange(lo, hi), torch.tensor(cu.tolist()[1:]), right=True)
    want = torch.arange(lo, hi) - cu.cpu()[seq]
    assert pos[lo:hi].tolist() == want.tolist()
    assert (pos[:lo] == -7).all() and (pos[hi:] == -7).all() and (place[:lo] == -7).all() and (place[hi:] == -7).all()
    assert place[lo:hi].tolist() == (pool.block_table.cpu()[seq, want // 64].long() * 64 + want % 64).tolist()


@pytest.mark.parametrize("how,new", [("decode", 1), (2, 2), (0, 70)])
@pytest.mark.parametrize("entry", [-1, 1 << 20])
@pytest.mark.parametrize("h,hk,d", [(7, 7, 64), (16, 4, 128), (8, 2, 256)])
def test_missing_block_is_not_written(h, hk, d, entry, how, new):
    """The table has no block of the pool where a row's block fills: nobody's block is written for it."""
    note(f"attn missing block h={h} hk={hk} d={d} entry={entry} how={how}")
    n, ctx, row = 8, 127, 3
    seqs = random_seqs(64, [ctx + new] * n, h, hk, d)

    def step(missing):
        L = Layer(h, hk, d, seqs)
        L.prefill([ctx] * n)
        (q, k, v), cu = L.pack([new] * n)
        plan = L.plan([new] * n, cu)
        gone = int(L.pool.block_table[row, 1])
        if missing:
            L.pool.block_table[row, 1] = entry
        before = contents(L)
        return call(L, q, k, v, cu, plan, how).view(n, new, h, d), before, contents(L), gone

    want, _, full, _ = step(False)
    got, before, after, gone = step(True)
    assert all(same_bits(got[i], want[i]) for i in range(n) if i != row)
    assert same_bits(got[row, 0], want[row, 0])  # its own block comes from the tail
    for x in range(4):
        assert torch.equal(after[x][gone], before[x][gone])
        rest = torch.arange(len(after[x]), device=DEV) != gone
        assert torch.equal(after[x][rest], full[x][rest])
    for x in (4, 5):
        assert torch.equal(after[x], full[x])


@pytest.mark.parametrize("how,new", [("decode", 1), (2, 2), (0, 70)])
@pytest.mark.parametrize("h,hk,d", [(7, 7, 64), (16, 4, 128), (8, 2, 256)])
def test_contexts_that_the_table_cannot_hold(h, hk, d, how, new):
    """ctx_len up to the end of 32 bits, in some entries: zeros, nothing of theirs written, the others as
    without them."""
    note(f"attn contexts past the table h={h} hk={hk} d={d} how={how}")
    n, ctx = 8, 127
    seqs = random_seqs(65, [ctx + new] * n, h, hk, d)

    def step(wrong):
        L = Layer(h, hk, d, seqs)
        L.prefill([ctx] * n)
        (q, k, v), cu = L.pack([new] * n)
        plan = L.plan([new] * n, cu)
        for i, x in wrong.items():
            plan.ctx_len[i] = x
        before = contents(L)
        return call(L, q, k, v, cu, plan, how).view(n, new, h, d), before, contents(L), L.pool.block_table

    want, _, full, table = step({})
    width = table.shape[1]
    wrong = {0: 2 ** 31 - 1, 3: 2 ** 31 - 100, 4: 1 << 30, 7: 64 * (width + 1) - new}
    got, before, after, _ = step(wrong)
    mine = torch.cat([table[i][table[i] >= 0] for i in wrong]).long()
    for i in range(n):
        if i in wrong:
            assert torch.count_nonzero(got[i]) == 0 and not got[i].isnan().any()
        else:
            assert same_bits(got[i], want[i])
    for x in range(4):
        assert torch.equal(after[x][mine], before[x][mine])
        rest = torch.ones(len(after[x]), dtype=torch.bool, device=DEV)
        rest[mine] = False
        assert torch.equal(after[x][rest], full[x][rest])
    for x in (4, 5):
        for i in range(n):
            assert torch.equal(after[x][i], (before if i in wrong else full)[x][i])


@pytest.mark.parametrize("how,new", [("decode", 1), (2, 2), (0, 30)])
def test_open_block_past_a_full_table(how, new):
    """Every full block is in the table and the open one has no entry yet: the answer is that of a wider table."""
    h, hk, d, n, ctx = 8, 8, 64, 8, 130
    note(f"attn open block past the table how={how}")
    seqs = random_seqs(66, [ctx + new] * n, h, hk, d)
    got = []
    for width in (None, 2):
        L = Layer(h, hk, d, seqs)
        L.prefill([ctx] * n)
        (q, k, v), cu = L.pack([new] * n)
        plan = L.plan([new] * n, cu)
        table = plan.block_table if width is None else plan.block_table[:, :width].contiguous()
        hand = gdn.AttnPlan(plan.ctx_len, plan.positions, plan.slot_map, plan.status, table, plan.slot_index)
        got.append((call(L, q, k, v, cu, hand, how), contents(L)))
    assert same_bits(got[0][0], got[1][0])
    assert all(torch.equal(a, b) for a, b in zip(got[0][1], got[1][1]))
