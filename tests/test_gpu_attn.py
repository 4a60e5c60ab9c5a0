"""GPU tests of attention over the 8-bit cache against the fp64 oracle, and of
the bits: prefill == continuation == decode, alone == packed."""

import numpy as np
import pytest
import torch

import bitwise_invariant_gated_amd as gdn
from gpu_util import note
from oracle import attention as ref

from attn_util import DEV, Layer, bf16, f64, random_seqs, same_bits, tolerance

pytestmark = pytest.mark.gpu

SHAPES = [(4, 2, 64), (3, 1, 128), (2, 2, 256), (8, 1, 256), (5, 1, 64), (16, 1, 128), (20, 1, 64)]


def expect(seq, first, scale):
    q, k, v = (f64(x) for x in seq)
    return ref.attention(q[first:], k, v, scale, first), tolerance(v)


@pytest.mark.parametrize("h,hk,d", SHAPES)
def test_prefill_matches_oracle(h, hk, d):
    lens = [1, 64, 65, 200, 0, 63]
    note(f"attn prefill h={h} hk={hk} d={d} lens={lens}")
    seqs = random_seqs(1, lens, h, hk, d)
    L = Layer(h, hk, d, seqs)
    for seq, o in zip(seqs, L.prefill(lens)):
        if len(o):
            want, tol = expect(seq, 0, d ** -0.5)
            assert np.abs(f64(o) - want).max() <= tol
    k, v = L.read()
    for i, (_, sk, sv) in enumerate(seqs):
        assert np.array_equal(f64(k[i]), ref.cached(f64(sk)))
        assert np.array_equal(f64(v[i]), ref.cached(f64(sv)))


@pytest.mark.parametrize("h,hk,d", SHAPES)
@pytest.mark.parametrize("start", [0, 62, 63, 511, 575])
def test_decode_matches_oracle_and_prefill(h, hk, d, start):
    note(f"attn decode h={h} hk={hk} d={d} start={start}")
    steps = 4
    seqs = random_seqs(2, [start + steps, start + 40 + steps], h, hk, d)
    lens = [s[0].shape[0] for s in seqs]
    whole = Layer(h, hk, d, seqs)
    full = whole.prefill(lens)
    L = Layer(h, hk, d, seqs, slots=[3, 1])
    if start:
        L.prefill([start, start + 40])
    else:
        L.prefill([0, 40])
    outs = [L.decode() for _ in range(steps)]
    for i, seq in enumerate(seqs):
        first = lens[i] - steps
        got = torch.cat([o[i] for o in outs])
        want, tol = expect(seq, first, d ** -0.5)
        assert np.abs(f64(got) - want).max() <= tol
        assert same_bits(got, full[i][first:])
    for a, b in zip(L.read(), whole.read()):
        assert all(same_bits(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("h,hk,d", [(4, 2, 64), (8, 1, 128), (2, 1, 256)])
def test_segments_give_the_bits_of_one_prompt(h, hk, d):
    lens = [700, 1100, 130]
    note(f"attn segments h={h} hk={hk} d={d}")
    seqs = random_seqs(3, lens, h, hk, d)
    whole = Layer(h, hk, d, seqs)
    full = whole.prefill(lens)
    L = Layer(h, hk, d, seqs)
    parts = [L.prefill(t, max_new=max(t)) for t in ([100, 3, 1], [1, 0, 64], [470, 600, 2], [129, 497, 63])]
    for i in range(3):
        assert same_bits(torch.cat([p[i] for p in parts]), full[i])
    for a, b in zip(L.read(), whole.read()):
        assert all(same_bits(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("h,hk,d", [(4, 4, 128), (6, 2, 64)])
def test_alone_equals_packed(h, hk, d):
    lens = [300, 1, 777, 64, 1030]
    note(f"attn alone h={h} hk={hk} d={d}")
    seqs = random_seqs(4, lens, h, hk, d)
    pre = [max(0, n - 3) for n in lens]
    L = Layer(h, hk, d, [s for s, n in zip(seqs, lens) if n > 3])
    first = L.prefill([n for n in pre if n])
    steps = [L.decode() for _ in range(3)]
    at = 0
    for seq, n in zip(seqs, lens):
        if n <= 3:
            continue
        A = Layer(h, hk, d, [seq])
        assert same_bits(A.prefill([n - 3])[0], first[at])
        for s in steps:
            assert same_bits(A.decode()[0], s[at])
        at += 1


def test_long_context_split_over_work_groups():
    """A few sequences whose partitions go to different work-groups, beside one of a single token."""
    h, hk, d = 8, 2, 128
    lens = [9000, 2, 5200]
    note("attn long split")
    seqs = random_seqs(5, lens, h, hk, d)
    L = Layer(h, hk, d, seqs)
    L.prefill([n - 1 for n in lens])
    got = L.decode()
    for i, seq in enumerate(seqs):
        want, tol = expect(seq, lens[i] - 1, d ** -0.5)
        assert np.abs(f64(got[i]) - want).max() <= tol
    whole = Layer(h, hk, d, seqs)
    full = whole.prefill(lens)
    assert all(same_bits(g, f[-1:]) for g, f in zip(got, full))


def test_more_partitions_than_records():
    """Sequences that share blocks: the batch has more partitions than the pool's
    size suggests, and sequences are dealt out whole; the bits stay."""
    h, hk, d, n, ctx = 2, 1, 64, 40, 1300
    note("attn shared blocks")
    base = random_seqs(6, [ctx + 1], h, hk, d)[0]
    one = Layer(h, hk, d, [base])
    one.prefill([ctx])
    # n rows over the same full blocks, each with its own copy of the tail
    rows = n
    table = one.pool.block_table[:1].repeat(rows, 1).contiguous()
    cache = gdn.AttnCache(one.cache.k8, one.cache.v8, one.cache.k_scale, one.cache.v_scale,
                          one.cache.tail_k[:1].repeat(rows, 1, 1, 1).contiguous(),
                          one.cache.tail_v[:1].repeat(rows, 1, 1, 1).contiguous())
    rng = np.random.default_rng(7)
    q = bf16(rng, n, h, d).to(DEV)
    k, v = (base[j][ctx:].repeat(n, 1, 1).to(DEV).contiguous() for j in (1, 2))
    i32 = dict(dtype=torch.int32, device=DEV)
    plan = gdn.AttnPlan(torch.full((n,), ctx, **i32), torch.full((n,), ctx, **i32),
                        torch.zeros(n, dtype=torch.int64, device=DEV), torch.zeros(1, **i32), table)
    ws = gdn.alloc_attn_workspace(one.shape, gdn.GDN_ATTN_OP_DECODE, n, n, cache.k8.shape[0], DEV)
    o = torch.empty_like(q)
    gdn.gdn_attn_decode_step(one.shape, q, k, v, plan, cache, o, ws)
    kc, vc = f64(base[1]), f64(base[2])
    for i in range(n):
        want = ref.attention(f64(q[i:i + 1]), kc, vc, d ** -0.5, ctx)
        assert np.abs(f64(o[i:i + 1]) - want).max() <= tolerance(vc)


def test_entries_without_a_request_give_zeros_and_touch_nothing():
    h, hk, d = 4, 2, 128
    note("attn inactive entries")
    seqs = random_seqs(8, [70, 70, 70], h, hk, d)
    L = Layer(h, hk, d, seqs)
    L.prefill([69, 69, 69])
    (q, k, v), cu = L.pack([1, 1, 1])
    before = [t.clone() for t in (L.cache.tail_k, L.cache.tail_v)]
    L.slot_index[1] = -1
    plan = gdn.alloc_attn_plan(L.pool, 3, 3, L.slot_index)
    gdn.gdn_attn_plan(L.pool, cu, plan)
    assert plan.ctx_len.tolist() == [69, -1, 69] and plan.slot_map.tolist()[1] == -1
    for op in (gdn.GDN_ATTN_OP_DECODE, gdn.GDN_ATTN_OP_PREFILL):
        ws = gdn.alloc_attn_workspace(L.shape, op, 3, 3, L.cache.k8.shape[0], DEV)
        o = torch.full_like(q, float("nan"))
        if op == gdn.GDN_ATTN_OP_DECODE:
            gdn.gdn_attn_decode_step(L.shape, q, k, v, plan, L.cache, o, ws)
        else:
            gdn.gdn_attn_prefill(L.shape, q, k, v, cu, plan, L.cache, o, ws)
        assert torch.count_nonzero(o[1]) == 0 and not o[1].isnan().any()
        for i in (0, 2):
            want, tol = expect(seqs[i], 69, d ** -0.5)
            assert np.abs(f64(o[i:i + 1]) - want).max() <= tol
        for now, was in zip((L.cache.tail_k, L.cache.tail_v), before):
            assert torch.equal(now[1].view(torch.int16), was[1].view(torch.int16))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_one_sequence_with_no_numbers_does_not_reach_others(d):
    """NaN and infinities in one sequence's k and v: its own rows after them show
    it, rows before them and other sequences do not, in prefill as in decode."""
    h, hk, n, bad = 2, 1, 150, 100
    note(f"attn non-finite d={d}")
    seqs = random_seqs(9, [n, n], h, hk, d)
    clean = [tuple(x.clone() for x in s) for s in seqs]
    seqs[0][1][bad, 0, 3] = float("nan")
    seqs[0][2][bad, 0, 5] = float("inf")
    L = Layer(h, hk, d, seqs)
    got = L.prefill([n, n])
    C = Layer(h, hk, d, clean)
    want = C.prefill([n, n])
    assert same_bits(got[1], want[1])
    assert same_bits(got[0][:bad], want[0][:bad])
    assert got[0][bad:].isnan().all()
    D = Layer(h, hk, d, seqs)
    D.prefill([n - 60, n - 60])
    steps = [D.decode() for _ in range(60)]
    for i in range(2):
        dec = torch.cat([s[i] for s in steps])
        assert torch.equal(dec.isnan(), got[i][n - 60:].isnan())
        ok = ~dec.isnan()
        assert torch.equal(dec[ok].view(torch.int16), got[i][n - 60:][ok].view(torch.int16))


def test_values_with_infinities_show_only_in_their_dims():
    """An infinite v in one dim: that dim is infinite (own block) or NaN (8 bits
    hold no infinity), every other dim is as without it."""
    h, hk, d, n, bad = 2, 1, 128, 140, 70
    note("attn infinite v")
    seqs = random_seqs(10, [n], h, hk, d)
    clean = [tuple(x.clone() for x in s) for s in seqs]
    seqs[0][2][bad, 0, 5] = float("inf")
    clean[0][2][bad, 0, 5] = 0.0
    a, b = Layer(h, hk, d, seqs).prefill([n])[0], Layer(h, hk, d, clean).prefill([n])[0]
    other = [x for x in range(d) if x != 5]
    assert same_bits(a[..., other], b[..., other])
    assert same_bits(a[:bad], b[:bad])
    assert torch.isinf(a[bad:128, :, 5]).all() and (a[bad:128, :, 5] > 0).all()
    assert a[128:, :, 5].isnan().all()


@pytest.mark.parametrize("amp", [2.0 ** -126, 1e-30, 1e30])
def test_scales_at_the_ends_of_the_range(amp):
    h, hk, d, n = 2, 1, 64, 130
    note(f"attn amplitude {amp}")
    rng = np.random.default_rng(11)
    q, k, v = bf16(rng, n, h, d), bf16(rng, n, hk, d), (bf16(rng, n, hk, d).float() * amp).bfloat16()
    v[:64] = 0  # and a block of zeros
    L = Layer(h, hk, d, [(q, k, v)])
    o = L.prefill([n])[0]
    want = ref.attention(f64(q), f64(k), f64(v), d ** -0.5)
    # bf16 keeps 8 bits down to 2^-126; below, values are multiples of 2^-133
    assert np.abs(f64(o) - want).max() <= tolerance(f64(v)) + 2.0 ** -133
    _, vc = L.read()
    assert np.array_equal(f64(vc[0]), ref.cached(f64(v)))


def test_large_scores_and_small_scale():
    h, hk, d, n = 2, 2, 128, 600
    note("attn peaked scores")
    seqs = random_seqs(12, [n], h, hk, d, q_std=40.0)
    for scale in (d ** -0.5, 1e-4):
        o = Layer(h, hk, d, seqs, scale=scale).prefill([n])[0]
        want, tol = expect(seqs[0], 0, scale)
        # scores of up to some hundreds carry 2^-24 of their size, times d / 8 rounded adds
        assert np.abs(f64(o) - want).max() <= 1.3 * tol


def test_views_of_a_projection():
    """q, k, v read in place out of rows that hold all three."""
    h, hk, d, n = 4, 2, 128, 100
    note("attn strided")
    rng = np.random.default_rng(13)
    rows = bf16(rng, n, (h + 2 * hk) * d)
    q, k, v = (x.reshape(n, -1, d) for x in rows.split([h * d, hk * d, hk * d], 1))
    L = Layer(h, hk, d, [(q, k, v)])
    want = L.prefill([n])[0]
    S = Layer(h, hk, d, [(q, k, v)])
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    plan = S.plan([n], cu)
    dev = rows.to(DEV)
    qd, kd, vd = (dev[:, a:b].view(n, -1, d) for a, b in ((0, h * d), (h * d, (h + hk) * d), ((h + hk) * d, (h + 2 * hk) * d)))
    o = torch.empty((n, h, d), dtype=torch.bfloat16, device=DEV)
    ws = gdn.alloc_attn_workspace(S.shape, gdn.GDN_ATTN_OP_PREFILL, n, 1, S.cache.k8.shape[0], DEV)
    gdn.gdn_attn_prefill(S.shape, qd, kd, vd, cu, plan, S.cache, o, ws)
    assert same_bits(o, want)


def test_pool_beyond_32_bit_offsets():
    """Block ids whose bytes lie past 2^32."""
    h, hk, d, n = 2, 1, 256, 200
    note("attn large pool")
    seqs = random_seqs(14, [n], h, hk, d)
    small = Layer(h, hk, d, seqs)
    want = small.prefill([n - 1])[0]
    step = small.decode()[0]
    blocks = (1 << 32) // (64 * d) + 40
    L = Layer(h, hk, d, seqs, extra_blocks=blocks, garbage=False)
    L.pool.free_blocks.copy_(torch.arange(L.pool.free_blocks.numel(), dtype=torch.int32, device=DEV))
    assert same_bits(L.prefill([n - 1])[0], want)
    assert int(L.pool.block_table[0, 0]) * 64 * d > 1 << 32
    assert same_bits(L.decode()[0], step)


def test_another_stream_and_graph_replay():
    """A decode step captured once and replayed gives each replay's eager result."""
    h, hk, d, n = 4, 2, 128, 3
    note("attn graph")
    lens = [200, 63, 600]
    seqs = random_seqs(15, [x + 5 for x in lens], h, hk, d)
    E = Layer(h, hk, d, seqs)
    E.prefill(lens)
    eager = [E.decode() for _ in range(5)]
    L = Layer(h, hk, d, seqs)
    L.prefill(lens)
    (q, k, v), cu = L.pack([1] * n)
    plan = gdn.alloc_attn_plan(L.pool, n, n, L.slot_index)
    ws = gdn.alloc_attn_workspace(L.shape, gdn.GDN_ATTN_OP_DECODE, n, n, L.cache.k8.shape[0], DEV)
    o = torch.empty_like(q)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        gdn.gdn_attn_plan(L.pool, cu, plan)
        gdn.gdn_attn_decode_step(L.shape, q, k, v, plan, L.cache, o, ws)
    for step in range(5):
        (a, b, c), _ = L.pack([1] * n)
        q.copy_(a), k.copy_(b), v.copy_(c)
        graph.replay()
        torch.cuda.synchronize()
        L.done = [x + 1 for x in L.done]
        for got, want in zip(torch.split(o, 1), eager[step]):
            assert same_bits(got, want), step
