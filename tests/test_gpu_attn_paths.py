"""GPU tests of the two kernels behind gdn_attn_prefill: which one runs is a matter
of sizes and of max_new, and no bit of a result may depend on it."""

import numpy as np
import pytest
import torch

import bitwise_invariant_gated_amd as gdn
from gpu_util import note
from oracle import attention as ref

from attn_util import DEV, Layer, bf16, f64, random_seqs, same_bits, tolerance

pytestmark = pytest.mark.gpu

# Without max_new a sequence may hold all tokens: 8 sequences of these heads are
# then too many chunks for the kernel that splits the keys; with max_new they are few.
SHAPES = [(7, 7, 64), (12, 4, 64), (6, 6, 128), (16, 4, 128), (4, 4, 256), (8, 2, 256)]
CTX = [0, 1, 63, 64, 449, 511, 512, 1100]
NEW = [70, 129, 2, 64, 130, 1, 65, 0]


def both(h, hk, d, seqs, ctx, new, scale=None):
    """Outputs and layers of `new` tokens after `ctx`, by either kernel."""
    out = []
    for most in (0, max(new)):
        L = Layer(h, hk, d, seqs, scale=scale)
        if any(ctx):
            L.prefill(ctx)
        out.append((L.prefill(new, max_new=most), L))
    return out


@pytest.mark.parametrize("h,hk,d", SHAPES)
def test_both_kernels_give_the_same_bits(h, hk, d):
    note(f"attn both kernels h={h} hk={hk} d={d}")
    seqs = random_seqs(31, [c + n for c, n in zip(CTX, NEW)], h, hk, d)
    (a, La), (b, Lb) = both(h, hk, d, seqs, CTX, NEW)
    for i, seq in enumerate(seqs):
        assert same_bits(a[i], b[i]), i
        if NEW[i]:
            q, k, v = (f64(x) for x in seq)
            want = ref.attention(q[CTX[i]:], k, v, d ** -0.5, CTX[i])
            assert np.abs(f64(a[i]) - want).max() <= tolerance(v), i
    for x, y in zip(La.read(), Lb.read()):
        assert all(same_bits(p, q) for p, q in zip(x, y))


@pytest.mark.parametrize("h,hk,d", [(7, 7, 64), (16, 4, 128), (8, 2, 256)])
def test_keys_and_values_that_are_not_numbers(h, hk, d):
    """In blocks that are 8 bits for some new rows and not there for others, in the
    block before them, and in the open one: rows that do not see them are as without
    them, rows that do show them, by either kernel."""
    note(f"attn non-finite both kernels h={h} hk={hk} d={d}")
    seqs = random_seqs(32, [c + n for c, n in zip(CTX, NEW)], h, hk, d)
    clean = [tuple(x.clone() for x in s) for s in seqs]
    at = {1: (100, "v"), 0: (40, "k"), 3: (127, "v"), 4: (449 + 70, "v"), 6: (512 + 10, "v"), 7: (1090, "v")}
    for i, (p, what) in at.items():
        for head in range(0, hk, 2):  # the others stay as they are
            if what == "v":
                seqs[i][2][p, head, 3] = float("nan")
                seqs[i][2][max(p - 7, 0), head, d - 1] = float("inf")
            else:
                seqs[i][1][p, head, 0] = float("nan")
    (a, _), (b, _) = both(h, hk, d, seqs, CTX, NEW)
    (c, _), _ = both(h, hk, d, clean, CTX, NEW)
    G = h // hk
    for i in range(len(seqs)):
        assert torch.equal(a[i].isnan(), b[i].isnan()), i
        ok = ~a[i].isnan()
        assert torch.equal(a[i][ok].view(torch.int16), b[i][ok].view(torch.int16)), i
        first = at[i][0] - 7 - CTX[i] if i in at and at[i][1] == "v" else at[i][0] - CTX[i] if i in at else NEW[i]
        first = min(max(first, 0), NEW[i])
        assert same_bits(a[i][:first], c[i][:first]), i  # rows before
        for head in range(1, hk, 2):  # heads beside
            assert same_bits(a[i][:, head * G:(head + 1) * G], c[i][:, head * G:(head + 1) * G]), i
        if i in at and at[i][1] == "v":  # only the dims that hold them
            assert same_bits(a[i][..., 4:d - 1], c[i][..., 4:d - 1]), i
            seen = a[i][max(at[i][0] - CTX[i], 0):, 0, 3]
            assert seen.isnan().all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("step", [0.02, 0.2, -0.2])
def test_scores_that_rise_or_fall_along_the_keys(d, step):
    """`step` a key, natural units: 1.8 or 18 in powers of two a block, so the
    reference of the exponents stays for some blocks or moves in each."""
    h, hk = 2, 1
    note(f"attn rising scores d={d} step={step}")
    seqs = random_seqs(33, [c + n for c, n in zip(CTX, NEW)], h, hk, d)
    for q, k, _ in seqs:
        q.mul_(0.25)
        q[..., 0] = 1.0
        k[..., 0] = (torch.arange(k.shape[0]) * step)[:, None].bfloat16()
    L = Layer(h, hk, d, seqs, scale=1.0)
    first = L.prefill([c + n - (c + n) // 2 for c, n in zip(CTX, NEW)])
    rest = L.prefill([(c + n) // 2 for c, n in zip(CTX, NEW)], max_new=max((c + n) // 2 for c, n in zip(CTX, NEW)))
    for i, seq in enumerate(seqs):
        got = torch.cat([first[i], rest[i]])
        q, k, v = (f64(x) for x in seq)
        want = ref.attention(q, k, v, 1.0)
        assert np.abs(f64(got) - want).max() <= tolerance(v), i


def test_more_units_than_records_among_new_tokens():
    """64 sequences over the same 312 blocks: chunks are dealt out whole, and every
    sequence has the bits that it has alone."""
    h, hk, d, n, ctx, new = 1, 1, 64, 64, 20010, 40
    note("attn shared blocks, new tokens")
    base = random_seqs(34, [ctx], h, hk, d)[0]
    one = Layer(h, hk, d, [base], extra_blocks=n)
    one.prefill([ctx])
    table = one.pool.block_table[:1].repeat(n, 1).contiguous()
    # the block that the call fills is every row's own
    table[:, ctx // 64] = one.pool.free_blocks[:n]
    tails = [t[:1].repeat(n, 1, 1, 1).contiguous() for t in (one.cache.tail_k, one.cache.tail_v)]
    cache = gdn.AttnCache(one.cache.k8, one.cache.v8, one.cache.k_scale, one.cache.v_scale,
                          *(t.clone() for t in tails))
    rng = np.random.default_rng(35)
    q, k, v = (bf16(rng, n * new, x, d).to(DEV) for x in (h, hk, hk))
    i32 = dict(dtype=torch.int32, device=DEV)

    def run(rows):
        m = len(rows)
        cache.tail_k.copy_(tails[0])
        cache.tail_v.copy_(tails[1])
        pick = torch.cat([torch.arange(i * new, (i + 1) * new) for i in rows]).to(DEV)
        plan = gdn.AttnPlan(torch.full((m,), ctx, **i32), torch.zeros(m * new, **i32),
                            torch.zeros(m * new, dtype=torch.int64, device=DEV), torch.zeros(1, **i32), table,
                            torch.tensor(rows, **i32))
        ws = gdn.alloc_attn_workspace(one.shape, gdn.GDN_ATTN_OP_PREFILL, m * new, m, cache.k8.shape[0], DEV)
        qq = q[pick].contiguous()
        o = torch.full_like(qq, float("nan"))
        gdn.gdn_attn_prefill(one.shape, qq, k[pick].contiguous(), v[pick].contiguous(),
                             torch.arange(0, m * new + 1, new, **i32), plan, cache, o, ws, max_new=new)
        return o.view(m, new, h, d)

    all_ = run(list(range(n)))
    for i in (0, 1, 31, 63):
        assert same_bits(run([i])[0], all_[i]), i
    kc, vc = (np.concatenate([f64(b), f64(x[63 * new:])]) for b, x in ((base[1], k), (base[2], v)))
    want = ref.attention(f64(q[63 * new:]), kc, vc, d ** -0.5, ctx)
    assert np.abs(f64(all_[63]) - want).max() <= tolerance(vc)


def test_calls_on_another_stream():
    """Everything on a stream of the caller's, inputs made there too."""
    h, hk, d = 4, 2, 128
    note("attn another stream")
    lens = [150, 700]
    seqs = random_seqs(36, [x + 2 for x in lens], h, hk, d)
    A = Layer(h, hk, d, seqs)
    want = A.prefill(lens) + A.decode() + A.decode()
    B = Layer(h, hk, d, seqs)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = B.prefill(lens) + B.decode() + B.decode()
        torch.cuda.current_stream().synchronize()
    assert all(same_bits(a, b) for a, b in zip(want, got))


def test_one_and_no_tokens():
    """Batches without a token, of one token in all, and of empty sequences."""
    h, hk, d = 2, 1, 64
    note("attn no tokens")
    seqs = random_seqs(37, [1, 2, 0], h, hk, d)
    L = Layer(h, hk, d, seqs)
    assert all(len(x) == 0 for x in L.prefill([0, 0, 0]))
    a = L.prefill([1, 0, 0])
    assert same_bits(a[0][0], seqs[0][2][0].to(DEV).expand(h, d))  # one key: o = v
    b = L.prefill([0, 2, 0], max_new=2)
    assert same_bits(b[1][0], seqs[1][2][0].to(DEV).expand(h, d))
    k, v = L.read()
    for i in range(3):
        assert same_bits(k[i], seqs[i][1].to(DEV)) and same_bits(v[i], seqs[i][2].to(DEV))


@pytest.mark.parametrize("h,hk,n", [(4, 2, 2), (16, 8, 20)])  # keys split; rows split
def test_prefill_in_a_graph(h, hk, n):
    """Plan and prefill captured once; each replay appends the next tokens as the eager call does."""
    d, new = 64, 70
    note(f"attn prefill graph h={h} hk={hk} n={n}")
    seqs = random_seqs(38, [4 * new] * n, h, hk, d)
    E = Layer(h, hk, d, seqs)
    eager = [E.prefill([new] * n, max_new=new) for _ in range(4)]
    L = Layer(h, hk, d, seqs)
    (q, k, v), cu = L.pack([new] * n)
    plan = gdn.alloc_attn_plan(L.pool, n, n * new, L.slot_index)
    ws = gdn.alloc_attn_workspace(L.shape, gdn.GDN_ATTN_OP_PREFILL, n * new, n, L.cache.k8.shape[0], DEV)
    o = torch.empty_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        gdn.gdn_attn_plan(L.pool, cu, plan)
        gdn.gdn_attn_prefill(L.shape, q, k, v, cu, plan, L.cache, o, ws, max_new=new)
    for step in range(4):
        for to, x in zip((q, k, v), L.pack([new] * n)[0]):
            to.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        L.done = [x + new for x in L.done]
        assert same_bits(o, torch.cat(eager[step])), step
