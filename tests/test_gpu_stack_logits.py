"""GPU tests of log probabilities, entropy, top alternatives and distillation, with their gradients,
against the fp64 oracle."""

import numpy as np
import pytest
import torch

import bitwise_invariant_gated_amd as gdn
from gpu_util import note
from oracle import stack as ref
from stack_util import (DEV, U, dev, distill, distill_bwd, entropy_bound, f64, half, log_q_bound, logprobs, logprobs_bwd, new,
                        same_bits)

pytestmark = pytest.mark.gpu

B, F = torch.bfloat16, torch.float32
INF = float("inf")
# at, before and behind the borders of a vector, a group and a part, and a row of many parts
VOCABS = [1, 2, 7, 8, 9, 100, 128, 129, 511, 1024, 1025, 2047, 2048, 2049, 4100, 8192, 8193, 10007, 131072, 131080]


def make(t, v, dtype, seed=0, masked=False, std=2.5):
    rng = np.random.default_rng(seed + 31 * t + v)
    x = rng.standard_normal((t, v)) * std
    x[np.arange(t), rng.integers(0, v, t)] += rng.random(t) * 14
    if masked:
        x[::2][rng.random((len(x[::2]), v)) < 0.5] = -np.inf
    target = rng.integers(0, v, t)
    return dev(x, dtype), dev(target, torch.int32), dev(0.5 + rng.random(t))


def rows(x, scale):
    """(logits, scale, z, log q) of every row, in 64 bits."""
    x = f64(x)
    s = np.ones(len(x)) if scale is None else f64(scale)
    for row, c in zip(x, s):
        m = row.max()
        yield row, c, (row - (0 if m == -np.inf else m)) * c, ref.log_softmax(row * c)


def near(got, want, bound):
    """Within the bound; infinities and what is not a number in the same places."""
    got, want = np.atleast_1d(got), np.atleast_1d(want)
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine], want[~fine], equal_nan=True)
    assert (np.abs(got[fine] - want[fine]) <= np.broadcast_to(bound, want.shape)[fine]).all(), (got, want)


def check_forward(s, x, target, scale, o, left=()):
    for i, (row, c, z, logq) in enumerate(rows(x, scale)):
        if i in left:
            assert o.logprobs[i] == 0 and o.entropy[i] == 0 and (o.stats[i] == 0).all()
            assert not s.top or ((o.top_ids[i] == -1).all() and (o.top_logprobs[i] == 0).all())
            continue
        bound = log_q_bound(z, logq)
        if target is not None:
            near(f64(o.logprobs[i]), logq[int(target[i])], bound[int(target[i])])
        near(f64(o.entropy[i]), ref.entropy(logq), entropy_bound(z, logq))
        m = row.max()
        assert float(o.stats[i, 0]) == m
        log_l = 0.0 if m == -np.inf else -logq.max()
        near(f64(o.stats[i, 1]), log_l, bound.max() if m == -np.inf else bound[row.argmax()])
        if s.top:
            want = ref.top(row, s.top)
            assert o.top_ids[i].tolist() == want.tolist()
            near(f64(o.top_logprobs[i]), logq[want], bound[want])


@pytest.mark.parametrize("v", VOCABS)
@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("masked", [False, True])
def test_forward(v, dtype, masked):
    for t, top in ((1, 1), (5, min(5, v)), (3, min(64, v))):
        note(f"logprobs {t} x {v} {dtype} top {top} masked={masked}")
        x, target, scale = make(t, v, dtype, masked=masked)
        s = gdn.LogitsShape(v, dtype, top)
        for sc in (scale, None):
            o = logprobs(s, x, target, sc)
            check_forward(s, x, target, sc, o)
        # fewer outputs: the same bits
        p = logprobs(gdn.LogitsShape(v, dtype), x, target, None, entropy=False)
        assert same_bits(p.logprobs, o.logprobs) and same_bits(p.stats, o.stats)
        p = logprobs(s, x, None, None, stats=False)
        assert same_bits(p.entropy, o.entropy) and same_bits(p.top_ids, o.top_ids) and same_bits(p.top_logprobs, o.top_logprobs)


def test_longest_vocabulary():
    v = 1 << 20
    for dtype in (B, F):
        note(f"logprobs 2 x {v} {dtype}")
        x, target, scale = make(2, v, dtype)
        s = gdn.LogitsShape(v, dtype, 64)
        o = logprobs(s, x, target, scale)
        check_forward(s, x, target, scale, o)


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("v", [40, 5000, 20000])
def test_equal_logits(v, dtype):
    """Ties go to the lowest index, also where they overflow what is held while the best are sought."""
    note(f"logprobs ties {v} {dtype}")
    rng = np.random.default_rng(v)
    x = np.zeros((7, v))
    x[1] = rng.integers(0, 2, v)
    x[2] = rng.integers(0, 3, v) * -1.0
    x[3, v // 2:] = 1
    x[4] = -np.arange(v) % 7
    x[5] = np.where(rng.random(v) < 0.5, 0.0, -0.0)
    x[6] = np.where(rng.random(v) < 0.01, -1.0, -np.inf)
    x[6, :3] = -np.inf
    x = dev(x, dtype)
    for top in (1, 20, min(64, v)):
        s = gdn.LogitsShape(v, dtype, top)
        o = logprobs(s, x, dev(np.full(7, v - 1), torch.int32))
        check_forward(s, x, dev(np.full(7, v - 1), torch.int32), None, o)


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("v", [100, 1025, 6000, 20000, 200000])
def test_ascending_logits(v, dtype):
    """Each better than all before it."""
    note(f"logprobs ascending {v} {dtype}")
    x = dev(np.stack([np.arange(v) * 0.01, -np.arange(v) * 0.01]), dtype)
    for top in (3, 64):
        s = gdn.LogitsShape(v, dtype, top)
        t = dev(np.array([v - 2, 1]), torch.int32)
        check_forward(s, x, t, None, logprobs(s, x, t))


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("v", [64, 1024, 1025, 8192, 8193, 131073, 300000])
def test_few_tokens_left(v, dtype):
    """A grammar leaves three tokens of the vocabulary, or none; all the best lie together, or all
    in one block; more alternatives are asked for than have any probability."""
    note(f"logprobs few left {v} {dtype}")
    rng = np.random.default_rng(v)
    x = np.full((5, v), -np.inf)
    x[0, rng.permutation(v)[:3]] = [1, -2, 1]
    x[2] = rng.standard_normal(v)
    x[2, v // 3: v // 3 + 130] += 20
    x[3] = rng.standard_normal(v)
    x[3, :min(v, 9000)] += 8 + 0.001 * np.arange(min(v, 9000))
    x[4] = -3
    x[4, v - 1] = -2
    x = dev(x, dtype)
    t = dev(np.argmax(f64(x), 1), torch.int32)
    for top in (1, 20, 64):
        s = gdn.LogitsShape(v, dtype, top)
        check_forward(s, x, t, None, logprobs(s, x, t))


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("v", [50, 5000])
def test_masked_and_special_rows(v, dtype):
    note(f"logprobs special {v} {dtype}")
    low = torch.finfo(dtype).min
    x, _, _ = make(9, v, dtype, seed=4)
    x[0] = -INF                      # nothing left
    x[1] = -INF
    x[1, v - 1] = 3                  # one token left
    x[2] = low                       # the type's lowest everywhere
    x[3, : v - 2] = low              # and almost everywhere
    x[4, 1] = float("nan")
    x[5, v - 2] = INF
    x[6, 2:] = torch.finfo(dtype).max
    x[7] = -INF
    x[7, 3] = float("nan")
    target = dev(np.array([1, v - 1, 0, v - 1, 0, 0, 3, 0, 2]), torch.int32)
    s = gdn.LogitsShape(v, dtype, 4)
    o = logprobs(s, x, target)
    want = x.clone()
    sane = [0, 1, 2, 3, 6, 8]
    pick = Part(o, sane)
    check_forward(s, want[sane], target[sane], None, pick)
    for i in (4, 5, 7):
        assert torch.isnan(o.logprobs[i]) and torch.isnan(o.entropy[i]) and torch.isnan(o.top_logprobs[i]).all()
    for i in (4, 5):  # a NaN ranks as -inf
        row = f64(x[i])
        assert o.top_ids[i].tolist() == ref.top(np.where(np.isnan(row), -np.inf, row), 4).tolist()
    # a masked token's own log probability
    o2 = logprobs(s, x, dev(np.full(9, 0), torch.int32))
    assert o2.logprobs[1] == -INF
    # gradients
    g, f = dev(np.linspace(0.5, 1.5, 9)), dev(np.linspace(-1, 1, 9))
    d = logprobs_bwd(s, x, target, o, g, f)
    assert (d[0] == 0).all()
    for i in (4, 5, 7):
        assert torch.isnan(d[i]).any()
    check_backward(s, x[sane], target[sane], None, g[sane], f[sane], d[sane])


class Part:
    def __init__(self, o, idx):
        for n, t in vars(o).items():
            setattr(self, n, None if t is None else t[idx])


def check_backward(s, x, target, scale, g, f, d):
    g = np.zeros(len(x)) if g is None else f64(g)
    f = np.zeros(len(x)) if f is None else f64(f)
    for i, (row, c, z, logq) in enumerate(rows(x, scale)):
        at = None if target is None else int(target[i])
        want = ref.logprobs_backward(row, c, at, g[i], f[i])
        q, h = np.exp(logq), ref.entropy(logq) if logq.max() > -np.inf else 0.0
        b = log_q_bound(z, logq) + 4 * U
        lq = np.where(logq > -np.inf, logq, 0)
        size = q * (abs(g[i]) * b + abs(f[i]) * (np.abs(lq + h) * b + b + entropy_bound(z, logq) + 8 * U * (np.abs(lq) + h + np.abs(lq + h))))
        size = c * (size + 8 * U * q * abs(g[i]))
        if at is not None:
            size[at] += 8 * U * c * abs(g[i])
        got = f64(d[i])
        assert (np.abs(got - want) <= half(s.dtype) * np.abs(want) * (1 + 2.0 ** -7) + 2 * size + 1e-37).all(), i


@pytest.mark.parametrize("v", VOCABS)
@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("masked", [False, True])
def test_backward(v, dtype, masked):
    note(f"logprobs_bwd {v} {dtype} masked={masked}")
    x, target, scale = make(4, v, dtype, seed=2, masked=masked)
    s = gdn.LogitsShape(v, dtype)
    rng = np.random.default_rng(v)
    g, f = dev(rng.standard_normal(4)), dev(rng.standard_normal(4))
    for sc, gg, ff in ((scale, g, f), (None, g, None), (scale, None, f)):
        o = logprobs(s, x, target, sc)
        d = logprobs_bwd(s, x, target, o, gg, ff, sc)
        check_backward(s, x, target if gg is not None else None, sc, gg, ff, d)
        assert same_bits(logprobs_bwd(s, x.clone(), target, o, gg, ff, sc), d)
        y = x.clone()  # in place
        assert same_bits(logprobs_bwd(s, y, target, o, gg, ff, sc, out=y), d)
    o = logprobs(s, x, None)
    check_backward(s, x, None, None, None, f, logprobs_bwd(s, x, None, o, None, f))


@pytest.mark.parametrize("dtype", [B, F])
def test_rows_left_out(dtype):
    """Padding of a batch: not read (it may hold anything), zeros in every output."""
    note(f"logprobs left out {dtype}")
    v = 3000
    x, target, scale = make(8, v, dtype, seed=6)
    for i, t in ((0, -1), (3, v), (4, 1 << 30), (7, -(1 << 31))):
        target[i] = t
        x[i] = float("nan")
        scale[i] = float("nan")
    left = (0, 3, 4, 7)
    s = gdn.LogitsShape(v, dtype, 6)
    o = logprobs(s, x, target, scale)
    check_forward(s, x, target, scale, o, left)
    g, f = dev(np.ones(8)), dev(np.ones(8))
    for i in left:
        g[i] = float("nan")
    d = logprobs_bwd(s, x, target, o, g, f, scale)
    assert (d[list(left)] == 0).all()
    keep = [1, 2, 5, 6]
    check_backward(s, x[keep], target[keep], scale[keep], g[keep], f[keep], d[keep])


def make_teacher(t, v, k, seed=0, given=False):
    rng = np.random.default_rng(seed + v + k)
    ids = np.stack([rng.permutation(v)[:k] if k <= v else rng.integers(0, v, k) for _ in range(t)])
    values = rng.standard_normal((t, k)) * 3
    if given:
        values = values - 2 - np.log(np.exp(values).sum(-1, keepdims=True))
    return dev(ids, torch.int32), dev(values)


def check_distill(s, x, ids, values, scale, loss, d=None, g=None):
    for i, (row, c, z, logq) in enumerate(rows(x, scale)):
        who, logp = ref.teacher(f64(ids[i]).astype(int), f64(values[i]), s.vocab, c, s.teacher_logprobs)
        b = log_q_bound(z, logq) + 4 * U
        some = logp > -np.inf
        p = np.where(some, np.exp(logp), 0)
        alp = np.where(some, np.abs(logp), 0)
        # log p: a difference, a product and the sum of up to 256 exponentials, as log q's
        zt = np.abs(logp - logp.max()) if some.any() else np.zeros_like(logp)
        bp = U * (64 + 16 * np.where(some, zt, 0) + 16 * np.sum(p * np.where(some, zt, 0)) + 4 * alp)
        lq = np.where(logq[who] > -np.inf, logq[who], 0)
        near(f64(loss[i]), ref.distill(row, c, f64(ids[i]).astype(int), f64(values[i]), s.teacher_logprobs),
             2 * np.sum(p * ((bp + b[who]) * (1 + np.abs(alp + lq)) + 16 * U * (alp + np.abs(lq)))) + 1e-37)
        if d is None:
            continue
        gi = f64(g)[i]
        want = ref.distill_backward(row, c, f64(ids[i]).astype(int), f64(values[i]), s.teacher_logprobs, gi)
        q = np.exp(logq)
        size = q * p.sum() * (b + 16 * U + (np.sum(p * bp) / p.sum() if p.sum() > 0 else 0))
        for e, pe, be in zip(who, p, bp):
            size[e] += pe * (be + 16 * U)
        got = f64(d[i])
        assert (np.abs(got - want) <= half(s.dtype) * np.abs(want) * (1 + 2.0 ** -7) + 2 * abs(gi) * c * size + 1e-37).all(), i


@pytest.mark.parametrize("v", VOCABS)
@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("given", [False, True])
def test_distill(v, dtype, given):
    for k in sorted({1, min(v, 5), min(v, 64), 65, 256}):
        note(f"distill 3 x {v} {dtype} top {k} given={given}")
        x, _, scale = make(3, v, dtype, seed=8)
        ids, values = make_teacher(3, v, k, given=given)
        s = gdn.LogitsShape(v, dtype, k, given)
        g = dev(np.array([1.0, -0.5, 2.0]))
        for sc in (scale, None):
            loss, stats = distill(s, x, ids, values, sc)
            d = distill_bwd(s, x, ids, values, stats, g, sc)
            check_distill(s, x, ids, values, sc, loss, d, g)
        y = x.clone()
        assert same_bits(distill_bwd(s, y, ids, values, stats, g, None, out=y), d)


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("given", [False, True])
def test_distill_entries(dtype, given):
    """Entries that are not there, that come twice, that weigh nothing; masked students."""
    note(f"distill entries {dtype} given={given}")
    v, k = 5000, 70
    x, _, scale = make(9, v, dtype, seed=10)
    ids, values = make_teacher(9, v, k, seed=1, given=given)
    ids[0] = -1                       # no teacher
    x[0, 3] = float("nan")
    ids[1, ::2], ids[1, 1] = -1, v    # some
    values[1, ::2] = float("nan")
    ids[2] = 17                       # one index, over and over
    ids[3, 10:40] = ids[3, 9]
    ids[3, 69] = ids[3, 0]
    values[4, 1:] = -INF              # all weight on one
    values[5] = -INF                  # none at all
    x[6, ids[6, 4].long()] = -INF     # a q of 0 where p is not
    x[7] = -INF                       # a student without a token
    x[8, : v // 2] = -INF
    ids[8] = torch.where(ids[8] < v // 2, -5, ids[8])
    s = gdn.LogitsShape(v, dtype, k, given)
    g = dev(np.linspace(0.5, 1, 9))
    loss, stats = distill(s, x, ids, values, scale)
    d = distill_bwd(s, x, ids, values, stats, g, scale)
    assert loss[0] == 0 and (d[0] == 0).all() and loss[5] == 0 and (d[5] == 0).all()
    assert loss[6] == INF and loss[7] == INF and (d[7] == 0).all() and torch.isfinite(d[6]).all()
    sane = [1, 2, 3, 4, 5, 6, 7, 8]
    values[1, ::2] = 0
    check_distill(s, x[sane], ids[sane], values[sane], scale[sane], loss[sane], d[sane], g[sane])


def test_gradients_are_the_differences():
    """By central differences of the fp64 value of the loss that the call gives."""
    v, k = 600, 9
    x, target, scale = make(2, v, F, seed=12, std=1.0)
    ids, values = make_teacher(2, v, k, seed=3)
    rng = np.random.default_rng(0)
    note("logits differences")
    s = gdn.LogitsShape(v, F, k)
    o = logprobs(gdn.LogitsShape(v, F), x, target, scale)
    one = dev(np.ones(2))
    d = [f64(logprobs_bwd(s, x, target, o, one, one, scale)), f64(distill_bwd(s, x, ids, values, distill(s, x, ids, values, scale)[1], one, scale))]
    xs, sc = f64(x), f64(scale)
    for _ in range(4):
        n = rng.standard_normal((2, v))
        e = 1e-5
        for which in range(2):
            got = []
            for sign in (1, -1):
                total = 0.0
                for i in range(2):
                    z = xs[i] + sign * e * n[i]
                    if which:
                        total += ref.distill(z, sc[i], f64(ids[i]).astype(int), f64(values[i]), False)
                    else:
                        logq = ref.log_softmax(z * sc[i])
                        total += logq[int(target[i])] + ref.entropy(logq)
                got.append(total)
            want = (got[0] - got[1]) / (2 * e)
            assert abs((d[which] * n).sum() - want) <= 1e-5 * np.sqrt(v)
