"""GPU tests of how the calls of gdn_stack.h are used: rows alone and in a batch, strides and
alignment, streams, captured graphs, rows far apart, and a run of all of them together."""

import numpy as np
import pytest
import torch

import bitwise_invariant_gated_amd as gdn
from gpu_util import note
from oracle import stack as ref
from stack_util import DEV, add_norm, add_norm_bwd, dev, distill, distill_bwd, f64, logprobs, logprobs_bwd, new, same_bits
from test_gpu_stack_logits import check_backward, check_distill, check_forward, make, make_teacher

pytestmark = pytest.mark.gpu

B, F = torch.bfloat16, torch.float32


def everything(v, dtype, x, target, scale, ids, values, g, k=8):
    """All outputs of all calls on rows of logits."""
    s = gdn.LogitsShape(v, dtype, k)
    o = logprobs(s, x, target, scale)
    loss, stats = distill(s, x, ids, values, scale)
    return [o.logprobs, o.entropy, o.stats, o.top_ids, o.top_logprobs, logprobs_bwd(s, x, target, o, g, g, scale), loss, stats,
            distill_bwd(s, x, ids, values, stats, g, scale)]


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("v", [333, 2049, 10007])
def test_a_row_does_not_depend_on_the_others(v, dtype):
    """Nor on where it lies: odd vocabularies put rows at every alignment of an element."""
    note(f"rows alone {v} {dtype}")
    t = 23
    x, target, scale = make(t, v, dtype, seed=1, masked=True)
    ids, values = make_teacher(t, v, 8)
    g = dev(np.linspace(-1, 1, t))
    want = everything(v, dtype, x, target, scale, ids, values, g)
    assert all(same_bits(a, b) for a, b in zip(everything(v, dtype, x, target, scale, ids, values, g), want))
    for i in (0, 1, 2, 7, t - 1):
        one = [a[i:i + 1].clone() for a in (x, target, scale, ids, values, g)]
        assert all(same_bits(a, b[i:i + 1]) for a, b in zip(everything(v, dtype, *one), want)), i
    # rows of a wider array, from any element on; what is between them stays
    for lead, pad in ((1, 0), (3, 5), (8, 56)):
        wide = torch.full((t, lead + v + pad), 5.0, dtype=dtype, device=DEV)
        inside = wide[:, lead:lead + v]
        inside.copy_(x)
        got = everything(v, dtype, inside, target, scale, ids, values, g)
        assert all(same_bits(a, b) for a, b in zip(got, want)), (lead, pad)
        s = gdn.LogitsShape(v, dtype, 8)
        o = logprobs(s, inside, target, scale)
        logprobs_bwd(s, inside, target, o, g, g, scale, out=inside)
        assert same_bits(inside, want[5])
        assert (wide[:, :lead] == 5).all() and (wide[:, lead + v:] == 5).all()


@pytest.mark.parametrize("dtype", [B, F])
def test_many_short_rows(dtype):
    note(f"many rows {dtype}")
    t, v = 70001, 9
    x, target, scale = make(t, v, dtype, seed=2)
    s = gdn.LogitsShape(v, dtype, 3)
    o = logprobs(s, x, target, scale)
    some = [0, 1, 2, 3, 4, 5, 35000, 65535, 65536, t - 1]
    part = logprobs(s, x[some].clone(), target[some].clone(), scale[some].clone())
    for n in ("logprobs", "entropy", "stats", "top_ids", "top_logprobs"):
        assert same_bits(getattr(o, n)[some], getattr(part, n))
    check_forward(s, x[some], target[some], scale[some], part)
    best = x.float().amax(1)
    assert torch.equal(x.float().gather(1, o.top_ids[:, :1].long())[:, 0], best)


@pytest.mark.parametrize("dtype", [B, F])
def test_rows_past_32_bit_offsets(dtype):
    """Rows 2^30 elements apart: the last begin past 2^32 elements."""
    note(f"far rows {dtype}")
    v, t, far = 5000, 6, 1 << 30
    x, target, scale = make(t, v, dtype, seed=3)
    ids, values = make_teacher(t, v, 8)
    g = dev(np.ones(t))
    room = torch.empty((t - 1) * far + v, dtype=dtype, device=DEV)
    rows = room.as_strided((t, v), (far, 1))
    rows.copy_(x)
    want = everything(v, dtype, x, target, scale, ids, values, g)
    assert all(same_bits(a, b) for a, b in zip(everything(v, dtype, rows, target, scale, ids, values, g), want))
    s = gdn.LogitsShape(v, dtype, 8)
    o = logprobs(s, rows, target, scale)
    assert same_bits(logprobs_bwd(s, rows, target, o, g, g, scale, out=rows), want[5])
    rows.copy_(x)
    assert same_bits(distill_bwd(s, rows, ids, values, distill(s, rows, ids, values, scale)[1], g, scale, out=rows), want[8])
    n = gdn.NormShape(1000, dtype)
    a = room.as_strided((t, 1000), (far, 1))
    a.copy_(x[:, :1000])
    w = dev(np.ones(1000))
    h, y, _, _ = add_norm(n, x[:, :1000].contiguous(), None, w)
    gdn.gdn_stack_add_norm(n, a, a, w, a, new(t, 1000, dtype=dtype))
    assert same_bits(a, (x[:, :1000].float() * 2).to(dtype))


def test_no_rows():
    note("no rows")
    s = gdn.LogitsShape(100, B, 3)
    e, i, f = torch.empty(0, 100, dtype=B, device=DEV), torch.empty(0, dtype=torch.int32, device=DEV), torch.empty(0, device=DEV)
    o = logprobs(s, e, i, f)
    logprobs_bwd(s, e, i, o, f, f, f)
    loss, stats = distill(s, e, torch.empty(0, 3, dtype=torch.int32, device=DEV), torch.empty(0, 3, device=DEV), f)
    assert loss.numel() == 0 and stats.shape == (0, 4)


class Step:
    """A stack's end and its gradients on fixed buffers: norm, logits, log probabilities, divergence,
    their gradients, the norm's gradient."""

    def __init__(self, t=37, width=264, v=4100, k=8, seed=0):
        rng = np.random.default_rng(seed)
        self.norm, self.shape = gdn.NormShape(width), gdn.LogitsShape(v, B, k)
        self.x, self.res = dev(rng.standard_normal((t, width)), B), dev(rng.standard_normal((t, width)), B)
        self.w, self.head = dev(1 + 0.1 * rng.standard_normal(width)), dev(rng.standard_normal((width, v)) * 0.2, B)
        self.target = dev(rng.integers(0, v, t), torch.int32)
        self.ids, self.values = make_teacher(t, v, k, seed)
        self.g = dev(rng.standard_normal(t))
        self.h, self.y, self.dx = (torch.empty_like(self.x) for _ in range(3))
        self.logits, self.d1, self.d2 = (torch.empty(t, v, dtype=B, device=DEV) for _ in range(3))
        self.lp, self.en, self.loss = new(t), new(t), new(t)
        self.st, self.st4, self.top_lp, self.top = new(t, 2), new(t, 4), new(t, k), new(t, k, dtype=torch.int32)
        self.dw = new(width)
        self.ws = gdn.alloc_logits_workspace(self.shape, t, DEV)
        self.ws_n = gdn.alloc_norm_workspace(self.norm, t, DEV)

    def run(self, stream=None):
        n, s, kw = self.norm, self.shape, dict(stream=stream)
        gdn.gdn_stack_add_norm(n, self.x, self.res, self.w, self.h, self.y, **kw)
        torch.mm(self.y, self.head, out=self.logits)
        gdn.gdn_stack_logprobs(s, self.logits, self.target, self.lp, self.en, self.top, self.top_lp, self.st, self.ws, **kw)
        gdn.gdn_stack_distill(s, self.logits, self.ids, self.values, self.loss, self.st4, self.ws, **kw)
        gdn.gdn_stack_logprobs_bwd(s, self.logits, self.target, self.st, self.en, self.g, self.g, self.d1, **kw)
        gdn.gdn_stack_distill_bwd(s, self.logits, self.ids, self.values, self.st4, self.g, self.d2, **kw)
        dy = torch.mm(self.d1, self.head.t())
        gdn.gdn_stack_add_norm_bwd(n, self.h, self.w, dy, self.res, self.dx, None, self.dw, self.ws_n, **kw)

    def outputs(self):
        return [t.clone() for t in (self.h, self.y, self.logits, self.lp, self.en, self.top, self.top_lp, self.st, self.loss, self.st4, self.d1,
                                    self.d2, self.dx, self.dw)]

    def forget(self):
        for t in (self.h, self.y, self.logits, self.lp, self.en, self.top_lp, self.st, self.loss, self.st4, self.d1, self.d2, self.dx, self.dw):
            t.fill_(float("nan"))
        self.top.fill_(99)
        self.ws.fill_(0xff)
        self.ws_n.fill_(0xff)


def test_run_together_against_the_oracle():
    note("stack's end")
    c = Step()
    c.run()
    check_forward(c.shape, c.logits, c.target, None, _named(c))
    check_distill(c.shape, c.logits, c.ids, c.values, None, c.loss, c.d2, c.g)
    check_backward(c.shape, c.logits, c.target, None, c.g, c.g, c.d1)
    want = ref.add_norm(f64(c.h), f64(c.w), 1e-6)
    assert (np.abs(f64(c.y) - want) <= 2.0 ** -8 * np.abs(want)).all()


def _named(c):
    class O:
        logprobs, entropy, stats, top_ids, top_logprobs = c.lp, c.en, c.st, c.top, c.top_lp
    return O


def test_captured_and_replayed():
    """Two graphs that share workspaces, replayed in turn with eager work and synchronisations between."""
    note("graphs")
    a, b = Step(seed=1), Step(t=5, width=2056, v=10007, k=8, seed=2)
    big = max(a.ws.numel(), b.ws.numel())
    a.ws = b.ws = torch.empty(big, dtype=torch.uint8, device=DEV)
    a.ws_n = b.ws_n = torch.empty(max(a.ws_n.numel(), b.ws_n.numel()), dtype=torch.uint8, device=DEV)
    wants = []
    for c in (a, b):
        c.run()
        wants.append(c.outputs())
    graphs = []
    for c in (a, b):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            c.run()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    for turn in range(3):
        for c, g, want in ((a, graphs[0], wants[0]), (b, graphs[1], wants[1])):
            c.forget()
            g.replay()
            assert all(same_bits(x, y) for x, y in zip(c.outputs(), want)), turn
        torch.cuda.synchronize()
        if turn == 1:  # new inputs in the same places
            for i, c in enumerate((a, b)):
                c.x.mul_(-0.5)
                c.run()
                wants[i] = c.outputs()


def test_on_other_streams_at_once():
    note("two streams")
    steps = [Step(seed=s) for s in (3, 4)]
    wants = []
    for c in steps:
        c.run()
        wants.append(c.outputs())
        c.forget()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(3):
        for c, st in zip(steps, streams):
            with torch.cuda.stream(st):
                c.run()
    torch.cuda.synchronize()
    for c, want in zip(steps, wants):
        assert all(same_bits(x, y) for x, y in zip(c.outputs(), want))
    # a stream given by hand, current or not
    c = steps[0]
    n = c.norm
    c.h.fill_(float("nan"))
    torch.cuda.synchronize()
    gdn.gdn_stack_add_norm(n, c.x, c.res, c.w, c.h, c.y, stream=streams[1])
    streams[1].synchronize()
    assert same_bits(c.h, wants[0][0])


def test_rows_of_larger_arrays():
    """Any rows of the logits with the same rows of what goes with them, at the alignment of an element."""
    note("later rows")
    t, v = 13, 10007
    for dtype in (B, F):
        x, target, scale = make(t, v, dtype, seed=5)
        ids, values = make_teacher(t, v, 7)
        g = dev(np.linspace(-1, 1, t))
        want = everything(v, dtype, x, target, scale, ids, values, g, k=7)
        for a in (1, 2, 3, 5):
            got = everything(v, dtype, *(u[a:] for u in (x, target, scale, ids, values, g)), k=7)
            assert all(same_bits(p, q[a:]) for p, q in zip(got, want)), a
