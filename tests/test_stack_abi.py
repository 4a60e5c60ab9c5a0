"""Checks of include/gdn_stack.h and its binding that need no GPU: symbols, workspace sizes, copies
and the refusal of bad arguments (no call here reaches a kernel launch)."""

import copy
import ctypes
import os
import pickle
import re

import pytest
import torch

import bitwise_invariant_gated_amd as gdn
from bitwise_invariant_gated_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000  # 16-byte aligned, never dereferenced: validation fails first
OK, INVALID, UNSUPPORTED, WORKSPACE = _lib.GDN_OK, _lib.GDN_ERR_INVALID_ARG, _lib.GDN_ERR_UNSUPPORTED, _lib.GDN_ERR_WORKSPACE
F32, BF16 = _lib.GDN_DTYPE_F32, _lib.GDN_DTYPE_BF16
BIG = 1 << 40


@pytest.fixture
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("library not built")
    return _lib.load()


def said(lib):
    return lib.gdn_cpr_last_error().decode()


def ref(x):
    return None if x is None else ctypes.byref(x)


def norm(width=64, dtype=BF16, residual=BF16, group=-1, zero=0, eps=1e-6):
    return _lib.NormShapeC(width, dtype, residual, group, zero, eps)


def logits(vocab=100, dtype=BF16, top=0, given=0):
    return _lib.LogitsShapeC(vocab, dtype, top, given)


def test_header_declares_exactly_the_bound_symbols(lib):
    with open(os.path.join(ROOT, "include", "gdn_stack.h")) as f:
        text = f.read()
    assert set(re.findall(r"\b(gdn_stack_[a-z_]+)\s*\(", text)) == set(_lib.STACK_EXPORTED)
    for name in _lib.STACK_EXPORTED:
        assert hasattr(lib, name), name


def test_workspace_sizes(lib):
    size = lib.gdn_stack_norm_workspace_size
    assert size(ref(norm(2048)), 1) >= 2048 * 4 and size(ref(norm(2048)), 1 << 20) >= 2048 * 4
    assert size(ref(norm(2048)), 0) > 0 and size(ref(norm(2048)), -1) == 0 and size(ref(norm(7)), 1) == 0 and size(None, 1) == 0
    size = lib.gdn_stack_logits_workspace_size
    assert size(ref(logits(5000)), 10) >= 10 * 3 * 16
    assert size(ref(logits(5000, top=3)), 10) >= 10 * 3 * (16 + 16 * 4)
    assert size(ref(logits(5000)), 0) > 0 and size(ref(logits(5000)), -1) == 0 and size(ref(logits(0)), 1) == 0 and size(None, 1) == 0
    assert size(ref(logits(1 << 20)), 1 << 28) == 0  # more parts than a launch can count


BAD_NORMS = [dict(width=0), dict(width=4), dict(width=12), dict(width=16392), dict(dtype=2), dict(residual=3),
             dict(dtype=F32, residual=BF16), dict(group=64), dict(group=-2), dict(width=64, group=128)]
BAD_LOGITS = [dict(vocab=0), dict(vocab=-1), dict(vocab=(1 << 20) + 1), dict(dtype=5), dict(top=-1), dict(top=257)]


@pytest.mark.parametrize("kw", BAD_NORMS)
def test_norm_shapes_refused(lib, kw):
    s = norm(**kw)
    assert lib.gdn_stack_add_norm(ref(s), 4, P, 0, P, 0, P, P, 0, P, 0, None, None, None) == UNSUPPORTED and said(lib)
    assert lib.gdn_stack_add_norm_bwd(ref(s), 4, P, 0, P, P, 0, P, 0, P, 0, None, 0, P, P, BIG, None) == UNSUPPORTED


@pytest.mark.parametrize("kw", BAD_LOGITS)
def test_logits_shapes_refused(lib, kw):
    s = logits(**kw)
    assert lib.gdn_stack_logprobs(ref(s), 4, P, 0, P, None, P, P, P, P, P, P, BIG, None) == UNSUPPORTED and said(lib)
    assert lib.gdn_stack_logprobs_bwd(ref(s), 4, P, 0, P, None, P, P, P, P, P, 0, None) == UNSUPPORTED
    assert lib.gdn_stack_distill(ref(s), 4, P, 0, P, P, None, P, P, P, BIG, None) == UNSUPPORTED
    assert lib.gdn_stack_distill_bwd(ref(s), 4, P, 0, P, P, None, P, P, P, 0, None) == UNSUPPORTED


def test_add_norm_refusals(lib):
    def call(s=norm(), n=4, x=P, xs=0, r=2 * P, rs=0, w=P, h=3 * P, hs=0, y=4 * P, ys=0, y8=None, sc=None):
        return lib.gdn_stack_add_norm(ref(s), n, x, xs, r, rs, w, h, hs, y, ys, y8, sc, None)

    assert call(s=None) == INVALID and call(n=-1) == INVALID and call(n=1 << 31) == UNSUPPORTED
    for eps in (-1.0, float("nan"), float("inf")):
        assert call(s=norm(eps=eps)) == INVALID and "eps" in said(lib)
    for kw, name in ((dict(x=None), "x is"), (dict(w=None), "w is"), (dict(x=P + 8), "x is"), (dict(r=P + 2), "residual"),
                     (dict(h=P + 4), "residual_out"), (dict(y=P + 4), "y is"), (dict(y8=P + 4, sc=P, s=norm(128, group=0)), "y8"),
                     (dict(xs=56), "x_stride"), (dict(rs=68), "residual_stride"), (dict(hs=-64), "residual_out_stride"),
                     (dict(ys=65), "y_stride"), (dict(y=None), "both"), (dict(y8=P), "together"), (dict(sc=P), "together"),
                     (dict(y8=5 * P, sc=6 * P), "group"), (dict(y=3 * P), "residual_out")):
        assert call(**kw) == INVALID and name in said(lib), kw
    # in place: the same rows, or none of them
    assert call(h=P, hs=72) == INVALID and call(y=P, ys=72) == INVALID and call(h=2 * P, hs=72) == INVALID
    assert call(s=norm(residual=F32), h=P) == INVALID and call(s=norm(residual=F32), y=2 * P) == INVALID
    assert call(n=0, x=None, y=None) == OK
    # a launch's threads are counted in 32 bits
    assert call(s=norm(4096), n=(1 << 24) - 15) == UNSUPPORTED and "too many" in said(lib)


def test_add_norm_bwd_refusals(lib):
    def call(s=norm(), n=4, h=P, hs=0, w=P, dy=2 * P, ys=0, dr=3 * P, rs=0, dx=4 * P, xs=0, dd=None, ds=0, dw=P, ws=P, size=BIG):
        return lib.gdn_stack_add_norm_bwd(ref(s), n, h, hs, w, dy, ys, dr, rs, dx, xs, dd, ds, dw, ws, size, None)

    assert call(s=None) == INVALID and call(n=-1) == INVALID
    for kw, name in ((dict(h=None), "h is"), (dict(w=None), "w is"), (dict(dy=None), "dy"), (dict(dw=None), "dw"), (dict(dx=None), "both"),
                     (dict(dx=P + 2), "dx"), (dict(dd=P + 2), "d_residual"), (dict(dr=P + 2), "d_residual_out"), (dict(dd=4 * P), "dx is"),
                     (dict(hs=9), "h_stride"), (dict(ys=32), "dy_stride"), (dict(xs=68), "dx_stride"), (dict(ds=68), "d_residual_stride"),
                     (dict(rs=68), "d_residual_out_stride")):
        assert call(**kw) == INVALID and name in said(lib), kw
    assert call(dx=2 * P, xs=72) == INVALID and call(dx=P, xs=72) == INVALID and call(dd=3 * P, ds=72) == INVALID
    assert call(s=norm(residual=F32), dx=P) == INVALID and call(s=norm(residual=F32), dd=2 * P) == INVALID
    assert call(ws=None) == WORKSPACE and call(size=64) == WORKSPACE and call(ws=P + 8) == INVALID


def test_logprobs_refusals(lib):
    def call(s=logits(top=3), n=4, x=P, xs=0, t=P, sc=P, lp=P, en=P, ids=P, tlp=P, st=P, ws=P, size=BIG):
        return lib.gdn_stack_logprobs(ref(s), n, x, xs, t, sc, lp, en, ids, tlp, st, ws, size, None)

    assert call(s=None) == INVALID and call(n=-1) == INVALID and call(n=1 << 31) == UNSUPPORTED
    assert call(s=logits(top=65)) == UNSUPPORTED and call(s=logits(vocab=2, top=3)) == UNSUPPORTED and "top" in said(lib)
    for kw, name in ((dict(x=None), "logits"), (dict(x=P + 1), "logits"), (dict(x=P + 2, s=logits(dtype=F32)), "logits"), (dict(xs=99), "logits_stride"),
                     (dict(t=P + 2), "targets"), (dict(sc=P + 2), "scale"), (dict(lp=P + 2), "logprobs"), (dict(en=P + 2), "entropy"),
                     (dict(ids=P + 2), "top_ids"), (dict(tlp=P + 2), "top_logprobs"), (dict(st=P + 2), "stats"), (dict(t=None), "together"),
                     (dict(lp=None), "together"), (dict(ids=None), "top_ids"), (dict(tlp=None), "top_logprobs"),
                     (dict(s=logits(), t=None, lp=None, en=None, st=None), "no output")):
        assert call(**kw) == INVALID and name in said(lib), kw
    assert call(ws=None) == WORKSPACE and call(size=100) == WORKSPACE and call(ws=P + 8) == INVALID
    assert call(n=0, x=None) == OK
    assert call(s=logits(vocab=9, top=3), n=(1 << 26) - 63) == UNSUPPORTED and "too many" in said(lib)
    assert call(s=logits(vocab=4097, top=3), n=1 << 25) == UNSUPPORTED


def test_logprobs_bwd_refusals(lib):
    def call(s=logits(), n=4, x=P, xs=0, t=P, sc=None, st=P, en=P, g=P, f=P, d=2 * P, ds=0):
        return lib.gdn_stack_logprobs_bwd(ref(s), n, x, xs, t, sc, st, en, g, f, d, ds, None)

    for kw, name in ((dict(x=None), "logits"), (dict(d=None), "d_logits"), (dict(d=P + 1), "d_logits"), (dict(ds=50), "d_logits_stride"), (dict(st=None), "stats"),
                     (dict(g=None, f=None), "both"), (dict(t=None), "targets"), (dict(en=None), "entropy"), (dict(d=P, ds=101), "in place"),
                     (dict(g=P + 2), "d_logprobs"), (dict(f=P + 2), "d_entropy"), (dict(en=P + 2), "entropy"), (dict(t=P + 2), "targets")):
        assert call(**kw) == INVALID and name in said(lib), kw
    assert call(n=0, x=None, d=None) == OK


def test_distill_refusals(lib):
    def call(s=logits(top=3), n=4, x=P, xs=0, ids=P, v=P, sc=None, loss=P, st=P, ws=P, size=BIG):
        return lib.gdn_stack_distill(ref(s), n, x, xs, ids, v, sc, loss, st, ws, size, None)

    def back(s=logits(top=3), n=4, x=P, xs=0, ids=P, v=P, sc=None, st=P, g=P, d=2 * P, ds=0):
        return lib.gdn_stack_distill_bwd(ref(s), n, x, xs, ids, v, sc, st, g, d, ds, None)

    assert call(s=logits(top=0)) == UNSUPPORTED and back(s=logits(top=0)) == UNSUPPORTED
    for kw, name in ((dict(x=None), "logits"), (dict(ids=None), "teacher_ids"), (dict(v=None), "teacher_values"), (dict(loss=None), "loss"),
                     (dict(ids=P + 2), "teacher_ids"), (dict(st=P + 8), "stats"), (dict(xs=3), "logits_stride")):
        assert call(**kw) == INVALID and name in said(lib), kw
    assert call(ws=None) == WORKSPACE and call(size=10) == WORKSPACE
    for kw, name in ((dict(x=None), "logits"), (dict(ids=None), "teacher_ids"), (dict(v=None), "teacher_values"), (dict(g=None), "d_loss"), (dict(st=None), "stats"),
                     (dict(d=None), "d_logits"), (dict(d=P, ds=128), "in place"), (dict(ds=3), "d_logits_stride")):
        assert back(**kw) == INVALID and name in said(lib), kw


WRONG = "expected|contiguous|overlap"


def test_binding_refusals(lib):
    """Tensors of another shape, type or layout are refused before the library sees them."""
    s = gdn.NormShape(64)
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64)
    for bad in (x.float(), x[:, :32], x.t(), x[None], x.expand(1, 4, 64)[0][:1].expand(4, 64)):
        with pytest.raises(ValueError, match=WRONG):
            gdn.gdn_stack_add_norm(s, bad, None, w, None, x)
    for kw in (dict(residual=x[:3]), dict(residual_out=x.float()), dict(y=x[:2]), dict(w=w[:8]), dict(w=w.double()), dict(w=torch.ones(128)[::2]),
               dict(y8=torch.zeros(4, 64)), dict(y_scale=torch.zeros(4))):
        args = dict(residual=None, w=w, residual_out=None, y=x)
        args.update(kw)
        with pytest.raises(ValueError, match=WRONG):
            gdn.gdn_stack_add_norm(s, x, **args)
    z = gdn.LogitsShape(100, torch.float32, top=2)
    lg, i, f, ws = torch.zeros(4, 100), torch.zeros(4, dtype=torch.int32), torch.zeros(4), torch.zeros(1 << 12, dtype=torch.uint8)
    good = dict(logits=lg, targets=i, logprobs=f, entropy=f, top_ids=torch.zeros(4, 2, dtype=torch.int32), top_logprobs=torch.zeros(4, 2),
                stats=torch.zeros(4, 2), workspace=ws)
    for kw in (dict(logits=lg[:, :99]), dict(logits=lg.bfloat16()), dict(targets=i.long()), dict(targets=i[:3]), dict(logprobs=f[:2]),
               dict(top_ids=good["top_ids"].t()), dict(top_logprobs=torch.zeros(4, 3)), dict(stats=f), dict(scale=f[:1])):
        with pytest.raises(ValueError, match=WRONG):
            gdn.gdn_stack_logprobs(z, **{**good, **kw})
    with pytest.raises(ValueError, match="workspace"):
        gdn.gdn_stack_logprobs(z, **{**good, "workspace": ws[::2]})
    with pytest.raises(ValueError, match=WRONG):
        gdn.gdn_stack_distill(z, lg, good["top_ids"].long(), good["top_logprobs"], f, None, ws)
    with pytest.raises(ValueError, match=WRONG):
        gdn.gdn_stack_distill_bwd(z, lg, good["top_ids"], good["top_logprobs"], torch.zeros(4, 2), f, lg)
    with pytest.raises(ValueError, match="unsupported"):
        gdn.LogitsShape(10, torch.float16)
    with pytest.raises(ValueError, match="unsupported"):
        gdn.NormShape(64, torch.bfloat16, torch.float64)


def test_tensors_off_the_current_device_are_refused(lib):
    """Kernels run on the current device: memory of the host, or of another, is not theirs to read."""
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64)
    with pytest.raises(ValueError, match="on cpu"):
        gdn.gdn_stack_add_norm(gdn.NormShape(64), x, None, w, None, x)
    with pytest.raises(ValueError, match="on cpu"):
        gdn.gdn_stack_add_norm_bwd(gdn.NormShape(64), x, w, x, None, x, None, w, torch.zeros(1 << 16, dtype=torch.uint8))
    s, lg, i, f, ws = gdn.LogitsShape(64, top=2), x, torch.zeros(4, dtype=torch.int32), torch.zeros(4), torch.zeros(1 << 12, dtype=torch.uint8)
    ids, values = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for call in (lambda: gdn.gdn_stack_logprobs(s, lg, i, f, None, ids, values, None, ws),
                 lambda: gdn.gdn_stack_logprobs_bwd(s, lg, i, torch.zeros(4, 2), None, f, None, lg),
                 lambda: gdn.gdn_stack_distill(s, lg, ids, values, f, None, ws),
                 lambda: gdn.gdn_stack_distill_bwd(s, lg, ids, values, torch.zeros(4, 4), f, lg)):
        with pytest.raises(ValueError, match="on cpu"):
            call()


@pytest.mark.parametrize("how", [copy.deepcopy, lambda x: pickle.loads(pickle.dumps(x))])
def test_shapes_can_be_copied(how):
    for s in (gdn.NormShape(64, torch.bfloat16, torch.float32, 0, 1e-5, True), gdn.LogitsShape(100, torch.float32, 7, True)):
        assert how(s) == s and how(s)._ref._obj is not s._ref._obj
        assert bytes(how(s)._ref._obj) == bytes(s._ref._obj)
