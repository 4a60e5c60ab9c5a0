"""Checks of the attention layer's C ABI and binding that need no GPU: symbols,
workspace sizes and the refusal of bad arguments (no call here reaches a
kernel launch)."""

import ctypes
import os
import re

import pytest
import torch

import bitwise_invariant_gated_amd as gdn
from bitwise_invariant_gated_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation fails first
OK, INVALID, UNSUPPORTED, WORKSPACE = _lib.GDN_OK, _lib.GDN_ERR_INVALID_ARG, _lib.GDN_ERR_UNSUPPORTED, _lib.GDN_ERR_WORKSPACE


@pytest.fixture
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("library not built")
    return _lib.load()


def test_header_declares_exactly_the_bound_symbols():
    with open(os.path.join(ROOT, "include", "gdn_attn.h")) as f:
        text = f.read()
    assert set(re.findall(r"\b(gdn_attn_[a-z_]+)\s*\(", text)) == set(_lib.ATTN_EXPORTED)
    assert int(re.search(r"#define GDN_ATTN_BLOCK (\d+)", text).group(1)) == _lib.GDN_ATTN_BLOCK


def test_library_exports_every_declared_symbol(lib):
    for name in _lib.ATTN_EXPORTED:
        assert hasattr(lib, name), name


def shape(h=4, hk=2, d=128, dtype=_lib.GDN_DTYPE_BF16):
    return _lib.AttnShapeC(h, hk, d, dtype)


def pool(ptr=FAKE, slots=4, width=8, blocks=16):
    return _lib.AttnPoolC(ptr, ptr, ptr, ptr, ptr, slots, width, blocks)


def step(ptr=FAKE, slot=None, width=8, slots=4, **kw):
    s = _lib.AttnStepC(ptr, ptr, ptr, ptr, ptr, slot, width, slots)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def cache(ptr=FAKE, blocks=16, slots=4, **kw):
    c = _lib.AttnCacheC(ptr, ptr, ptr, ptr, ptr, ptr, blocks, slots)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def ref(x):
    return None if x is None else ctypes.byref(x)


def said(lib):
    return lib.gdn_cpr_last_error().decode()


BAD_SHAPES = [dict(h=0), dict(h=3, hk=2), dict(hk=-1), dict(hk=5), dict(d=96), dict(d=32), dict(dtype=7), dict(h=1 << 20, hk=1)]


@pytest.mark.parametrize("kw", BAD_SHAPES)
def test_shapes_refused_everywhere(lib, kw):
    s = shape(**kw)
    for op in range(3):
        assert lib.gdn_attn_workspace_size(ref(s), op, 100, 4, 16) == 0
    r = _lib.AttnRopeC(32, 0, 0, 10, 1e-6)
    assert lib.gdn_attn_qk_norm_rope(ref(s), ref(r), 4, FAKE, FAKE, 0, 0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0, 0, None) == UNSUPPORTED
    assert lib.gdn_attn_prefill(ref(s), 1, 4, 0, FAKE, FAKE, FAKE, 0, 0, 0, FAKE, ref(step()), ref(cache()), 1.0, FAKE, FAKE, 1 << 40, None) == UNSUPPORTED
    assert lib.gdn_attn_decode_step(ref(s), 4, FAKE, FAKE, FAKE, 0, 0, 0, ref(step()), ref(cache()), 1.0, FAKE, FAKE, 1 << 40, None) == UNSUPPORTED
    assert lib.gdn_attn_cache_read(ref(s), 1, 4, FAKE, ref(step()), ref(cache()), FAKE, FAKE, None) == UNSUPPORTED
    assert said(lib)


def test_workspace_sizes(lib):
    size = lib.gdn_attn_workspace_size
    s = shape(16, 4, 128)
    # the old tails of N sequences, K and V
    assert size(ref(s), _lib.GDN_ATTN_OP_PREFILL, 1000, 5, 100) >= 5 * 4 * 64 * 128 * 2 * 2
    # a record per head and partition of 512 keys, and one more per sequence
    assert size(ref(s), _lib.GDN_ATTN_OP_DECODE, 5, 5, 800) >= (100 + 5) * 16 * (128 + 8) * 4
    assert size(ref(s), _lib.GDN_ATTN_OP_NORM_ROPE_BWD, 1000, 0, 0) >= 2 * 128 * 4
    for op in range(3):
        assert size(ref(s), op, 1000, 5, 100) % 256 == 0
        assert size(ref(s), op, -1, 5, 100) == 0 and size(ref(s), op, 10, -5, 100) == 0 and size(ref(s), op, 10, 5, -1) == 0
    assert size(ref(s), 9, 1000, 5, 100) == 0 and size(None, 0, 1000, 5, 100) == 0


def test_plan_and_release_refusals(lib):
    def plan(p=pool(), n=2, t=10, cu=FAKE, s=step()):
        return lib.gdn_attn_plan(ref(p), n, t, cu, 1, ref(s), None)

    assert plan(p=None) == INVALID and "pool" in said(lib)
    assert plan(n=-1) == INVALID and plan(t=-1) == INVALID and plan(t=1 << 40) == UNSUPPORTED
    assert plan(cu=None) == INVALID and plan(cu=FAKE + 4) == INVALID and "aligned" in said(lib)
    assert plan(s=None) == INVALID
    for field in ("ctx_len", "positions", "slot_map", "status"):
        assert plan(s=step(**{field: None})) == INVALID and field in said(lib)
        assert plan(s=step(**{field: FAKE + 8})) == INVALID
    assert plan(s=step(slot=FAKE + 4)) == INVALID
    for field in ("block_table", "blocks_held", "free_blocks", "free_count", "seq_len"):
        p = pool()
        setattr(p, field, None)
        assert plan(p=p) == INVALID and field in said(lib)
        assert lib.gdn_attn_release(ref(p), 1, FAKE, None) == INVALID
    for kw in (dict(slots=0), dict(width=0), dict(blocks=0), dict(blocks=-3)):
        assert plan(p=pool(**kw)) == INVALID
    assert plan(n=0, t=3) == INVALID
    assert lib.gdn_attn_release(ref(pool()), -1, FAKE, None) == INVALID
    assert lib.gdn_attn_release(ref(pool()), 1, FAKE + 4, None) == INVALID
    assert lib.gdn_attn_release(ref(pool()), 0, None, None) == OK and said(lib) == ""


def test_norm_rope_refusals(lib):
    def fwd(s=None, r=None, t=4, q=FAKE, k=FAKE, qs=0, ks=0, wq=FAKE, wk=FAKE, cs=FAKE, pos=FAKE, qo=2 * FAKE, ko=3 * FAKE, qos=0, kos=0):
        s = s or shape()
        r = r or _lib.AttnRopeC(32, 0, 0, 10, 1e-6)
        return lib.gdn_attn_qk_norm_rope(ref(s), ref(r), t, q, k, qs, ks, wq, wk, cs, pos, qo, ko, qos, kos, None)

    for name in ("q", "k", "wq", "wk", "cs", "pos", "qo", "ko"):
        assert fwd(**{name: None}) == INVALID, name
        assert fwd(**{name: FAKE + 8}) == INVALID, name
    assert fwd(t=-1) == INVALID and fwd(t=1 << 31) == UNSUPPORTED and fwd(t=1 << 29) == UNSUPPORTED
    for rd in (-8, 4, 12, 136):
        assert fwd(r=_lib.AttnRopeC(rd, 0, 0, 10, 1e-6)) == UNSUPPORTED, rd
    assert fwd(r=_lib.AttnRopeC(32, 0, 0, 0, 1e-6)) == INVALID
    for eps in (-1e-6, float("nan"), float("inf")):
        assert fwd(r=_lib.AttnRopeC(32, 0, 0, 10, eps)) == INVALID
    for stride in (4 * 128 - 8, 4 * 128 + 4, -512):
        assert fwd(qs=stride) == INVALID and fwd(qos=stride) == INVALID and "stride" in said(lib)
    assert fwd(ks=128) == INVALID and fwd(kos=2 * 128 + 1) == INVALID
    assert fwd(q=2 * FAKE, qs=1024, qos=512) == INVALID and "in place" in said(lib)
    assert fwd(t=0, q=None, k=None, cs=None, pos=None, qo=None, ko=None) == OK

    def bwd(t=4, ws=FAKE, nbytes=1 << 30, dwq=FAKE, dq=FAKE, gq=FAKE, gqs=0, dqs=0):
        r = _lib.AttnRopeC(32, 0, 0, 10, 1e-6)
        return lib.gdn_attn_qk_norm_rope_bwd(ref(shape()), ref(r), t, FAKE, FAKE, 0, 0, FAKE, FAKE, FAKE, FAKE, gq, FAKE,
                                             gqs, 0, dq, FAKE, dqs, 0, dwq, FAKE, ws, nbytes, None)

    assert bwd(ws=None) == WORKSPACE and bwd(nbytes=16) == WORKSPACE and "workspace" in said(lib)
    assert bwd(ws=FAKE + 4) == INVALID and bwd(dwq=None) == INVALID and bwd(dq=None) == INVALID and bwd(gq=None) == INVALID
    assert bwd(gqs=1024) == INVALID and bwd(dqs=4) == INVALID


def test_attention_refusals(lib):
    big = 1 << 40

    def both(want, text=None, s=None, n=3, q=FAKE, k=FAKE, v=FAKE, qs=0, ks=0, vs=0, st=step(), c=cache(), scale=0.1, o=FAKE, ws=FAKE, nbytes=big):
        s = s or shape()
        got = [lib.gdn_attn_prefill(ref(s), n, n, 0, q, k, v, qs, ks, vs, FAKE, ref(st), ref(c), scale, o, ws, nbytes, None),
               lib.gdn_attn_decode_step(ref(s), n, q, k, v, qs, ks, vs, ref(st), ref(c), scale, o, ws, nbytes, None)]
        assert got == [want, want], got
        if text:
            assert text in said(lib)

    both(UNSUPPORTED, "bf16", s=shape(dtype=_lib.GDN_DTYPE_F32))
    both(INVALID, "negative", n=-1)
    for name in ("q", "k", "v", "o"):
        both(INVALID, name, **{name: None})
        both(INVALID, "aligned", **{name: FAKE + 2})
    both(INVALID, "step", st=None)
    both(INVALID, "cache", c=None)
    both(INVALID, "block_table", st=step(block_table=None))
    both(INVALID, "ctx_len", st=step(ctx_len=None))
    both(INVALID, st=step(slot=FAKE + 1))
    both(INVALID, st=step(width=0))
    both(INVALID, "rows", st=step(slots=5))
    for field in ("k8", "v8", "k_scale", "v_scale", "tail_k", "tail_v"):
        both(INVALID, field, c=cache(**{field: None}))
        both(INVALID, "aligned", c=cache(**{field: FAKE + 8}))
    both(INVALID, c=cache(blocks=0))
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        both(INVALID, "scale", scale=scale)
    both(INVALID, "stride", qs=4 * 128 + 4)
    both(INVALID, "stride", ks=128)
    both(INVALID, "stride", vs=-256)
    both(WORKSPACE, "workspace", ws=None)
    both(WORKSPACE, "workspace", nbytes=0)
    both(INVALID, "aligned", ws=FAKE + 8)
    assert lib.gdn_attn_prefill(ref(shape()), 0, 5, 0, FAKE, FAKE, FAKE, 0, 0, 0, FAKE, ref(step()), ref(cache()), 0.1, FAKE, FAKE, big, None) == INVALID
    assert lib.gdn_attn_prefill(ref(shape()), 1, 5, -1, FAKE, FAKE, FAKE, 0, 0, 0, FAKE, ref(step()), ref(cache()), 0.1, FAKE, FAKE, big, None) == INVALID
    assert lib.gdn_attn_prefill(ref(shape()), 1, 5, 0, FAKE, FAKE, FAKE, 0, 0, 0, None, ref(step()), ref(cache()), 0.1, FAKE, FAKE, big, None) == INVALID
    # nothing to do is no error
    assert lib.gdn_attn_prefill(ref(shape()), 2, 0, 0, None, None, None, 0, 0, 0, FAKE, ref(step()), ref(cache()), 0.1, None, None, 0, None) == OK
    assert lib.gdn_attn_decode_step(ref(shape()), 0, None, None, None, 0, 0, 0, ref(step()), ref(cache()), 0.1, None, None, 0, None) == OK
    assert said(lib) == ""


def test_cache_read_refusals(lib):
    def read(s=None, n=1, t=4, cu=FAKE, st=step(), c=cache(), k=FAKE, v=FAKE):
        return lib.gdn_attn_cache_read(ref(s or shape()), n, t, cu, ref(st), ref(c), k, v, None)

    assert read(s=shape(dtype=_lib.GDN_DTYPE_F32)) == UNSUPPORTED
    assert read(n=-1) == INVALID and read(cu=None) == INVALID and read(k=None) == INVALID and read(v=FAKE + 4) == INVALID
    assert read(st=None) == INVALID and read(c=None) == INVALID and read(n=0) == INVALID
    assert read(t=0, k=None, v=None) == OK


def test_binding_refuses_tensors_of_another_kind():
    s = gdn.AttnShape(4, 2, 64)
    with pytest.raises(ValueError):
        gdn.AttnShape(4, 2, 64, torch.float16)
    c = gdn.alloc_attn_cache(s, 4, 2, "cpu")
    with pytest.raises(ValueError):
        gdn.AttnCache(c.k8, c.v8[:2], c.k_scale, c.v_scale, c.tail_k, c.tail_v)
    with pytest.raises(ValueError):
        gdn.AttnCache(c.k8.float(), c.v8, c.k_scale, c.v_scale, c.tail_k, c.tail_v)
    p = gdn.alloc_attn_pool(2, 4, 4, "cpu")
    with pytest.raises(ValueError):
        gdn.AttnPool(p.block_table, p.blocks_held[:1], p.free_blocks, p.free_count, p.seq_len)
    with pytest.raises(ValueError):
        gdn.AttnPool(p.block_table.long(), p.blocks_held, p.free_blocks, p.free_count, p.seq_len)
    plan = gdn.alloc_attn_plan(p, 2, 2)
    with pytest.raises(ValueError):
        gdn.alloc_attn_plan(p, 2, 2, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        gdn.gdn_attn_plan(p, torch.zeros(2, dtype=torch.int32), plan)
    q, k = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    o, ws = torch.zeros_like(q), torch.zeros(256, dtype=torch.uint8)
    for bad in (dict(q=q.float()), dict(q=q[:, :3]), dict(k=k[:1]), dict(q=q.transpose(0, 1)), dict(k=k[:1].expand(2, 2, 64)),
                dict(o=o[:1]), dict(o=o.float()), dict(v=torch.zeros(2, 2, 128, dtype=torch.bfloat16)[..., ::2])):
        a = dict(q=q, k=k, v=k, o=o) | bad
        with pytest.raises(ValueError):
            gdn.gdn_attn_decode_step(s, a["q"], a["k"], a["v"], plan, c, a["o"], ws)
    with pytest.raises(ValueError):
        gdn.gdn_attn_decode_step(gdn.AttnShape(4, 4, 64), q, q, q, plan, c, o, ws)
    with pytest.raises(ValueError):
        gdn.gdn_attn_decode_step(s, q[:1], k[:1], k[:1], plan, c, o[:1], ws)
    with pytest.raises(ValueError):
        gdn.gdn_attn_prefill(s, q, k, k, torch.zeros(2, dtype=torch.int32), plan, c, o, ws)
    r, w, cs, pos = gdn.AttnRope(32), torch.ones(64), torch.zeros(10, 32), torch.zeros(2, dtype=torch.int32)
    for bad in (dict(w=w[:32]), dict(w=w.bfloat16()), dict(cs=cs[:, :16]), dict(cs=cs.double()), dict(pos=pos.long()),
                dict(pos=pos[:1]), dict(o=o[:1])):
        a = dict(w=w, cs=cs, pos=pos, o=o) | bad
        with pytest.raises(ValueError):
            gdn.gdn_attn_qk_norm_rope(s, r, q, k, a["w"], w, a["cs"], a["pos"], a["o"], torch.zeros_like(k))
