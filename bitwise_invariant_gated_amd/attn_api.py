"""Python binding of the attention layer's C ABI (include/gdn_attn.h).

Argument marshalling only, as in api.py.  q, k, v and the tensors of the norm
and rotation may be views whose tokens are a stride apart (a projection's
rows); their heads and dims are contiguous.
"""

from __future__ import annotations

import ctypes
import dataclasses
from typing import Optional

import torch

from . import _lib
from .api import _DTYPES, _ptr

BLOCK = _lib.GDN_ATTN_BLOCK


@dataclasses.dataclass(frozen=True)
class AttnShape:
    num_heads: int
    num_kv_heads: int
    head_dim: int
    dtype: torch.dtype = torch.bfloat16

    def __post_init__(self):
        if self.dtype not in _DTYPES:
            raise ValueError(f"unsupported dtype {self.dtype}")
        object.__setattr__(self, "kv_heads", self.num_kv_heads or self.num_heads)
        object.__setattr__(self, "_ref", ctypes.byref(_lib.AttnShapeC(self.num_heads, self.num_kv_heads, self.head_dim,
                                                                      _DTYPES[self.dtype])))

    def __reduce__(self):
        return AttnShape, (self.num_heads, self.num_kv_heads, self.head_dim, self.dtype)


@dataclasses.dataclass(frozen=True)
class AttnRope:
    rotary_dim: int
    interleaved: bool = False
    eps: float = 1e-6
    zero_centered: bool = False


@dataclasses.dataclass(frozen=True)
class AttnPool:
    """Device arrays of a gdn_attn_pool (layouts in gdn_attn.h)."""

    block_table: torch.Tensor
    blocks_held: torch.Tensor
    free_blocks: torch.Tensor
    free_count: torch.Tensor
    seq_len: torch.Tensor

    def __post_init__(self):
        t = (self.block_table, self.blocks_held, self.free_blocks, self.free_count, self.seq_len)
        _check_types(t, torch.int32)
        slots, width = self.block_table.shape
        if self.blocks_held.numel() != slots or self.seq_len.numel() != slots or self.free_count.numel() != 1:
            raise ValueError("pool arrays do not match the block table")
        object.__setattr__(self, "_ref", ctypes.byref(_lib.AttnPoolC(*map(_ptr, t), slots, width, self.free_blocks.numel())))

    def __reduce__(self):
        return AttnPool, _fields(self)


def alloc_attn_pool(num_slots: int, max_blocks: int, num_blocks: int, device="cuda") -> AttnPool:
    """An empty pool: every block free, the lowest id to be given out first."""
    i32 = dict(dtype=torch.int32, device=device)
    return AttnPool(torch.full((num_slots, max_blocks), -1, **i32), torch.zeros(num_slots, **i32),
                    torch.arange(num_blocks - 1, -1, -1, **i32), torch.full((1,), num_blocks, **i32),
                    torch.zeros(num_slots, **i32))


@dataclasses.dataclass(frozen=True)
class AttnPlan:
    """Device arrays of a gdn_attn_step: what a step's plan gives every layer."""

    ctx_len: torch.Tensor
    positions: torch.Tensor
    slot_map: torch.Tensor
    status: torch.Tensor
    block_table: torch.Tensor
    slot_index: Optional[torch.Tensor] = None

    def __post_init__(self):
        _check_types((self.ctx_len, self.positions, self.status, self.block_table), torch.int32)
        _check_types((self.slot_map,), torch.int64)
        if self.slot_index is not None:
            _check_types((self.slot_index,), torch.int32)
            if self.slot_index.numel() != self.ctx_len.numel():
                raise ValueError("slot_index and ctx_len differ in length")
        slots, width = self.block_table.shape
        object.__setattr__(self, "_ref", ctypes.byref(_lib.AttnStepC(
            _ptr(self.ctx_len), _ptr(self.positions), _ptr(self.slot_map), _ptr(self.status), _ptr(self.block_table),
            _ptr(self.slot_index), width, slots)))

    def __reduce__(self):
        return AttnPlan, _fields(self)


def alloc_attn_plan(pool: AttnPool, num_seqs: int, total_tokens: int,
                    slot_index: Optional[torch.Tensor] = None) -> AttnPlan:
    dev = pool.block_table.device
    i32 = dict(dtype=torch.int32, device=dev)
    return AttnPlan(torch.empty(num_seqs, **i32), torch.empty(total_tokens, **i32),
                    torch.empty(total_tokens, dtype=torch.int64, device=dev), torch.empty(1, **i32), pool.block_table,
                    slot_index)


@dataclasses.dataclass(frozen=True)
class AttnCache:
    """Device arrays of one layer's gdn_attn_cache (layouts in gdn_attn.h)."""

    k8: torch.Tensor
    v8: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor
    tail_k: torch.Tensor
    tail_v: torch.Tensor

    def __post_init__(self):
        blocks, hk = self.k_scale.shape
        slots, _, _, d = self.tail_k.shape
        want = dict(k8=(blocks, hk, d // BLOCK, BLOCK, BLOCK), v8=(blocks, hk, d, BLOCK), v_scale=(blocks, hk),
                    tail_k=(slots, hk, BLOCK, d), tail_v=(slots, hk, d, BLOCK))
        for name, shape in want.items():
            if tuple(getattr(self, name).shape) != shape:
                raise ValueError(f"{name} has shape {tuple(getattr(self, name).shape)}, {shape} expected")
        _check_types((self.k8, self.v8), torch.uint8)
        _check_types((self.k_scale, self.v_scale), torch.float32)
        _check_types((self.tail_k, self.tail_v), torch.bfloat16)
        object.__setattr__(self, "_ref", ctypes.byref(_lib.AttnCacheC(
            _ptr(self.k8), _ptr(self.v8), _ptr(self.k_scale), _ptr(self.v_scale), _ptr(self.tail_k),
            _ptr(self.tail_v), blocks, slots)))

    def __reduce__(self):
        return AttnCache, _fields(self)

    def check(self, shape: AttnShape) -> None:
        if self.tail_k.shape[1] != shape.kv_heads or self.tail_k.shape[3] != shape.head_dim:
            raise ValueError("the cache is of another shape")


def alloc_attn_cache(shape: AttnShape, num_blocks: int, num_slots: int, device="cuda") -> AttnCache:
    hk, d = shape.kv_heads, shape.head_dim
    u8 = dict(dtype=torch.uint8, device=device)
    f32 = dict(dtype=torch.float32, device=device)
    dt = dict(dtype=shape.dtype, device=device)
    return AttnCache(torch.zeros((num_blocks, hk, d // BLOCK, BLOCK, BLOCK), **u8),
                     torch.zeros((num_blocks, hk, d, BLOCK), **u8), torch.zeros((num_blocks, hk), **f32),
                     torch.zeros((num_blocks, hk), **f32), torch.zeros((num_slots, hk, BLOCK, d), **dt),
                     torch.zeros((num_slots, hk, d, BLOCK), **dt))


def gdn_attn_workspace_size(shape: AttnShape, op: int, total_tokens: int, num_seqs: int = 0,
                            num_blocks: int = 0) -> int:
    return int(_lib.load().gdn_attn_workspace_size(shape._ref, op, total_tokens, num_seqs, num_blocks))


def alloc_attn_workspace(shape: AttnShape, op: int, total_tokens: int, num_seqs: int = 0, num_blocks: int = 0,
                         device="cuda") -> torch.Tensor:
    n = gdn_attn_workspace_size(shape, op, total_tokens, num_seqs, num_blocks)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def _stream(stream) -> int:
    """The stream's handle, or that of the current one, without making a torch.cuda.Stream
    of it (2.5 us, where a call of one token takes 7 in all)."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _fields(x) -> tuple:
    """What a copy is made from: the arrays; the C handle (_ref) is made anew over the copy's."""
    return tuple(getattr(x, f.name) for f in dataclasses.fields(x))


def _check_types(tensors, dtype) -> None:
    for t in tensors:
        if t.dtype != dtype:
            raise ValueError(f"{dtype} tensor expected, {t.dtype} given")


def _rows(t: torch.Tensor, heads: int, d: int, dtype, name: str):
    """(tokens, pointer, token stride) of a [T, heads, d] tensor whose heads and dims are contiguous."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != d or t.dtype is not dtype:
        raise ValueError(f"{name}: [T, {heads}, {d}] of {dtype} expected, {tuple(shape)} of {t.dtype} given")
    n = shape[0]
    s0, s1, s2 = t.stride()
    if n and (s2 != 1 or (heads > 1 and s1 != d)):
        raise ValueError(f"{name}: heads and dims must be contiguous")
    if n <= 1:
        s0 = 0  # a single token's stride is not used
    elif s0 < heads * d:
        raise ValueError(f"{name}: tokens overlap")
    return n, t.data_ptr(), s0


def gdn_attn_plan(pool: AttnPool, cu_seqlens, plan: AttnPlan, advance: bool = True, stream=None) -> None:
    """Block tables, positions and slot maps of a step's new tokens (gdn_attn_plan)."""
    n = plan.ctx_len.numel()
    if cu_seqlens.numel() != n + 1 or cu_seqlens.dtype != torch.int32:
        raise ValueError(f"cu_seqlens: int32 of {n + 1} expected")
    _lib.check(_lib.load().gdn_attn_plan(pool._ref, n, plan.positions.numel(), _ptr(cu_seqlens),
                                         int(advance), plan._ref, _stream(stream)))


def gdn_attn_release(pool: AttnPool, slot_index, stream=None) -> None:
    """The blocks of the given cache rows go back to the pool."""
    _check_types((slot_index,), torch.int32)
    _lib.check(_lib.load().gdn_attn_release(pool._ref, slot_index.numel(), _ptr(slot_index),
                                            _stream(stream)))


def _rope_c(rope: AttnRope, cos_sin, positions, tokens: int):
    n_pos = 0
    if rope.rotary_dim:
        if cos_sin.dtype is not torch.float32 or cos_sin.dim() != 2 or cos_sin.shape[1] != rope.rotary_dim:
            raise ValueError(f"cos_sin: float32 [positions, {rope.rotary_dim}] expected")
        if positions.dtype is not torch.int32 or positions.numel() < tokens:
            raise ValueError("positions: int32 of every token expected")
        n_pos = cos_sin.shape[0]
    return ctypes.byref(_lib.AttnRopeC(rope.rotary_dim, rope.interleaved, rope.zero_centered, n_pos, rope.eps))


def _weight(w, d: int, name: str):
    if w.dtype is not torch.float32 or w.numel() != d:
        raise ValueError(f"{name}: float32 of {d} expected")
    return _ptr(w)


def gdn_attn_qk_norm_rope(shape: AttnShape, rope: AttnRope, q, k, w_q, w_k, cos_sin, positions, q_out, k_out,
                          stream=None) -> None:
    """RMS norm of every head of q and k and the rotation; q_out, k_out may be q, k."""
    h, hk, d, dt = shape.num_heads, shape.kv_heads, shape.head_dim, shape.dtype
    t, qp, qs = qrows = _rows(q, h, d, dt, "q")
    tk, kp, ks = krows = _rows(k, hk, d, dt, "k")
    tqo, qo, qos = qrows if q_out is q else _rows(q_out, h, d, dt, "q_out")
    tko, ko, kos = krows if k_out is k else _rows(k_out, hk, d, dt, "k_out")
    if not t == tk == tqo == tko:
        raise ValueError("q, k and their outputs differ in tokens")
    _lib.check(_lib.load().gdn_attn_qk_norm_rope(
        shape._ref, _rope_c(rope, cos_sin, positions, t), t, qp, kp, qs, ks, _weight(w_q, d, "w_q"),
        _weight(w_k, d, "w_k"), _ptr(cos_sin), _ptr(positions), qo, ko, qos, kos, _stream(stream)))


def gdn_attn_qk_norm_rope_bwd(shape: AttnShape, rope: AttnRope, q, k, w_q, w_k, cos_sin, positions, d_q_out, d_k_out,
                              dq, dk, dw_q, dw_k, workspace, stream=None) -> None:
    """Gradients of gdn_attn_qk_norm_rope: dq, dk in the input type, dw_q, dw_k in fp32."""
    h, hk, d, dt = shape.num_heads, shape.kv_heads, shape.head_dim, shape.dtype
    t, qp, qs = _rows(q, h, d, dt, "q")
    tk, kp, ks = _rows(k, hk, d, dt, "k")
    tgq, gq, gqs = _rows(d_q_out, h, d, dt, "d_q_out")
    tgk, gk, gks = _rows(d_k_out, hk, d, dt, "d_k_out")
    toq, oq, oqs = _rows(dq, h, d, dt, "dq")
    tok, ok, oks = _rows(dk, hk, d, dt, "dk")
    if not t == tk == tgq == tgk == toq == tok:
        raise ValueError("q, k and their gradients differ in tokens")
    _lib.check(_lib.load().gdn_attn_qk_norm_rope_bwd(
        shape._ref, _rope_c(rope, cos_sin, positions, t), t, qp, kp, qs, ks, _weight(w_q, d, "w_q"), _weight(w_k, d, "w_k"),
        _ptr(cos_sin), _ptr(positions), gq, gk, gqs, gks, oq, ok, oqs, oks, _weight(dw_q, d, "dw_q"),
        _weight(dw_k, d, "dw_k"), _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def _attention_args(shape: AttnShape, q, k, v, cache: AttnCache, o, scale):
    h, hk, d, dt = shape.num_heads, shape.kv_heads, shape.head_dim, shape.dtype
    cache.check(shape)
    t, qp, qs = _rows(q, h, d, dt, "q")
    tk, kp, ks = _rows(k, hk, d, dt, "k")
    tv, vp, vs = _rows(v, hk, d, dt, "v")
    if tk != t or tv != t or tuple(o.shape) != (t, h, d) or o.dtype != dt:
        raise ValueError("q, k, v and o differ in tokens, shape or type")
    return (qp, kp, vp, qs, ks, vs), d ** -0.5 if scale is None else scale


def gdn_attn_prefill(shape: AttnShape, q, k, v, cu_seqlens, plan: AttnPlan, cache: AttnCache, o, workspace,
                     scale: Optional[float] = None, max_new: int = 0, stream=None) -> None:
    """Attention of every sequence's new tokens over its cache and themselves; appends
    them.  scale: None for 1 / sqrt(head_dim); max_new: an upper bound of any
    sequence's new tokens, if known."""
    args, scale = _attention_args(shape, q, k, v, cache, o, scale)
    n = cu_seqlens.numel() - 1
    if cu_seqlens.dtype != torch.int32 or plan.ctx_len.numel() != n:
        raise ValueError("cu_seqlens: int32 of one more than the plan's sequences expected")
    _lib.check(_lib.load().gdn_attn_prefill(
        shape._ref, n, q.shape[0], max_new, *args, _ptr(cu_seqlens), plan._ref,
        cache._ref, scale, _ptr(o), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))


def gdn_attn_decode_step(shape: AttnShape, q, k, v, plan: AttnPlan, cache: AttnCache, o, workspace,
                         scale: Optional[float] = None, stream=None) -> None:
    """gdn_attn_prefill for one new token of every sequence."""
    args, scale = _attention_args(shape, q, k, v, cache, o, scale)
    n = q.shape[0]
    if plan.ctx_len.numel() != n:
        raise ValueError("one token for each of the plan's sequences expected")
    _lib.check(_lib.load().gdn_attn_decode_step(
        shape._ref, n, *args, plan._ref, cache._ref, scale, _ptr(o),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def gdn_attn_cache_read(shape: AttnShape, cu_seqlens, total_tokens: int, plan: AttnPlan, cache: AttnCache, k_out=None,
                        v_out=None, stream=None):
    """The cached keys and values, [T, Hk, d] each, of the plan's rows; row i holds
    cu_seqlens[i + 1] - cu_seqlens[i] tokens."""
    cache.check(shape)
    want = (total_tokens, shape.kv_heads, shape.head_dim)
    if k_out is None:
        k_out = torch.empty(want, dtype=shape.dtype, device=cache.k8.device)
    if v_out is None:
        v_out = torch.empty(want, dtype=shape.dtype, device=cache.k8.device)
    for t in (k_out, v_out):
        if tuple(t.shape) != want or t.dtype != shape.dtype:
            raise ValueError(f"outputs: {want} of {shape.dtype} expected")
    if cu_seqlens.dtype != torch.int32:
        raise ValueError("cu_seqlens: int32 expected")
    _lib.check(_lib.load().gdn_attn_cache_read(
        shape._ref, cu_seqlens.numel() - 1, total_tokens, _ptr(cu_seqlens), plan._ref,
        cache._ref, _ptr(k_out), _ptr(v_out), _stream(stream)))
    return k_out, v_out
