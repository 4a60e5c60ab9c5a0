"""Helpers of the tests of gdn_stack.h: calls that allocate their outputs, filled with what must not
be left, and the bounds that the arithmetic gives."""

from __future__ import annotations

import numpy as np
import torch

import bitwise_invariant_gated_amd as gdn

DEV = "cuda"
F8 = torch.float8_e4m3fn


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def dev(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV).to(dtype)


def half(dtype):
    """The rounding of a result to its type, of its magnitude."""
    return torch.finfo(dtype).eps / 2


def new(*shape, dtype=torch.float32):
    if dtype in (torch.int32, torch.uint8):
        return torch.full(shape, 99, dtype=dtype, device=DEV)
    return torch.full(shape, float("nan"), dtype=dtype, device=DEV)


def add_norm(s, x, residual, w, y=True, h=True):
    """(h, y, y8, y_scale)."""
    t = x.shape[0]
    h = new(t, s.width, dtype=s.residual_dtype) if h else None
    y = new(t, s.width, dtype=s.dtype) if y else None
    y8 = sc = None
    if s.group >= 0:
        y8, sc = new(t, s.width, dtype=torch.uint8), new(t, s.width // s.group if s.group else 1)
    gdn.gdn_stack_add_norm(s, x, residual, w, h, y, y8, sc)
    return h, y, y8, sc


def add_norm_bwd(s, h, w, dy, d_res, both=False):
    """(dx, d_residual, dw)."""
    t = h.shape[0]
    dx, dd, dw = new(t, s.width, dtype=s.dtype), new(t, s.width, dtype=s.residual_dtype) if both else None, new(s.width)
    gdn.gdn_stack_add_norm_bwd(s, h, w, dy, d_res, dx, dd, dw, gdn.alloc_norm_workspace(s, t, DEV))
    return dx, dd, dw


class Out:
    pass


def logprobs(s, logits, targets=None, scale=None, entropy=True, stats=True):
    t, o = logits.shape[0], Out()
    o.logprobs = None if targets is None else new(t)
    o.entropy = new(t) if entropy else None
    o.stats = new(t, 2) if stats else None
    o.top_ids, o.top_logprobs = (new(t, s.top, dtype=torch.int32), new(t, s.top)) if s.top else (None, None)
    ws = gdn.alloc_logits_workspace(s, t, DEV).fill_(0xff)  # NaN: nothing of it may be read before it is written
    gdn.gdn_stack_logprobs(s, logits, targets, o.logprobs, o.entropy, o.top_ids, o.top_logprobs, o.stats, ws, scale=scale)
    return o


def logprobs_bwd(s, logits, targets, o, g, f, scale=None, out=None):
    out = new(*logits.shape, dtype=s.dtype) if out is None else out
    gdn.gdn_stack_logprobs_bwd(s, logits, targets, o.stats, o.entropy, g, f, out, scale=scale)
    return out


def distill(s, logits, ids, values, scale=None):
    """(loss, stats)."""
    t = logits.shape[0]
    loss, stats = new(t), new(t, 4)
    gdn.gdn_stack_distill(s, logits, ids, values, loss, stats, gdn.alloc_logits_workspace(s, t, DEV).fill_(0xff), scale=scale)
    return loss, stats


def distill_bwd(s, logits, ids, values, stats, g, scale=None, out=None):
    out = new(*logits.shape, dtype=s.dtype) if out is None else out
    gdn.gdn_stack_distill_bwd(s, logits, ids, values, stats, g, out, scale=scale)
    return out


def same_bits(a, b):
    if a is None or b is None:
        return a is b
    view = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.contiguous().view(view), b.contiguous().view(view))


# Logits.  In units of u = 2^-24, with z = scale (s - m) <= 0: the distance, its product with
# scale * log2(e) and that constant's own rounding put 5 u |z| on an exponent, and the exponential
# itself 2 u; a part's exponents and its record's factor add up to the same |z| once more, 10 u |z|
# in all.  A sum over a row (32 terms to a lane, 8 lane steps, 8 records, 8 lane steps) has 60 u of
# itself, and its logarithm 2 u and 2 u of its own size.  So log q is off by
#   16 u |z| + 64 u + 16 u E|z| + 2 u |L| + u |log q|, E over the row's distribution.
U = 2.0 ** -24


def log_q_bound(z, logq):
    """Of one row, per column (0 where masked)."""
    p = np.exp(logq)
    some = p > 0
    az = np.where(logq > -np.inf, np.abs(z), 0)
    log_l = abs(-logq.max()) if some.any() else 0
    return U * (16 * az + 64 + 16 * np.sum(p[some] * az[some]) + 4 * log_l + 2 * np.where(logq > -np.inf, np.abs(logq), 0))


def entropy_bound(z, logq):
    """H = L - E z: the same errors, of every term's weight and of its distance."""
    p = np.exp(logq)
    some = p > 0
    if not some.any():
        return 0.0
    az = np.abs(z[some])
    e1, e2 = np.sum(p[some] * az), np.sum(p[some] * az * az)
    return U * (64 + 16 * e1 + 16 * e2 + 80 * e1 + 16 * e1 * e1 + 4 * abs(logq.max()))


# Norm.  A row's sum of squares has at most 64 + 8 additions one after the other, all positive:
# 72 u, halved by the root; mean, eps, root, quotient and the two products 7 u more.
NORM = 2.0 ** -18
