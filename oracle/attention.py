"""fp64 NumPy oracle of the attention layer (include/gdn_attn.h): the cache's
rule, causal attention by it, the per-head norm with the rotation and its
gradient, and the block plan.  Plain loops, no code shared with the HIP path."""

from __future__ import annotations

import numpy as np

BLOCK = 64
TOP = 240 * 2.0 ** 120  # the largest cached magnitude


def e4m3_values() -> np.ndarray:
    """What the codes 0 .. 126 stand for (127 is NaN; bit 7 is the sign)."""
    codes = np.arange(127)
    e, f = codes >> 3, codes & 7
    return np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e.astype(np.float64) - 10))


def to_e4m3(x: np.ndarray) -> np.ndarray:
    """Values rounded to the nearest e4m3 value, ties to the even code; what is
    not finite to NaN.  |x| <= 448."""
    v = e4m3_values()
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    assert a.max(initial=0.0) <= 448.0
    hi = np.clip(np.searchsorted(v, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = v[hi] - a, a - v[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return np.where(np.isfinite(x), np.copysign(v[code], x), np.nan)


def block_scale(x: np.ndarray) -> float:
    """2^e, the least e >= -100 with the largest finite magnitude <= 448 2^e."""
    fin = np.abs(x[np.isfinite(x)])
    most, e = float(fin.max(initial=0.0)), -100
    while most > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def cached(x: np.ndarray) -> np.ndarray:
    """[L, Hk, d] as the cache holds it: full blocks in 8 bits, the rest as it is."""
    out = np.array(x, dtype=np.float64)
    for b in range(x.shape[0] // BLOCK):
        for h in range(x.shape[1]):
            blk = out[b * BLOCK:(b + 1) * BLOCK, h]
            s = block_scale(blk)
            # 256 * 2^120 is no bf16 number
            most = np.where(np.isfinite(blk), TOP, np.inf)
            out[b * BLOCK:(b + 1) * BLOCK, h] = to_e4m3(np.clip(blk, -most, most) / s) * s
    return out


def attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, first: int = 0) -> np.ndarray:
    """One sequence from position 0: k, v [L, Hk, d], q [L - first, H, d] of the
    positions first .. L - 1 -> o of those positions."""
    L, hk, d = k.shape
    H = q.shape[1]
    grp = H // hk
    kc, vc = cached(k), cached(v)
    o = np.zeros(q.shape)
    for p in range(first, L):
        lo = p // BLOCK * BLOCK
        for j in range(hk):
            kk = np.concatenate([kc[:lo, j], k[lo:p + 1, j]])
            vv = np.concatenate([vc[:lo, j], v[lo:p + 1, j]])
            s = q[p - first, j * grp:(j + 1) * grp] @ kk.T * scale
            w = np.exp(s - s.max(-1, keepdims=True))
            o[p - first, j * grp:(j + 1) * grp] = (w / w.sum(-1, keepdims=True)) @ vv
    return o


def rotate(x: np.ndarray, cos: np.ndarray, sin: np.ndarray, interleaved: bool) -> np.ndarray:
    """x [T, H, d], cos, sin [T, rd / 2]."""
    y = x.copy()
    half = cos.shape[1]
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = cos[:, i, None], sin[:, i, None]
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


def norm_rope(x, w, cos, sin, eps, interleaved):
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return rotate(x * r * w, cos, sin, interleaved)


def norm_rope_backward(x, w, cos, sin, eps, interleaved, dy):
    """(dx, dw, sum of |terms| of dw, largest r (|h| + |x m|))."""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dn = rotate(dy, cos, -sin, interleaved)
    h = dn * w
    m = r * r * (h * x).mean(-1, keepdims=True)
    dx = r * (h - x * m)
    size = (r * (np.abs(h) + np.abs(x * m))).max(initial=0.0)
    return dx, (dn * x * r).sum((0, 1)), np.abs(dn * x * r).sum((0, 1)), size


class Pool:
    """The block pool, request by request."""

    def __init__(self, slots: int, width: int, blocks: int):
        self.table = np.full((slots, width), -1, np.int64)
        self.held = [0] * slots
        self.free = list(range(blocks - 1, -1, -1))
        self.len = [0] * slots

    def plan(self, rows, news, advance=True):
        """(ctx_len, positions, slot_map, refused)."""
        there, asked = len(self.free), 0
        ctx, pos, place, refused = [], [], [], 0
        for r, m in zip(rows, news):
            if r < 0:
                ctx.append(-1)
                pos += range(m)
                place += [-1] * m
                continue
            want = -(-(self.len[r] + m) // BLOCK)
            need = max(0, want - self.held[r])
            asked += need
            ok = need == 0 or (asked <= there and want <= self.table.shape[1])
            for _ in range(need if ok else 0):
                self.table[r, self.held[r]] = self.free.pop()
                self.held[r] += 1
            ctx.append(self.len[r] if ok else -1)
            refused += not ok
            for p in range(self.len[r], self.len[r] + m):
                pos.append(p)
                place.append(self.table[r, p // BLOCK] * BLOCK + p % BLOCK if ok else -1)
            if ok and advance:
                self.len[r] += m
        return ctx, pos, place, refused

    def release(self, rows):
        for r in reversed(rows):
            if r < 0:
                continue
            for j in reversed(range(self.held[r])):
                self.free.append(int(self.table[r, j]))
                self.table[r, j] = -1
            self.held[r] = self.len[r] = 0
