"""The attention layer's operators, case by case: what each is called with, its plain form in
elementary torch operations, and its value in 64 bits.

The operators are the softmax-attention layer that hybrid models place between Gated DeltaNet
layers: block tables and slot maps from request lengths ("plan"), the per-head norm of q and k with
the position rotation and its gradient ("norm_rope", "norm_rope_bwd"), and attention over a paged
cache held in 8 bits ("decode": one token per sequence, "prefill": any number of new tokens after
any context).

The cache's rule, which every form below follows: blocks of 64 tokens; a block is held as e4m3 with
one power-of-two scale per block and key/value head, 2^e with the least e >= -100 for which the
block's largest finite magnitude is at most 448 * 2^e; a query reads its own block (up to itself) in
the input type and every earlier block in 8 bits.  Layouts: k8 [blocks, Hk, d / 64, 64 tokens, 64 dims],
v8 [blocks, Hk, d, 64 tokens], tail_k [slots, Hk, 64, d], tail_v [slots, Hk, d, 64]; the tail of a
sequence holds the tokens of the block that its last token is in.
"""

import itertools
import random

import torch

own = False
DEV = "cuda"
BLOCK = 64


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # a serving step's plan: every request of a batch of 256 decodes one token
        dict(name="plan_step_256", op="plan", n=256, new=1, ctx=4096, mix=1, release=False),
        # a wave of 128 ragged prompts is admitted (about 98,000 tokens) and later leaves
        dict(name="plan_wave_128", op="plan", n=128, new=1024, ctx=0, mix=2, release=True),
        # the norm and rotation of one decoded token: latency alone; a quarter of each head is rotated
        dict(name="norm_rope_1_token", op="norm_rope", t=1, h=16, hk=2, d=256, rd=64, inter=False, f32=False, fused=True),
        # a training-sized pass over 10,240 tokens, q and k read out of a fused projection's rows
        dict(name="norm_rope_10240", op="norm_rope", t=10240, h=16, hk=16, d=128, rd=128, inter=False, f32=False, fused=True),
        # its gradient
        dict(name="norm_rope_bwd_10240", op="norm_rope_bwd", t=10240, h=16, hk=16, d=128, rd=128, inter=False, f32=False, fused=True),
        # odd length, grouped heads, adjacent pairs rotated in half of each head, all in 32 bits
        dict(name="norm_rope_bwd_2047_f32", op="norm_rope_bwd", t=2047, h=12, hk=4, d=64, rd=32, inter=True, f32=True, fused=False),
        # one chat session's next token
        dict(name="decode_1x2000_d256", op="decode", n=1, ctx=2000, mix=0, h=16, hk=2, d=256),
        # a full serving batch of ragged contexts
        dict(name="decode_256x4096", op="decode", n=256, ctx=4096, mix=3, h=16, hk=4, d=128),
        # a few long documents
        dict(name="decode_3x100003", op="decode", n=3, ctx=100003, mix=0, h=32, hk=4, d=128),
        # a batch of fresh prompts, a key/value head for every query head
        dict(name="prefill_5x2048", op="prefill", n=5, new=2048, ctx=0, mix=0, h=16, hk=16, d=128),
        # one long fresh prompt, wide heads shared by eight
        dict(name="prefill_1x10240_d256", op="prefill", n=1, new=10240, ctx=0, mix=0, h=16, hk=2, d=256),
        # short further turns after long contexts
        dict(name="continue_16x37_d64", op="prefill", n=16, new=37, ctx=8000, mix=4, h=32, hk=8, d=64),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["plan", "norm_rope", "norm_rope_bwd", "decode", "decode", "prefill", "prefill"])
    if op == "plan":
        if rng.random() < 0.5:
            return dict(op=op, n=_log(rng, 1, 1024), new=_log(rng, 1, 8), ctx=_log(rng, 1, 16384), mix=rng.randrange(1, 1000), release=False)
        n = _log(rng, 1, 512)
        return dict(op=op, n=n, new=_log(rng, 1, min(16384, 130000 // n)), ctx=0, mix=rng.randrange(1, 1000), release=True)
    hk = rng.choice([1, 2, 3, 4, 8, 16])
    h = hk * rng.choice([g for g in (1, 2, 3, 4, 5, 8, 16) if g * hk <= 32])
    d = rng.choice([64, 128, 256])
    if op.startswith("norm_rope"):
        f32 = rng.random() < 0.3
        most = 10240 * 32 * 128 // ((h + hk) * d) // (2 if f32 else 1)
        rd = rng.choice([r for r in (16, 32, 64, 128, 256) if r <= d])
        return dict(op=op, t=_log(rng, 1, most), h=h, hk=hk, d=d, rd=rd, inter=rng.random() < 0.3, f32=f32, fused=rng.random() < 0.5)
    if op == "decode":
        n = _log(rng, 1, 256)
        most = min(131072, 256 * 4096 * 4 * 128 // (n * hk * d))
        return dict(op=op, n=n, ctx=_log(rng, 1, most), mix=rng.randrange(0, 1000), h=h, hk=hk, d=d)
    n = _log(rng, 1, 32)
    new = _log(rng, 2, max(2, min(10240 // n, int(10240 * (16 / (n * h)) ** 0.5))))
    room = min(16384, 16 * 10240 * 10240 // (n * h * new) - new, 131072 * 16 // (n * hk))
    ctx = _log(rng, 1, room) if room > 1 and rng.random() < 0.7 else 0
    return dict(op=op, n=n, new=new, ctx=ctx, mix=rng.randrange(0, 1000), h=h, hk=hk, d=d)


def _lengths(case):
    """(tokens in the cache, new tokens) of every sequence.  mix = 0: all alike; otherwise ragged, with some of one token and
    contexts that end on and beside a block's end."""
    n, ctx, new, mix = case["n"], case["ctx"], case.get("new", 1), case["mix"]
    if not mix:
        return [ctx] * n, [new] * n
    r = random.Random(mix)
    lens = [new if new <= 1 or i == 0 else max(1, int(new * r.uniform(0.5, 1.0))) if r.random() < 0.9 else 1 for i in range(n)]
    ctxs = [ctx if i == 0 else max(0, int(ctx * r.uniform(0.5, 1.0))) for i in range(n)]
    for i in range(1, n):
        if ctxs[i] > BLOCK and r.random() < 0.1:
            ctxs[i] = ctxs[i] // BLOCK * BLOCK - r.choice([0, 1])
    return ctxs, lens


def work(case):
    op = case["op"]
    if op == "plan":
        ctxs, lens = _lengths(case)
        new_blocks = sum(-(-(c + m) // BLOCK) - -(-c // BLOCK) for c, m in zip(ctxs, lens))
        b = sum(lens) * (4 + 8) + case["n"] * 24 + new_blocks * 8 * (3 if case["release"] else 1)
        return {"bytes": b, "flops": 0}
    if op.startswith("norm_rope"):
        t, d, size = case["t"], case["d"], 4 if case["f32"] else 2
        rows = t * (case["h"] + case["hk"])
        passes = 2 if op == "norm_rope" else 3
        return {"bytes": rows * d * size * passes + t * (case["rd"] * 4 + 4) + 8 * d * (passes - 1), "flops": rows * d * (8 if passes == 2 else 20)}
    ctxs, lens = _lengths(case)
    h, hk, d = case["h"], case["hk"], case["d"]
    tokens = sum(lens)
    cached = sum(c // BLOCK * BLOCK for c in ctxs)
    tails = sum(c % BLOCK for c in ctxs)
    filled = sum((c + m) // BLOCK - c // BLOCK for c, m in zip(ctxs, lens))
    b = cached * hk * 2 * d + tails * hk * 2 * d * 2 + tokens * (h * d * 4 + hk * d * 4) + filled * hk * (2 * BLOCK * d + 8)
    b += sum(min(m, (c + m - 1) % BLOCK + 1) for c, m in zip(ctxs, lens)) * hk * 2 * d * 2
    pairs = sum(m * c + m * (m + 1) // 2 for c, m in zip(ctxs, lens))
    return {"bytes": b, "flops": 4 * h * d * pairs}


# ---------------------------------------------------------------------------
# inputs

def _int(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


def _tables(case, g):
    """Block tables of the cached blocks (none for the new ones), the free stack and shuffled cache rows."""
    ctxs, lens = _lengths(case)
    n = case["n"]
    held = [-(-c // BLOCK) for c in ctxs]
    need = [-(-(c + m) // BLOCK) for c, m in zip(ctxs, lens)]
    slots, width, blocks = n + 3, max(need) + 1, sum(need) + 5
    slot = torch.randperm(slots, generator=g, device=DEV)[:n].to(torch.int32)
    ids = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    table = torch.full((slots, width), -1, dtype=torch.int32, device=DEV)
    col = torch.arange(width, device=DEV)[None, :]
    own_rows = torch.full((n, width), -1, dtype=torch.int32, device=DEV)
    own_rows[col < _int(held)[:, None]] = ids[: sum(held)]
    table[slot.long()] = own_rows
    counts = torch.zeros(slots, dtype=torch.int32, device=DEV)
    counts[slot.long()] = _int(held)
    free = torch.zeros(blocks, dtype=torch.int32, device=DEV)
    free[: blocks - sum(held)] = ids[sum(held):]
    cu = [0, *itertools.accumulate(lens)]
    return dict(ctxs=ctxs, lens=lens, need=need, slots=slots, width=width, blocks=blocks, slot=slot, table=table, counts=counts,
                free=free, free_count=_int([blocks - sum(held)]), cu=_int(cu), tokens=cu[-1])


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]

    def randn(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)

    if op.startswith("norm_rope"):
        t, h, hk, d, rd = (case[x] for x in ("t", "h", "hk", "d", "rd"))
        dt = torch.float32 if case["f32"] else torch.bfloat16
        s = dict(case=case)
        if case["fused"]:  # rows of a projection that makes q, k and v at once
            rows = randn(t, (h + 2 * hk) * d, std=1.5, dtype=dt)
            s["q"] = rows[:, : h * d].view(t, h, d)
            s["k"] = rows[:, h * d: (h + hk) * d].view(t, hk, d)
        else:
            s["q"], s["k"] = randn(t, h, d, std=1.5, dtype=dt), randn(t, hk, d, std=1.5, dtype=dt)
        s["w_q"] = 1.0 + randn(d, std=0.2, dtype=torch.float32)
        s["w_k"] = 1.0 + randn(d, std=0.2, dtype=torch.float32)
        n_pos = max(t, 4096)
        s["positions"] = torch.randint(0, n_pos, (t,), generator=g, device=DEV, dtype=torch.int32)
        freq = 10000.0 ** (-torch.arange(0, rd, 2, device=DEV, dtype=torch.float64) / rd)
        angle = torch.arange(n_pos, device=DEV, dtype=torch.float64)[:, None] * freq[None, :]
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        if op == "norm_rope_bwd":
            s["d_q_out"], s["d_k_out"] = randn(t, h, d, dtype=dt), randn(t, hk, d, dtype=dt)
        return s

    tb = _tables(case, g)
    s = dict(case=case, **tb)
    if op == "plan":
        seq_len = torch.zeros(tb["slots"], dtype=torch.int32, device=DEV)
        seq_len[tb["slot"].long()] = _int(tb["ctxs"])
        s["seq_len"] = seq_len
        return s

    h, hk, d = case["h"], case["hk"], case["d"]
    t, slots, blocks, width = tb["tokens"], tb["slots"], tb["blocks"], tb["width"]
    s["q"] = randn(t, h, d, std=1.5)
    s["k"] = randn(t, hk, d)
    s["v"] = randn(t, (h + 2 * hk) * d)[:, (h + hk) * d:].view(t, hk, d)  # the projection's rows hold it
    s["k8"] = torch.empty((blocks, hk, d // 64, 64, 64), dtype=torch.uint8, device=DEV)
    s["v8"] = torch.empty((blocks, hk, d, 64), dtype=torch.uint8, device=DEV)
    s["k_scale"] = torch.empty((blocks, hk), device=DEV)
    s["v_scale"] = torch.empty((blocks, hk), device=DEV)
    for lo in range(0, blocks, 4096):  # a few blocks at a time, for their memory
        hi = min(blocks, lo + 4096)
        x, s["k_scale"][lo:hi] = _quantise(randn(hi - lo, hk, 64, d))
        s["k8"][lo:hi] = x.unflatten(3, (d // 64, 64)).transpose(2, 3)
        x, s["v_scale"][lo:hi] = _quantise(randn(hi - lo, hk, 64, d, std=0.5))
        s["v8"][lo:hi] = x.transpose(2, 3)
    s["tail_k"], s["tail_v"] = randn(slots, hk, 64, d), randn(slots, hk, d, 64, std=0.5)
    # what the step's plan hands to every layer
    lens, ctx = _int(tb["lens"], torch.int64), _int(tb["ctxs"], torch.int64)
    seq = torch.repeat_interleave(torch.arange(case["n"], device=DEV), lens, output_size=t)
    pos = torch.arange(t, device=DEV) - tb["cu"].long()[seq] + ctx[seq]
    new = _int(tb["need"], torch.int64) - tb["counts"].long()[tb["slot"].long()]
    row = torch.repeat_interleave(torch.arange(case["n"], device=DEV), new, output_size=int(new.sum()))
    col = torch.arange(row.numel(), device=DEV) - (new.cumsum(0) - new)[row] + tb["counts"].long()[tb["slot"].long()][row]
    top = int(tb["free_count"])
    s["table"][tb["slot"].long()[row], col] = tb["free"][top - row.numel(): top].flip(0)
    s["ctx_len"], s["positions"] = ctx.to(torch.int32), pos.to(torch.int32)
    s["slot_map"] = s["table"][tb["slot"].long()[seq], pos // BLOCK].long() * BLOCK + pos % BLOCK
    s["max_new"], s["seq"] = max(tb["lens"]), seq
    return s


# ---------------------------------------------------------------------------
# one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"plan": _own_plan, "norm_rope": _own_norm_rope, "norm_rope_bwd": _own_norm_rope_bwd, "decode": _own_attention, "prefill": _own_attention}[op](s)
    return {"plan": _plan, "norm_rope": _norm_rope, "norm_rope_bwd": _norm_rope_bwd, "decode": _attention, "prefill": _attention}[op](s)


def _own_plan(s):
    import bitwise_invariant_gated_amd as gdn

    c = s["case"]
    if "pool" not in s:
        s["pool"] = gdn.AttnPool(s["table"], s["counts"], s["free"], s["free_count"], s["seq_len"])
        s["plan"] = gdn.alloc_attn_plan(s["pool"], c["n"], s["tokens"], slot_index=s["slot"])
    plan = s["plan"]
    gdn.gdn_attn_plan(s["pool"], s["cu"], plan, advance=False)
    out = dict(ctx_len=plan.ctx_len, positions=plan.positions, slot_map=plan.slot_map, status=plan.status)
    if c["release"]:
        gdn.gdn_attn_release(s["pool"], s["slot"])
    return dict(out, table=s["table"], counts=s["counts"], free=s["free"], free_count=s["free_count"])


def _plan(s):
    c, slot, cu = s["case"], s["slot"].long(), s["cu"].long()
    n, t, width = c["n"], s["tokens"], s["width"]
    ctx, held, lens = s["seq_len"][slot].long(), s["counts"][slot].long(), cu[1:] - cu[:-1]
    want = (ctx + lens + BLOCK - 1) // BLOCK
    need = (want - held).clamp(min=0)
    # all of one request's blocks or none; those that need none always go on
    ok = (need == 0) | ((need.cumsum(0) <= s["free_count"]) & (want <= width))
    take = torch.where(ok, need, 0)
    first = take.cumsum(0) - take
    col = torch.arange(width, device=DEV)[None, :]
    fresh = (col >= held[:, None]) & (col < (held + take)[:, None])
    at = s["free_count"].long() - 1 - (first[:, None] + col - held[:, None])
    rows = torch.where(fresh, s["free"][at.clamp(0, s["blocks"] - 1)], s["table"][slot])
    s["table"][slot] = rows
    s["counts"][slot] = (held + take).to(torch.int32)
    s["free_count"] -= take.sum().to(torch.int32)
    tok = torch.arange(t, device=DEV)
    seq = torch.searchsorted(cu[1:], tok, right=True)
    pos = tok - cu[seq] + ctx[seq]
    where = rows.reshape(-1)[seq * width + torch.clamp(pos // BLOCK, max=width - 1)].long() * BLOCK + pos % BLOCK
    out = dict(ctx_len=torch.where(ok, ctx, -1).to(torch.int32), positions=pos.to(torch.int32), slot_map=torch.where(ok[seq], where, -1),
               status=(~ok).sum().to(torch.int32).reshape(1))
    if c["release"]:  # the last taken block ends on top of what was free, so that it is the first to go out again
        held = s["counts"][slot].long()
        last = held.flip(0).cumsum(0).flip(0) - held
        at = s["free_count"].long() + last[:, None] + held[:, None] - 1 - col
        got = col < held[:, None]
        s["free"][at[got]] = s["table"][slot][got]
        s["free_count"] += held.sum().to(torch.int32)
        s["table"][slot] = -1
        s["counts"][slot] = 0
    return dict(out, table=s["table"], counts=s["counts"], free=s["free"], free_count=s["free_count"])


EPS = 1e-6


def _own_rope(s):
    import bitwise_invariant_gated_amd as gdn

    c = s["case"]
    if "shape" not in s:
        s["shape"] = gdn.AttnShape(c["h"], c["hk"], c["d"], torch.float32 if c["f32"] else torch.bfloat16)
        s["rope"] = gdn.AttnRope(c["rd"], interleaved=c["inter"], eps=EPS)
        s["out"] = (torch.empty((c["t"], c["h"], c["d"]), dtype=s["q"].dtype, device=DEV), torch.empty((c["t"], c["hk"], c["d"]), dtype=s["q"].dtype, device=DEV))
        if c["op"] == "norm_rope_bwd":
            s["dw"] = torch.empty(c["d"], device=DEV), torch.empty(c["d"], device=DEV)
            s["ws"] = gdn.alloc_attn_workspace(s["shape"], gdn.GDN_ATTN_OP_NORM_ROPE_BWD, c["t"], device=DEV)
    return gdn


def _own_norm_rope(s):
    gdn = _own_rope(s)
    q, k = s["out"]
    gdn.gdn_attn_qk_norm_rope(s["shape"], s["rope"], s["q"], s["k"], s["w_q"], s["w_k"], s["cos_sin"], s["positions"], q, k)
    return dict(q=q, k=k)


def _own_norm_rope_bwd(s):
    gdn = _own_rope(s)
    (dq, dk), (dw_q, dw_k) = s["out"], s["dw"]
    gdn.gdn_attn_qk_norm_rope_bwd(s["shape"], s["rope"], s["q"], s["k"], s["w_q"], s["w_k"], s["cos_sin"], s["positions"],
                                  s["d_q_out"], s["d_k_out"], dq, dk, dw_q, dw_k, s["ws"])
    return dict(dq=dq, dk=dk, dw_q=dw_q, dw_k=dw_k)


def _halves(x, inter):
    """The two members of every rotated pair."""
    return (x[..., 0::2], x[..., 1::2]) if inter else x.chunk(2, -1)


def _join(a, b, inter):
    return torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)


def _rotate(x, s, back=False):
    c = s["case"]
    cos, sin = s["cos_sin"][s["positions"].long()][:, None, :].chunk(2, -1)
    if back:
        sin = -sin
    a, b = _halves(x[..., : c["rd"]], c["inter"])
    return torch.cat([_join(a * cos - b * sin, b * cos + a * sin, c["inter"]), x[..., c["rd"]:]], -1)


def _norm_rope(s):
    def one(x, w):
        x = x.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        return _rotate(x * r * w, s).to(s["q"].dtype)

    return dict(q=one(s["q"], s["w_q"]), k=one(s["k"], s["w_k"]))


def _norm_rope_bwd(s):
    def one(x, w, dy):
        x = x.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        dn, xh = _rotate(dy.float(), s, back=True), x * r
        dxh = dn * w
        dx = r * (dxh - xh * (dxh * xh).mean(-1, keepdim=True))
        return dx.to(s["q"].dtype), (dn * xh).sum((0, 1))

    dq, dw_q = one(s["q"], s["w_q"], s["d_q_out"])
    dk, dw_k = one(s["k"], s["w_k"], s["d_k_out"])
    return dict(dq=dq, dk=dk, dw_q=dw_q, dw_k=dw_k)


def _own_attention(s):
    import bitwise_invariant_gated_amd as gdn

    c = s["case"]
    if "cache" not in s:
        s["shape"] = gdn.AttnShape(c["h"], c["hk"], c["d"])
        s["cache"] = gdn.AttnCache(s["k8"], s["v8"], s["k_scale"], s["v_scale"], s["tail_k"], s["tail_v"])
        s["plan"] = gdn.AttnPlan(s["ctx_len"], s["positions"], s["slot_map"], _int([0]), s["table"], s["slot"])
        s["o"] = torch.empty_like(s["q"])
        op = gdn.GDN_ATTN_OP_DECODE if c["op"] == "decode" else gdn.GDN_ATTN_OP_PREFILL
        s["ws"] = gdn.alloc_attn_workspace(s["shape"], op, s["tokens"], c["n"], s["blocks"], device=DEV)
    if c["op"] == "decode":
        gdn.gdn_attn_decode_step(s["shape"], s["q"], s["k"], s["v"], s["plan"], s["cache"], s["o"], s["ws"])
    else:
        gdn.gdn_attn_prefill(s["shape"], s["q"], s["k"], s["v"], s["cu"], s["plan"], s["cache"], s["o"], s["ws"], max_new=s["max_new"])
    return _cache_out(s, s["o"])


def _cache_out(s, o):
    f8 = torch.float8_e4m3fn
    return dict(o=o, k8=s["k8"].view(f8), v8=s["v8"].view(f8), k_scale=s["k_scale"], v_scale=s["v_scale"], tail_k=s["tail_k"], tail_v=s["tail_v"])


def _quantise(x):
    """Blocks [..., Hk, 64, d] -> their e4m3 bytes and scales [..., Hk]."""
    x = x.float()
    most = torch.where(torch.isfinite(x), x.abs(), 0).amax((-2, -1))
    m, e = torch.frexp(most)  # most = m * 2^e, 448 = 0.875 * 2^9
    scale = torch.exp2((e - 9 + (m > 0.875)).float().clamp(min=-100))
    return (x / scale[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _attention(s):
    c = s["case"]
    n, t, h, hk, d = c["n"], s["tokens"], c["h"], c["hk"], c["d"]
    grp, scale, slot = h // hk, d ** -0.5, s["slot"].long()
    ctx, pos, seq = s["ctx_len"].long(), s["positions"].long(), s["seq"]
    end = ctx + s["cu"].long()[1:] - s["cu"].long()[:-1]
    local = pos - ctx[seq]
    # the tokens from each sequence's first open block on, in the input type: old tail rows, then new tokens
    base = ctx // BLOCK * BLOCK
    span = (BLOCK - 1 + s["max_new"] + BLOCK - 1) // BLOCK * BLOCK
    raw_k = torch.zeros((n, span, hk, d), dtype=s["q"].dtype, device=DEV)
    raw_v = torch.zeros((n, span, hk, d), dtype=s["q"].dtype, device=DEV)
    kept = (torch.arange(BLOCK, device=DEV) < (ctx - base)[:, None])[:, :, None, None]
    raw_k[:, :BLOCK] = torch.where(kept, s["tail_k"][slot].transpose(1, 2), 0)
    raw_v[:, :BLOCK] = torch.where(kept, s["tail_v"][slot].permute(0, 3, 1, 2), 0)
    raw_k[seq, pos - base[seq]] = s["k"]
    raw_v[seq, pos - base[seq]] = s["v"]
    # blocks that are full now go into the cache
    wide = torch.arange(span // BLOCK, device=DEV)[None, :]
    full = (base[:, None] // BLOCK + wide + 1) * BLOCK <= end[:, None]
    k8, k_scale = _quantise(raw_k.unflatten(1, (-1, BLOCK))[full].transpose(1, 2))
    v8, v_scale = _quantise(raw_v.unflatten(1, (-1, BLOCK))[full].transpose(1, 2))
    ids = s["table"][slot].long().gather(1, (base[:, None] // BLOCK + wide).clamp(max=s["width"] - 1))[full]
    s["k8"][ids] = k8.unflatten(3, (d // 64, 64)).transpose(2, 3)
    s["v8"][ids] = v8.transpose(2, 3)
    s["k_scale"][ids], s["v_scale"][ids] = k_scale, v_scale
    # and the last token's block stays in the tail
    last = pos // BLOCK == (end[seq] - 1) // BLOCK
    s["tail_k"][slot[seq[last]], :, pos[last] % BLOCK] = s["k"][last]
    s["tail_v"][slot[seq[last]], :, :, pos[last] % BLOCK] = s["v"][last]
    # the cache in 32 bits, [n, hk, tokens, d]
    f8 = torch.float8_e4m3fn
    ids = s["table"][slot].long().clamp(min=0)
    all_k = s["k8"].view(f8)[ids].float().transpose(3, 4).flatten(4) * s["k_scale"][ids][..., None, None]
    all_v = s["v8"].view(f8)[ids].float().transpose(3, 4) * s["v_scale"][ids][..., None, None]
    all_k, all_v = all_k.transpose(1, 2).flatten(2, 3), all_v.transpose(1, 2).flatten(2, 3)
    width = all_k.shape[2]
    # scores of the earlier blocks, for queries padded to [n, hk, max_new * grp, d]
    q = torch.zeros((n, s["max_new"], h, d), device=DEV)
    q[seq, local] = s["q"].float()
    q = q.unflatten(2, (hk, grp)).transpose(1, 2).flatten(2, 3)
    first = torch.zeros((n, s["max_new"]), dtype=torch.int64, device=DEV)
    first[seq, local] = pos // BLOCK * BLOCK
    seen = torch.arange(width, device=DEV) < first[:, :, None]
    far = torch.matmul(q, all_k.transpose(2, 3).contiguous()).unflatten(2, (s["max_new"], grp)) * scale
    far = torch.where(seen[:, None, :, None, :], far, -torch.inf)
    # and of the own block's tokens, per token
    cols = (pos // BLOCK * BLOCK - base[seq])[:, None] + torch.arange(BLOCK, device=DEV)[None, :]
    near_k, near_v = raw_k[seq[:, None], cols].float().transpose(1, 2), raw_v[seq[:, None], cols].float().transpose(1, 2)
    near = torch.matmul(s["q"].float().unflatten(1, (hk, grp)), near_k.transpose(2, 3).contiguous()) * scale
    near = torch.where(torch.arange(BLOCK, device=DEV) <= (pos % BLOCK)[:, None, None, None], near, -torch.inf)
    # one softmax over both
    most = torch.maximum(far.amax(-1).transpose(1, 2)[seq, local], near.amax(-1))
    pad = torch.zeros((n, s["max_new"], hk, grp), device=DEV)
    pad[seq, local] = most
    far = torch.exp(far - pad.transpose(1, 2)[..., None])
    near = torch.exp(near - most[..., None])
    total = far.sum(-1).transpose(1, 2)[seq, local] + near.sum(-1)
    o = torch.matmul(far.flatten(2, 3), all_v).unflatten(2, (s["max_new"], grp)).transpose(1, 2)[seq, local]
    o = (o + torch.matmul(near, near_v)) / total[..., None]
    return _cache_out(s, o.flatten(1, 2).to(s["q"].dtype))


# ---------------------------------------------------------------------------
# the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return _exact_plan(s)
    if op.startswith("norm_rope"):
        return _exact_norm_rope(s)
    return _exact_attention(s)


def _exact_plan(s):
    """The requests one after the other, on the host."""
    c = s["case"]
    slot, cu, lens = s["slot"].tolist(), s["cu"].tolist(), s["seq_len"].tolist()
    table, counts = s["table"].tolist(), s["counts"].tolist()
    free = s["free"].tolist()
    top, asked = int(s["free_count"]), 0
    there = top
    ctx_len, positions, slot_map, refused = [], [], [], 0
    for i, r in enumerate(slot):
        m = cu[i + 1] - cu[i]
        want = -(-(lens[r] + m) // BLOCK)
        need = max(0, want - counts[r])
        asked += need
        fine = need == 0 or (asked <= there and want <= s["width"])
        for _ in range(need if fine else 0):
            top -= 1
            table[r][counts[r]] = free[top]
            counts[r] += 1
        refused += not fine
        ctx_len.append(lens[r] if fine else -1)
        for p in range(lens[r], lens[r] + m):
            positions.append(p)
            slot_map.append(table[r][p // BLOCK] * BLOCK + p % BLOCK if fine else -1)
    if c["release"]:
        for r in reversed(slot):
            for j in reversed(range(counts[r])):
                free[top] = table[r][j]
                top += 1
            table[r] = [-1] * s["width"]
            counts[r] = 0
    return dict(ctx_len=_int(ctx_len), positions=_int(positions), slot_map=_int(slot_map, torch.int64), status=_int([refused]),
                table=_int(table), counts=_int(counts), free=_int(free), free_count=_int([top]))


def _exact_norm_rope(s):
    c = s["case"]
    rd, out = c["rd"], {}
    table = s["cos_sin"].double()[s["positions"].long()]
    for x, w in (("q", "w_q"), ("k", "w_k")):
        a, b = s[x].double().requires_grad_(), s[w].double().requires_grad_()
        y = b * a / torch.sqrt(a.pow(2).sum(-1, keepdim=True) / c["d"] + EPS)
        z = list(y.unbind(-1))
        for i in range(rd // 2):  # pair by pair
            u, v = (2 * i, 2 * i + 1) if c["inter"] else (i, i + rd // 2)
            cos, sin = table[:, i, None], table[:, rd // 2 + i, None]
            z[u], z[v] = z[u] * cos - z[v] * sin, z[v] * cos + z[u] * sin
        y = torch.stack(z, -1)
        if c["op"] == "norm_rope":
            out[x] = y.detach()
        else:
            out["d" + x], out["d" + w] = torch.autograd.grad(y, (a, b), s["d_%s_out" % x].double())
    return out


def _e4m3_values():
    """What each of the 256 codes stands for: sign, 4 bits of exponent with bias 7, 3 of fraction, all ones for no number."""
    got = []
    for code in range(256):
        e, f = code >> 3 & 15, code & 7
        x = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        got.append(float("nan") if code & 127 == 127 else -x if code & 128 else x)
    return got


def _exact_attention(s):
    c = s["case"]
    h, hk, d = c["h"], c["hk"], c["d"]
    grp = h // hk
    values = torch.tensor(_e4m3_values(), dtype=torch.float64, device=DEV)
    good = torch.tensor([x for x in _e4m3_values()[:127]], dtype=torch.float64, device=DEV)  # ascending magnitudes
    k8, v8, ks, vs = s["k8"], s["v8"], s["k_scale"].double(), s["v_scale"].double()
    tail_k, tail_v = s["tail_k"].double(), s["tail_v"].double()
    o = torch.empty((s["tokens"], h, d), dtype=torch.float64, device=DEV)
    cu, slots = s["cu"].tolist(), s["slot"].tolist()

    def to8(x):
        """Codes and scale of one head's block [64, d], to the nearest value, to the even code between two."""
        most, e = float(x.abs().max()), -100
        if most > 0:
            while e < 120 and most > 448 * 2.0 ** e:
                e += 1
        y = x.abs() * 2.0 ** -e
        hi = torch.searchsorted(good, y).clamp(max=126)
        lo = (hi - 1).clamp(min=0)
        up, down = good[hi] - y, y - good[lo]
        code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
        return torch.where(torch.signbit(x), code + 128, code).to(torch.uint8), 2.0 ** e

    for i, (ctx, m) in enumerate(zip(s["ctxs"], s["lens"])):
        blocks = s["table"][slots[i]].long().tolist()
        k, v = s["k"][cu[i]: cu[i] + m].double(), s["v"][cu[i]: cu[i] + m].double()
        lo = ctx // BLOCK * BLOCK
        k = torch.cat([tail_k[slots[i], :, : ctx - lo].transpose(0, 1), k])
        v = torch.cat([tail_v[slots[i], :, :, : ctx - lo].permute(2, 0, 1), v])
        for b in range(lo // BLOCK, (ctx + m) // BLOCK):
            for j in range(hk):
                code, ks[blocks[b], j] = to8(k[b * BLOCK - lo: (b + 1) * BLOCK - lo, j])
                for part in range(d // 64):
                    k8[blocks[b], j, part] = code[:, 64 * part: 64 * part + 64]
                code, vs[blocks[b], j] = to8(v[b * BLOCK - lo: (b + 1) * BLOCK - lo, j])
                v8[blocks[b], j] = code.t()
        first = (ctx + m - 1) // BLOCK * BLOCK
        for p in range(max(first, ctx), ctx + m):
            tail_k[slots[i], :, p - first] = k[p - lo]
            tail_v[slots[i], :, :, p - first] = v[p - lo]
        ids = s["table"][slots[i]].long()[: (ctx + m - 1) // BLOCK]
        for j in range(hk):
            old_k = torch.cat([values[k8[ids, j, part].long()].flatten(0, 1) for part in range(d // 64)], -1) * ks[ids, j].repeat_interleave(BLOCK)[:, None]
            old_v = values[v8[ids, j].long()].transpose(1, 2).flatten(0, 1) * vs[ids, j].repeat_interleave(BLOCK)[:, None]
            step = max(BLOCK, (1 << 27) // max(1, grp * (ctx + m)) // BLOCK * BLOCK)
            for a in range(lo, ctx + m, step):  # queries a .. b, by whole blocks
                ab, b = max(a, ctx), min(a + step, ctx + m)
                if ab >= b:
                    continue
                q = s["q"][cu[i] + ab - ctx: cu[i] + b - ctx, j * grp: (j + 1) * grp].double().flatten(0, 1)
                at = torch.arange(ab, b, device=DEV).repeat_interleave(grp)[:, None]
                x = torch.cat([q @ old_k.t(), q @ k[a - lo: b - lo, j].t()], 1) * d ** -0.5
                old, new = torch.arange(len(old_k), device=DEV)[None, :], torch.arange(a, b, device=DEV)[None, :]
                seen = torch.cat([old < at // BLOCK * BLOCK, (new <= at) & (new >= at // BLOCK * BLOCK)], 1)
                p = torch.softmax(x.masked_fill(~seen, -torch.inf), 1)
                y = p[:, : len(old_k)] @ old_v + p[:, len(old_k):] @ v[a - lo: b - lo, j]
                o[cu[i] + ab - ctx: cu[i] + b - ctx, j * grp: (j + 1) * grp] = y.unflatten(0, (b - ab, grp))
    f8 = torch.float8_e4m3fn
    return dict(o=o, k8=k8.view(f8).float(), v8=v8.view(f8).float(), k_scale=ks, v_scale=vs, tail_k=tail_k, tail_v=tail_v)
