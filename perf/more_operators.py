"""Operators around the layers of a stack, case by case: what each is called with, its plain form
in elementary torch operations, and its value in 64 bits.

They are what a hybrid stack needs between its layers and at its end: the root-mean-square norm with
the residual's addition, in the input type and in 8 bits with scales, and its gradient ("add_norm",
"add_norm_bwd"); the log probabilities of given tokens with the entropy and the top alternatives, and
their gradient ("logprobs", "logprobs_bwd"); the divergence from a teacher's top entries, and its
gradient ("distill", "distill_bwd").

Definitions.
  add_norm   h = x + residual, rounded to the residual's type; y = h w / sqrt(mean(h^2) + eps), with h as
             rounded; y8 = y / s in e4m3 with s = max(amax(y), 2^-100) / 448 per row or per 128 columns.
  logprobs   with z = scale * logits of a row (scale: one number per row): log softmax(z) of the target,
             the entropy of softmax(z), and the `top` largest logits' indices (ties to the lowest) with
             their log softmax.  A row whose target is no index of the vocabulary is left out: zeros, and
             indices -1.  stats: the row's largest logit and log sum exp(z - max z).
  distill    sum over the teacher's entries of p (log p - log softmax(z)), where p is the softmax of
             scale * values over the row's entries, or exp(values).  Entries whose index is no index of
             the vocabulary are not there.  stats: those of logprobs, then the same two of the teacher's
             values (0 and 0 where they are log probabilities).
"""

import math

import torch

own = False
DEV = "cuda"
EPS = 1e-6
GROUP = 128


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # one decoded token between two layers: latency alone
        dict(name="add_norm_1_token", op="add_norm", t=1, w=2048, f32=False, res32=False, add=True, y=True, group=-1),
        # a packed batch of prompts, 16 heads of 128: the norm before a projection in the input type
        dict(name="add_norm_10240", op="add_norm", t=10240, w=2048, f32=False, res32=False, add=True, y=True, group=-1),
        # the same before a projection in 8 bits, a scale to 128 columns, over a stream in 32 bits
        dict(name="add_norm_8bit_10240", op="add_norm", t=10240, w=4096, f32=False, res32=True, add=True, y=False, group=GROUP),
        # a decode batch, both outputs, a scale to a row; odd sizes
        dict(name="add_norm_8bit_255", op="add_norm", t=255, w=5000, f32=False, res32=False, add=True, y=True, group=0),
        # the gradient over a trainer's tokens
        dict(name="add_norm_bwd_10240", op="add_norm_bwd", t=10240, w=2048, f32=False, res32=False, add=True),
        # the same, all in 32 bits, odd sizes, no residual gradient: the norm before the logits
        dict(name="add_norm_bwd_2047_f32", op="add_norm_bwd", t=2047, w=1000, f32=True, res32=True, add=False),
        # a decode step of 256 requests, 20 alternatives each, a temperature per request
        dict(name="logprobs_256_top20", op="logprobs", t=256, v=131072, pad=0, f32=False, top=20, scaled=True, masked=False, left=False),
        # one request's next token, logits in 32 bits, an odd vocabulary
        dict(name="logprobs_1_top5_f32", op="logprobs", t=1, v=100003, pad=0, f32=True, top=5, scaled=False, masked=False, left=False),
        # a trainer scoring rollouts: log probabilities and entropy
        dict(name="logprobs_4096", op="logprobs", t=4096, v=131072, pad=0, f32=False, top=0, scaled=False, masked=False, left=False),
        # the gradient of both; padded rows left out, some vocabularies masked
        dict(name="logprobs_bwd_2048", op="logprobs_bwd", t=2048, v=131072, pad=0, f32=False, scaled=True, masked=True, left=True),
        # the divergence from 64 teacher entries a token
        dict(name="distill_2048_top64", op="distill", t=2048, v=131072, pad=0, f32=False, k=64, logp=False, scaled=True, masked=False),
        # its gradient, odd vocabulary in 32 bits, padded rows, the teacher's entries as log probabilities
        dict(name="distill_bwd_513_top17_f32", op="distill_bwd", t=513, v=50001, pad=7, f32=True, k=17, logp=True, scaled=False, masked=False),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["add_norm", "add_norm", "add_norm_bwd", "logprobs", "logprobs", "logprobs_bwd", "distill", "distill_bwd"])
    f32 = rng.random() < 0.3
    if op.startswith("add_norm"):
        w = 8 * _log(rng, 8, 1024)
        t = _log(rng, 1, min(20000, 10240 * 2048 // w))
        c = dict(op=op, t=t, w=w, f32=f32, res32=f32 or rng.random() < 0.4, add=rng.random() < 0.85)
        if op == "add_norm":
            group = rng.choice([-1, 0, GROUP if w % GROUP == 0 else 0])
            c.update(y=group < 0 or rng.random() < 0.5, group=group)
        return c
    v = _log(rng, 64, 200000)
    t = _log(rng, 1, min(8192, (2048 if op != "logprobs" else 4096) * 131072 // (2 if f32 else 1) // v))
    c = dict(op=op, t=t, v=v, pad=rng.choice([0, 0, -v % 64, 5]), f32=f32, scaled=rng.random() < 0.5, masked=rng.random() < 0.3)
    if op.startswith("logprobs"):
        c["left"] = rng.random() < 0.3
        if op == "logprobs":
            c["top"] = rng.choice([0, 0, _log(rng, 1, 64)])
    else:
        c.update(k=_log(rng, 1, min(v, 128)), logp=rng.random() < 0.5)
    return c


def work(case):
    t, size = case["t"], 4 if case["f32"] else 2
    if case["op"].startswith("add_norm"):
        w, res = case["w"], 4 if case["res32"] else 2
        if case["op"] == "add_norm_bwd":
            per = res + size + (res if case["add"] else 0) + size + (res if case["add"] and res != size else 0)
            return {"bytes": t * w * per + 8 * w, "flops": 12 * t * w}
        per = size + (2 * res if case["add"] else 0) + (size if case["y"] else 0) + (1 if case["group"] >= 0 else 0)
        scales = 0 if case["group"] < 0 else 4 * t * (w // GROUP if case["group"] else 1)
        return {"bytes": t * w * per + scales + 4 * w, "flops": 6 * t * w}
    n = t * case["v"]
    if case["op"].endswith("_bwd"):
        return {"bytes": 2 * n * size + t * 24 + 8 * t * case.get("k", 0), "flops": 8 * n}
    return {"bytes": n * size + t * 24 + 8 * t * (case.get("k", 0) + case.get("top", 0)), "flops": 7 * n}


# ---------------------------------------------------------------------------
# inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c = dict(case)
    t = c["t"]
    dt = torch.float32 if c["f32"] else torch.bfloat16

    def randn(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=DEV, dtype=dtype)

    s = dict(case=c)
    if c["op"].startswith("add_norm"):
        w, rdt = c["w"], torch.float32 if c["res32"] else torch.bfloat16
        s["w"] = 1.0 + 0.2 * randn(w)
        if c["op"] == "add_norm":
            s["x"] = randn(t, w, dtype=dt)
            s["residual"] = randn(t, w, dtype=rdt) * 4 if c["add"] else None
        else:
            s["h"] = randn(t, w, dtype=rdt) * 4
            s["dy"] = randn(t, w, dtype=dt)
            s["d_res"] = randn(t, w, dtype=rdt) if c["add"] else None
        return s

    v = c["v"]
    rows = torch.arange(t, device=DEV)
    # logits: a wide bulk and, in most rows, a few tokens that stand out; the rows may be padded
    buf = randn(t, v + c["pad"], dtype=dt) * 2.5
    s["logits"] = buf[:, :v]
    reach = torch.where(rows % 5 == 0, max(1, v // 3), v) if c["masked"] else torch.full((t,), v, device=DEV)
    target = (torch.rand((t,), generator=g, device=DEV, dtype=torch.float64) * reach).long()
    rise = torch.rand((t,), generator=g, device=DEV) * 14
    s["logits"][rows, target] += rise.to(dt)
    if c["masked"]:  # a grammar leaves these rows a third of the vocabulary
        s["logits"][::5, max(1, v // 3):] = -torch.inf
    s["scale"] = 0.6 + 0.8 * torch.rand((t,), generator=g, device=DEV) if c["scaled"] else None
    if c["op"].startswith("logprobs"):
        if c["left"]:  # padding of a batch of fixed size
            target = torch.where(rows % 7 == 3, -1, target)
        s["target"] = target.to(torch.int32)
        if c["op"] == "logprobs_bwd":
            kept = _stats(s)
            s["stats"], s["entropy"] = kept["stats"], kept["entropy"]
            s["d_logprobs"] = randn(t) / math.sqrt(t)
            s["d_entropy"] = 0.01 * randn(t) / math.sqrt(t)
        return s
    k = c["k"]
    # the teacher's entries: the target and others, each once, values falling; a tenth of the rows has fewer
    start = (torch.rand((t,), generator=g, device=DEV, dtype=torch.float64) * v).long()
    step = 1 + (torch.rand((t,), generator=g, device=DEV, dtype=torch.float64) * max(1, v // k - 1)).long()
    ids = (start[:, None] + step[:, None] * torch.arange(k, device=DEV)) % v
    ids = torch.where(ids % v < reach[:, None], ids, -1)
    few = (rows % 10 == 9)[:, None] & (torch.arange(k, device=DEV) >= max(1, k // 2))
    s["ids"] = torch.where(few, -1, ids).to(torch.int32)
    values = (rise[:, None] + 3 * randn(t, k)).sort(-1, descending=True).values
    if c["logp"]:
        values = values - torch.logsumexp(values, -1, keepdim=True) - 0.05
    s["values"] = values.contiguous()
    if c["op"] == "distill_bwd":
        s["stats"] = torch.cat([_stats(s)["stats"], _teacher(s)[1]], -1)
        s["d_loss"] = (0.5 + torch.rand((t,), generator=g, device=DEV)) / t
    return s


# ---------------------------------------------------------------------------
# one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"add_norm": _own_add_norm, "add_norm_bwd": _own_add_norm_bwd, "logprobs": _own_logprobs, "logprobs_bwd": _own_logprobs_bwd,
                "distill": _own_distill, "distill_bwd": _own_distill_bwd}[op](s)
    return {"add_norm": _add_norm, "add_norm_bwd": _add_norm_bwd, "logprobs": _logprobs, "logprobs_bwd": _logprobs_bwd,
            "distill": _distill, "distill_bwd": _distill_bwd}[op](s)


# the framework's calls: outputs and workspaces are allocated once, as a program with a fixed batch does

def _own_norm(s):
    import bitwise_invariant_gated_amd as gdn

    c = s["case"]
    if "shape" not in s:
        dt, rdt = (torch.float32 if f else torch.bfloat16 for f in (c["f32"], c["res32"]))
        s["shape"] = gdn.NormShape(c["w"], dt, rdt, group=c.get("group", -1), eps=EPS)
        t, w = c["t"], c["w"]
        if c["op"] == "add_norm":
            s["h"] = torch.empty((t, w), dtype=rdt, device=DEV) if c["add"] else None
            s["y"] = torch.empty((t, w), dtype=dt, device=DEV) if c["y"] else None
            s["y8"] = s["y_scale"] = None
            if c["group"] >= 0:
                s["y8"] = torch.empty((t, w), dtype=torch.uint8, device=DEV)
                s["y_scale"] = torch.empty((t, w // c["group"] if c["group"] else 1), device=DEV)
        else:
            s["dx"] = torch.empty((t, w), dtype=dt, device=DEV)
            s["d_residual"] = torch.empty((t, w), dtype=rdt, device=DEV) if c["add"] and rdt != dt else None
            s["dw"] = torch.empty(w, device=DEV)
            s["ws"] = gdn.alloc_norm_workspace(s["shape"], t, DEV)
    return gdn


def _own_add_norm(s):
    gdn = _own_norm(s)
    gdn.gdn_stack_add_norm(s["shape"], s["x"], s["residual"], s["w"], s["h"], s["y"], s["y8"], s["y_scale"])
    return dict(h=s["h"], y=s["y"], y8=None if s["y8"] is None else s["y8"].view(torch.float8_e4m3fn), y_scale=s["y_scale"])


def _own_add_norm_bwd(s):
    gdn = _own_norm(s)
    gdn.gdn_stack_add_norm_bwd(s["shape"], s["h"], s["w"], s["dy"], s["d_res"], s["dx"], s["d_residual"], s["dw"], s["ws"])
    return dict(dx=s["dx"], d_residual=s["d_residual"], dw=s["dw"])


def _own_logits(s):
    import bitwise_invariant_gated_amd as gdn

    c = s["case"]
    if "shape" not in s:
        t, v = c["t"], c["v"]
        dt = torch.float32 if c["f32"] else torch.bfloat16
        i32, f32 = dict(dtype=torch.int32, device=DEV), dict(dtype=torch.float32, device=DEV)
        top = c.get("top", c.get("k", 0))
        s["shape"] = gdn.LogitsShape(v, dt, top, teacher_logprobs=c.get("logp", False))
        if c["op"].endswith("_bwd"):
            s["d_logits"] = torch.empty((t, v), dtype=dt, device=DEV)
        else:
            s["ws"] = gdn.alloc_logits_workspace(s["shape"], t, DEV)
            if c["op"] == "logprobs":
                s["logprobs"], s["entropy"], s["stats"] = torch.empty(t, **f32), torch.empty(t, **f32), torch.empty((t, 2), **f32)
                s["top_ids"], s["top_logprobs"] = (torch.empty((t, top), **i32), torch.empty((t, top), **f32)) if top else (None, None)
            else:
                s["loss"], s["stats"] = torch.empty(t, **f32), torch.empty((t, 4), **f32)
    return gdn


def _own_logprobs(s):
    gdn = _own_logits(s)
    gdn.gdn_stack_logprobs(s["shape"], s["logits"], s["target"], s["logprobs"], s["entropy"], s["top_ids"], s["top_logprobs"], s["stats"],
                           s["ws"], scale=s["scale"])
    return {n: s[n] for n in ("logprobs", "entropy", "stats", "top_ids", "top_logprobs")}


def _own_logprobs_bwd(s):
    gdn = _own_logits(s)
    gdn.gdn_stack_logprobs_bwd(s["shape"], s["logits"], s["target"], s["stats"], s["entropy"], s["d_logprobs"], s["d_entropy"], s["d_logits"],
                               scale=s["scale"])
    return dict(d_logits=s["d_logits"])


def _own_distill(s):
    gdn = _own_logits(s)
    gdn.gdn_stack_distill(s["shape"], s["logits"], s["ids"], s["values"], s["loss"], s["stats"], s["ws"], scale=s["scale"])
    return dict(loss=s["loss"], stats=s["stats"])


def _own_distill_bwd(s):
    gdn = _own_logits(s)
    gdn.gdn_stack_distill_bwd(s["shape"], s["logits"], s["ids"], s["values"], s["stats"], s["d_loss"], s["d_logits"], scale=s["scale"])
    return dict(d_logits=s["d_logits"])


# the plain forms, in 32 bits, rounded once at the end

def _add_norm(s):
    c = s["case"]
    h = s["x"].float()
    if c["add"]:
        h = (h + s["residual"].float()).to(s["residual"].dtype)
    f = h.float()
    y = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS) * s["w"]
    out = dict(h=h if c["add"] else None, y=y.to(s["x"].dtype) if c["y"] else None, y8=None, y_scale=None)
    if c["group"] >= 0:
        z = y.unflatten(1, (-1, c["group"] or c["w"]))
        scale = z.abs().amax(-1).clamp(min=2.0 ** -100) / 448
        out["y8"] = (z / scale[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).flatten(1)
        out["y_scale"] = scale
    return out


def _add_norm_bwd(s):
    h, dy = s["h"].float(), s["dy"].float()
    r = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    n = h * r
    dn = dy * s["w"]
    dh = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    if s["d_res"] is not None:
        dh = dh + s["d_res"].float()
    both = s["d_res"] is not None and s["h"].dtype != s["dy"].dtype
    return dict(dx=dh.to(s["dy"].dtype), d_residual=dh.to(s["h"].dtype) if both else None, dw=(dy * n).sum(0))


def _scaled(s):
    """The distance of every logit from its row's largest, scaled; the largest; log sum exp of the distances."""
    x = s["logits"].float()
    m = x.amax(-1)
    d = x - m[:, None]
    if s["scale"] is not None:
        d = d * s["scale"][:, None]
    return d, m, d.exp().sum(-1).log()


def _stats(s):
    d, m, log_l = _scaled(s)
    logq = d - log_l[:, None]
    entropy = -torch.where(d > -torch.inf, logq.exp() * logq, 0).sum(-1)
    return dict(stats=torch.stack([m, log_l], -1), entropy=entropy)


def _logprobs(s):
    c = s["case"]
    d, m, log_l = _scaled(s)
    keep = (s["target"] >= 0) & (s["target"] < c["v"])
    logq = d - log_l[:, None]
    at = s["target"].long().clamp(0, c["v"] - 1)[:, None]
    out = dict(logprobs=torch.where(keep, logq.gather(1, at)[:, 0], 0),
               entropy=torch.where(keep, -torch.where(d > -torch.inf, logq.exp() * logq, 0).sum(-1), 0),
               stats=torch.where(keep[:, None], torch.stack([m, log_l], -1), 0), top_ids=None, top_logprobs=None)
    if c["top"]:
        ids = s["logits"].sort(dim=-1, descending=True, stable=True).indices[:, : c["top"]]
        out["top_ids"] = torch.where(keep[:, None], ids, -1).to(torch.int32)
        out["top_logprobs"] = torch.where(keep[:, None], logq.gather(1, ids), 0)
    return out


def _log_q(s):
    """Log probabilities from the forward's statistics."""
    d = s["logits"].float() - s["stats"][:, :1]
    if s["scale"] is not None:
        d = d * s["scale"][:, None]
    return d - s["stats"][:, 1:2]


def _logprobs_bwd(s):
    c = s["case"]
    logq = _log_q(s)
    q = logq.exp()
    keep = (s["target"] >= 0) & (s["target"] < c["v"])
    g, gh = torch.where(keep, s["d_logprobs"], 0), torch.where(keep, s["d_entropy"], 0)
    dz = -q * (g[:, None] + torch.where(q > 0, gh[:, None] * (logq + s["entropy"][:, None]), 0))
    dz.scatter_add_(1, s["target"].long().clamp(0, c["v"] - 1)[:, None], g[:, None])
    if s["scale"] is not None:
        dz = dz * s["scale"][:, None]
    return dict(d_logits=dz.to(s["logits"].dtype))


def _teacher(s):
    """p and log p of the teacher's entries, 0 and -inf for those that are not there, and the two statistics."""
    c = s["case"]
    there = (s["ids"] >= 0) & (s["ids"] < c["v"])
    x = torch.where(there, s["values"], -torch.inf)
    if c["logp"]:
        return x, torch.zeros((c["t"], 2), device=DEV)
    m = x.amax(-1, keepdim=True)
    none = m == -torch.inf
    d = x - torch.where(none, 0, m)
    if s["scale"] is not None:
        d = d * s["scale"][:, None]
    log_l = torch.where(none, 0, d.exp().sum(-1, keepdim=True).log())
    return d - log_l, torch.cat([torch.where(none, 0, m), log_l], -1)


def _distill(s):
    c = s["case"]
    d, m, log_l = _scaled(s)
    logp, stats = _teacher(s)
    logq = d.gather(1, s["ids"].long().clamp(0, c["v"] - 1)) - log_l[:, None]
    terms = torch.where(logp > -torch.inf, logp.exp() * (logp - logq), 0)
    return dict(loss=terms.sum(-1), stats=torch.cat([m[:, None], log_l[:, None], stats], -1))


def _distill_bwd(s):
    c = s["case"]
    p = _teacher(s)[0].exp()
    dz = p.sum(-1, keepdim=True) * _log_q(s).exp()
    dz.scatter_add_(1, s["ids"].long().clamp(0, c["v"] - 1), -p)
    dz = dz * s["d_loss"][:, None]
    if s["scale"] is not None:
        dz = dz * s["scale"][:, None]
    return dict(d_logits=dz.to(s["logits"].dtype))


# ---------------------------------------------------------------------------
# the definition in 64 bits, a number of rows at a time

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("add_norm"):
        return _exact_norm(s)
    step = max(1, (1 << 26) // case["v"])
    parts = [_exact_rows(s, slice(a, min(a + step, case["t"]))) for a in range(0, case["t"], step)]
    return {n: None if parts[0][n] is None else torch.cat([p[n] for p in parts]) for n in parts[0]}


def _exact_norm(s):
    c = s["case"]
    w = s["w"].double().requires_grad_()
    if c["op"] == "add_norm_bwd":
        h = s["h"].double().requires_grad_()
        y = h / (h.pow(2).sum(-1, keepdim=True) / c["w"] + EPS).sqrt() * w
        dh, dw = torch.autograd.grad(y, (h, w), s["dy"].double())
        if c["add"]:
            dh = dh + s["d_res"].double()
        return dict(dx=dh, d_residual=dh if c["add"] and s["h"].dtype != s["dy"].dtype else None, dw=dw)
    h = s["x"].double()
    total = h + s["residual"].double() if c["add"] else h
    if c["add"]:
        h = total.to(s["residual"].dtype).double()
    y = h / (h.pow(2).sum(-1, keepdim=True) / c["w"] + EPS).sqrt() * w.detach()
    out = dict(h=h if c["add"] else None, y=y if c["y"] else None, y8=None, y_scale=None)
    if c["group"] >= 0:
        z = y.reshape(c["t"], -1, c["group"] or c["w"])
        scale = torch.maximum(z.abs().max(-1).values, torch.tensor(2.0 ** -100, device=DEV, dtype=torch.float64)) / 448
        u = (z / scale[..., None]).reshape(c["t"], c["w"])
        # e4m3: three bits of fraction, down to steps of 2^-9; half to even
        unit = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))) - 3)
        out["y8"], out["y_scale"] = (u / unit).round() * unit, scale
    return out


def _exact_rows(s, at):
    c = s["case"]
    x = s["logits"][at].double()
    t, v = x.shape
    scale = torch.ones((t, 1), dtype=torch.float64, device=DEV) if s["scale"] is None else s["scale"][at].double()[:, None]
    z = x * scale
    lse = torch.logsumexp(z, -1, keepdim=True)
    logq = z - lse
    q = logq.exp()
    stats = torch.cat([x.max(-1, keepdim=True).values, lse - x.max(-1, keepdim=True).values * scale], -1)
    if c["op"].startswith("logprobs"):
        target = s["target"][at].long()
        there = (target >= 0) & (target < v)
        onehot_at = target.clamp(0, v - 1)[:, None]
        entropy = torch.special.entr(q).sum(-1)
        if c["op"] == "logprobs":
            out = dict(logprobs=torch.where(there, logq.gather(1, onehot_at)[:, 0], 0.0), entropy=torch.where(there, entropy, 0.0),
                       stats=torch.where(there[:, None], stats, 0.0), top_ids=None, top_logprobs=None)
            if c["top"]:
                # by the logit, then by the index: the k best one after the other
                left, ids = x.clone(), []
                for _ in range(c["top"]):
                    best = left.max(-1, keepdim=True).values
                    i = (left == best).to(torch.uint8).argmax(-1, keepdim=True)
                    left.scatter_(1, i, -torch.inf)
                    ids.append(i)
                ids = torch.cat(ids, 1)
                out["top_ids"] = torch.where(there[:, None], ids, -1).to(torch.int32) if c["top"] <= v // 4 else None
                out["top_logprobs"] = torch.where(there[:, None], logq.gather(1, ids), 0.0) if c["top"] <= v // 4 else None
            return out
        g, gh = s["d_logprobs"][at].double()[:, None], s["d_entropy"][at].double()[:, None]
        dz = -g * q - gh * torch.where(q > 0, q * (logq + entropy[:, None]), 0.0)
        dz.scatter_add_(1, onehot_at, g)
        return dict(d_logits=torch.where(there[:, None], dz * scale, 0.0))
    ids, values = s["ids"][at].long(), s["values"][at].double()
    there = (ids >= 0) & (ids < v)
    values = torch.where(there, values, -torch.inf)
    some = there.any(-1, keepdim=True)
    most = torch.where(some, values.max(-1, keepdim=True).values, 0.0)
    log_p = values
    teacher = torch.zeros((t, 2), dtype=torch.float64, device=DEV)
    if not c["logp"]:
        total = torch.where(some, torch.logsumexp((values - most) * scale, -1, keepdim=True), 0.0)
        log_p = (values - most) * scale - total
        teacher = torch.cat([most, total], -1)
    p = log_p.exp()
    if c["op"] == "distill":
        terms = torch.where(p > 0, p * (log_p - logq.gather(1, ids.clamp(0, v - 1))), 0.0)
        return dict(loss=terms.sum(-1), stats=torch.cat([stats, teacher], -1))
    dz = q * p.sum(-1, keepdim=True)
    dz.scatter_add_(1, ids.clamp(0, v - 1), -p)
    return dict(d_logits=dz * scale * s["d_loss"][at].double()[:, None])
