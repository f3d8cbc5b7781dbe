"""Cases of the dense MoE operators: routing, grouped products, 8-bit products, block norms.

`run` computes a case's operator in its plain form (elementary torch operations in 32 or 64
bits), or, where `own` is true, by the framework's call.  Shapes are those of the
repository's blocks (hidden 2048 x 768 channels x 128 experts top-8, hidden 4096 x 1536
channels, and the tiny 256 x 512 x 8 experts) and ranges around them.
"""
import math

import torch

own = False

FLT_MAX = torch.finfo(torch.float32).max


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 64 sequences: the plan of a small batch, launch latency counts
        {"name": "route_decode_64", "op": "route", "tokens": 64, "experts": 128, "top_e": 8,
         "renorm": True, "bf16": False, "padded": False},
        # a batch of prompts padded to one length: masked tokens take no part
        {"name": "route_prompt_8192", "op": "route", "tokens": 8192, "experts": 128, "top_e": 8,
         "renorm": True, "bf16": False, "padded": True},
        # a single token through its 8 experts' gate and up rows: pure weight streaming
        {"name": "swiglu_token_1", "op": "swiglu", "tokens": 1, "d": 2048, "inter": 768,
         "experts": 128, "top_e": 8, "records": True},
        # a prompt of 4096 tokens, gate and up straight from the packed channel records
        {"name": "swiglu_prompt_4096", "op": "swiglu", "tokens": 4096, "d": 2048, "inter": 768,
         "experts": 128, "top_e": 8, "records": True},
        # the same prompt's down product; the records hold the down columns channel by channel
        {"name": "down_prompt_4096", "op": "down", "tokens": 4096, "d": 2048, "inter": 768,
         "experts": 128, "top_e": 8, "records": True, "f32": False, "spare": 0},
        # the large block at a decode batch: nearly every expert is used by a token or two
        {"name": "down_large_33", "op": "down", "tokens": 33, "d": 4096, "inter": 1536,
         "experts": 128, "top_e": 8, "records": True, "f32": False, "spare": 0},
        # the large block on a prompt of odd length, weights in model layout [E][2][I][d]
        {"name": "swiglu_large_2039", "op": "swiglu", "tokens": 2039, "d": 4096, "inter": 1536,
         "experts": 128, "top_e": 8, "records": False},
        # an 8-bit projection for one token: quantise, then stream the weight
        {"name": "int8_token_1", "op": "int8", "tokens": 1, "k": 4096, "n": 4096, "experts": 0,
         "top_e": 0, "swiglu": False},
        # an 8-bit projection of a long prompt: bound by the matrix units
        {"name": "int8_prompt_8192", "op": "int8", "tokens": 8192, "k": 4096, "n": 4096,
         "experts": 0, "top_e": 0, "swiglu": False},
        # 8-bit experts on a ragged prompt of 1021 tokens: about 64 rows an expert
        {"name": "int8_experts_1021", "op": "int8", "tokens": 1021, "k": 2048, "n": 768,
         "experts": 128, "top_e": 8, "swiglu": True},
        # the glue of one decode step, fp32 residual stream
        {"name": "norm_decode_4", "op": "norm", "tokens": 4, "d": 2048, "h_f32": True,
         "post": True, "gate": "channel", "weights": True},
        # the glue of a prompt, bf16 residual stream, a gate per token
        {"name": "norm_prompt_8192", "op": "norm", "tokens": 8192, "d": 4096, "h_f32": False,
         "post": True, "gate": "token", "weights": True},
    ]


def _log(rng, lo, hi):
    """An integer spread evenly over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_COST = 7e11  # multiply-adds x 2 of the largest listed product, rounded up


def draw(rng):
    op = rng.choice(["route", "swiglu", "down", "int8", "int8", "norm"])
    if op == "route":
        experts = rng.choice([8, 16, 60, 128, 160, 256, 512])
        return {"op": op, "tokens": _log(rng, 1, 8192), "experts": experts,
                "top_e": rng.randint(1, min(16, experts)), "renorm": rng.random() < 0.5,
                "bf16": rng.random() < 0.3, "padded": rng.random() < 0.4}
    if op == "norm":
        return {"op": op, "tokens": _log(rng, 1, 8192), "d": _log(rng, 64, 4096),
                "h_f32": rng.random() < 0.5, "post": rng.random() < 0.6,
                "gate": rng.choice(["none", "channel", "token", "full"]),
                "weights": rng.random() < 0.7}
    if op == "int8" and rng.random() < 0.5:
        return {"op": op, "tokens": _log(rng, 1, 8192), "k": 16 * _log(rng, 4, 256),
                "n": _log(rng, 64, 4096), "experts": 0, "top_e": 0, "swiglu": False}
    experts = rng.choice([1, 8, 16, 60, 128])
    top_e = rng.randint(1, min(8, experts))
    d, inter = 64 * _log(rng, 4, 64), _log(rng, 33, 1536)
    if d > 2048 and inter > 768 and experts > 64:
        d = 2048
    tokens = _log(rng, 1, 8192)
    while 4.0 * tokens * top_e * d * inter > _COST:
        tokens = tokens // 2 + 1
    if op == "int8":
        return {"op": op, "tokens": tokens, "k": d, "n": inter, "experts": experts,
                "top_e": top_e, "swiglu": rng.random() < 0.5}
    if op == "swiglu":
        return {"op": op, "tokens": tokens, "d": d, "inter": inter, "experts": experts,
                "top_e": top_e, "records": rng.random() < 0.5}
    records = rng.random() < 0.6
    return {"op": op, "tokens": tokens, "d": d, "inter": inter if records else (inter + 7) // 8 * 8,
            "experts": experts, "top_e": top_e, "records": records, "f32": rng.random() < 0.3,
            "spare": rng.choice([0, 0, 7, 100])}


def _used(c):
    """Experts that a batch of uniformly routed tokens uses, on average."""
    e = c["experts"]
    return e * (1.0 - (1.0 - c["top_e"] / e) ** c["tokens"])


def work(c):
    t = c["tokens"]
    if c["op"] == "route":
        e, k = c["experts"], c["top_e"]
        return {"bytes": t * e * (2 if c["bf16"] else 4) + 16 * t * k + 4 * (e + 1), "flops": 3 * t * e}
    if c["op"] == "norm":
        d, hs = c["d"], 4 if c["h_f32"] else 2
        gate = {"none": 0, "channel": d, "token": t, "full": t * d}[c["gate"]]
        weights = 2 * d * (2 if c["post"] else 1) if c["weights"] else 0
        return {"bytes": t * d * (2 * hs + 4) + 2 * gate + weights, "flops": 10 * t * d}
    if c["op"] == "int8":
        k, n = c["k"], c["n"]
        if not c["experts"]:
            return {"bytes": 2 * t * k + n * k + 4 * n + 2 * t * n, "flops": 2.0 * t * n * k}
        m, r = (2 if c["swiglu"] else 1), t * c["top_e"]
        return {"bytes": 2 * t * k + _used(c) * m * n * (k + 4) + 4 * r + 2 * r * n,
                "flops": 2.0 * m * r * n * k}
    d, i, r = c["d"], c["inter"], t * c["top_e"]
    if c["op"] == "swiglu":
        return {"bytes": 2 * t * d + 4 * r + _used(c) * 4 * i * d + 2 * r * i, "flops": 4.0 * r * i * d}
    return {"bytes": 2 * r * i + _used(c) * 2 * i * d + r * d * (4 if c["f32"] else 2),
            "flops": 2.0 * r * i * d}


# ------------------------------------------------------------------ inputs

def _plan(c, g):
    """A routing as a router's mild preferences give it: token of every row, rows sorted by
    expert; the experts' offsets; for the padded plain products the used experts and, for
    each, its rows (filled up with the row behind the last)."""
    t, e, k = c["tokens"], c["experts"], c["top_e"]
    logits = torch.randn(t, e, generator=g, device="cuda") + 0.5 * torch.randn(e, generator=g, device="cuda")
    ids = torch.topk(logits, k, dim=1).indices
    order = torch.argsort(ids.reshape(-1), stable=True)
    counts = torch.bincount(ids.reshape(-1), minlength=e)
    offsets = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    act = torch.nonzero(counts).reshape(-1)
    col = torch.arange(int(counts.max()), device="cuda")
    slot = torch.where(col[None] < counts[act, None], offsets[act].long()[:, None] + col[None], t * k)
    return {"offsets": offsets, "rows": (order // k).to(torch.int32), "act": act, "slot": slot}


def _int8_weight(shape, g):
    w = torch.randn(shape, generator=g, device="cuda") * 0.02
    s = w.abs().amax(-1) / 127.0
    return torch.round(w / s[..., None]).to(torch.int8), s


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = c["tokens"]
    rnd = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    s = {"op": c["op"], "case": c}
    if c["op"] == "route":
        x = rnd(t, c["experts"]) * 0.9
        s["logits"] = x.bfloat16() if c["bf16"] else x
        s["mask"] = None
        if c["padded"]:  # prompts of one batch, each padded to an eighth of the tokens
            span = max(1, t // 8)
            length = torch.randint(1, span + 1, (t // span + 1,), generator=g, device="cuda")
            i = torch.arange(t, device="cuda")
            s["mask"] = (i % span) < length[i // span]
        return s
    if c["op"] == "norm":
        d = c["d"]
        h, y = rnd(t, d) * 4.0, rnd(t, d)
        s["h"], s["y"] = (h if c["h_f32"] else h.bfloat16()), y.bfloat16()
        s["h_out"], s["x"] = torch.empty_like(s["h"]), torch.empty_like(s["y"])
        shape = {"none": None, "channel": (d,), "token": (t, 1), "full": (t, d)}[c["gate"]]
        s["gate"] = None if shape is None else torch.sigmoid(rnd(*shape)).bfloat16()
        s["pre"] = (1 + 0.1 * rnd(d)).bfloat16() if c["weights"] else None
        s["post"] = (1 + 0.1 * rnd(d)).bfloat16() if c["weights"] and c["post"] else None
        return s
    if c["op"] == "int8":
        s["x"] = rnd(t, c["k"]).bfloat16()
        if not c["experts"]:
            s["w"], s["ws"] = _int8_weight((c["n"], c["k"]), g)
            return s
        shape = (c["experts"],) + ((2,) if c["swiglu"] else ()) + (c["n"], c["k"])
        s["w"], s["ws"] = _int8_weight(shape, g)
        s.update(_plan(c, g))
        return s
    e, i, d = c["experts"], c["inter"], c["d"]
    s.update(_plan(c, g))
    r = t * c["top_e"]
    if c["records"]:  # channel records [E][I][gate row | up row | down column]
        rec = (rnd(e, i, 3 * d) * 0.02).bfloat16().view(e, i, 3, d)
        w = rec[:, :, :2].permute(0, 2, 1, 3) if c["op"] == "swiglu" else rec[:, :, 2].transpose(1, 2)
    else:
        w = (rnd(*((e, 2, i, d) if c["op"] == "swiglu" else (e, d, i))) * 0.02).bfloat16()
    s["w"] = w
    if c["op"] == "swiglu":
        s["x"] = rnd(t, d).bfloat16()
    else:  # hidden rows on a pitch of whole 16-byte pieces, a few spare rows behind the last
        s["x"] = (rnd(r, (i + 7) // 8 * 8) * 0.5).bfloat16()[:, :i]
        s["out"] = torch.zeros((r + c["spare"], d), device="cuda",
                               dtype=torch.float32 if c["f32"] else torch.bfloat16)
    return s


# ------------------------------------------------------------------ plain forms

def _route(s):
    c, l = s["case"], s["logits"].float()
    t, e = l.shape
    k = c["top_e"]
    ok = l > -math.inf  # false for NaN too
    if s["mask"] is not None:
        ok = ok & s["mask"][:, None]
    l = torch.where(ok, l.clamp(max=FLT_MAX), -math.inf)
    top, idx = torch.sort(l, dim=1, descending=True, stable=True)
    top, idx = top[:, :k], idx[:, :k]
    kept = top > -math.inf
    big = torch.where(kept[:, :1], top[:, :1], 0.0)
    p = torch.exp(top - big)
    den = p.sum(1) if c["renorm"] else torch.exp(l - big).sum(1)
    wts = torch.where(kept, p / torch.where(den > 0, den, 1.0)[:, None], 0.0)
    ids = torch.where(kept, idx, -1)
    flat = torch.where(ids < 0, e, ids).reshape(-1)
    order = torch.argsort(flat, stable=True)
    srt = flat[order]
    offsets = torch.searchsorted(srt, torch.arange(e + 1, device=l.device))
    rows = torch.where(srt < e, order // k, -1)
    pos = torch.empty_like(order)
    pos[order] = torch.where(srt < e, torch.arange(t * k, device=l.device), -1)
    i32 = torch.int32
    return {"ids": ids.to(i32), "weights": wts, "offsets": offsets.to(i32), "rows": rows.to(i32),
            "pos": pos.view(t, k).to(i32)}


def _padded_product(x, w, s, dtype):
    """The rows of each used expert, padded to one length, times its weight [n][k]."""
    xp = torch.cat([x, x.new_zeros(1, x.shape[1])])[s["slot"]].to(dtype)
    return torch.matmul(xp, w[s["act"]].to(dtype).transpose(1, 2))


def _unpad(y, s, rows):
    out = y.new_zeros((rows + 1, y.shape[2]))
    out[s["slot"].reshape(-1)] = y.reshape(-1, y.shape[2])
    return out[:rows]


def _silu_mul(g, u):
    return g / (1 + torch.exp(-g)) * u


def _swiglu(s):
    x, w, r = s["x"][s["rows"].long()], s["w"], s["rows"].numel()
    h = _silu_mul(_padded_product(x, w[:, 0], s, torch.float32), _padded_product(x, w[:, 1], s, torch.float32))
    return _unpad(h, s, r).bfloat16()


def _down(s):
    r = s["rows"].numel()
    y = _unpad(_padded_product(s["x"], s["w"], s, torch.float32), s, r)
    return torch.cat([y, y.new_zeros(s["out"].shape[0] - r, y.shape[1])]).to(s["out"].dtype)


def _quantize(x):
    x = x.float()
    big = x.abs().amax(1)
    q = torch.round(x * torch.where(big > 0, 127.0 / big, 0.0)[:, None])
    return q, big / 127.0


def _int8(s):
    q, qs = _quantize(s["x"])
    w, ws = s["w"], s["ws"]
    # the integer sums pass 2^24: 64 bits hold them exactly
    if not s["case"]["experts"]:
        acc = torch.matmul(q.double(), w.double().t())
        return (acc.float() * qs[:, None] * ws[None]).bfloat16()
    rows = s["rows"].long()
    r, q, qs = rows.numel(), q[rows], qs[rows]
    qp = torch.cat([qs, qs.new_zeros(1)])[s["slot"]][..., None]
    part = lambda w, ws: _padded_product(q, w, s, torch.float64).float() * qp * ws[s["act"]][:, None]  # noqa: E731
    y = _silu_mul(part(w[:, 0], ws[:, 0]), part(w[:, 1], ws[:, 1])) if s["case"]["swiglu"] else part(w, ws)
    return _unpad(y, s, r).bfloat16()


EPS, SKIP, RESIDUAL = 1e-6, 1.0, 0.22


def _norm(s):
    rms = lambda v: v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)  # noqa: E731
    b = s["y"].float()
    if s["case"]["post"]:
        b = rms(b)
        if s["post"] is not None:
            b = b * s["post"].float()
    if s["gate"] is not None:
        b = b * s["gate"].float()
    h = SKIP * s["h"].float() + RESIDUAL * b
    x = rms(h)
    if s["pre"] is not None:
        x = x * s["pre"].float()
    return {"h": h.to(s["h"].dtype), "x": x.bfloat16()}


_PLAIN = {"route": _route, "swiglu": _swiglu, "down": _down, "int8": _int8, "norm": _norm}


# ------------------------------------------------------------------ the framework's calls

def _own(s):
    import token_top_expert_b200 as msb
    c = s["case"]
    if s["op"] == "route":
        r = msb.route(s["logits"], c["top_e"], renorm=c["renorm"], mask=s["mask"])
        return {"ids": r.ids, "weights": r.weights, "offsets": r.offsets, "rows": r.rows, "pos": r.pos}
    if s["op"] == "swiglu":
        return msb.grouped_swiglu(s["x"], s["w"], s["offsets"], rows=s["rows"])
    if s["op"] == "down":
        return msb.grouped_matmul(s["x"], s["w"], s["offsets"], out=s["out"])
    if s["op"] == "int8":
        if not c["experts"]:
            return msb.linear_int8(s["x"], s["w"], s["ws"])
        f = msb.swiglu_int8 if c["swiglu"] else msb.linear_int8
        return f(s["x"], s["w"], s["ws"], offsets=s["offsets"], rows=s["rows"])
    h, x = msb.block_norm(s["h"], s["y"], s["x"], h_out=s["h_out"], pre_weight=s["pre"],
                          post_norm=c["post"], post_weight=s["post"], gate=s["gate"],
                          skip_scale=SKIP, residual_scale=RESIDUAL, eps=EPS)
    return {"h": h, "x": x}


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ------------------------------------------------------------------ 64-bit definitions

def exact(c, seed):
    s = prepare(c, seed)
    f64 = torch.float64
    if c["op"] == "route":
        l = s["logits"].to(f64)
        if s["mask"] is not None:
            l = l.masked_fill(~s["mask"][:, None], -math.inf)
        p = torch.softmax(l, 1).nan_to_num(0.0)
        top = torch.topk(p, c["top_e"], dim=1).values
        if c["renorm"]:
            top = (top / top.sum(1, keepdim=True)).nan_to_num(0.0)
        return {"ids": None, "weights": top, "offsets": None, "rows": None, "pos": None}
    if c["op"] == "norm":
        y, h = s["y"].to(f64), s["h"].to(f64)
        if c["post"]:
            y = y * torch.rsqrt(y.square().mean(1, keepdim=True) + EPS)
            y = y if s["post"] is None else y * s["post"].to(f64)
        h = SKIP * h + RESIDUAL * (y if s["gate"] is None else y * s["gate"].to(f64))
        x = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
        return {"h": h, "x": x if s["pre"] is None else x * s["pre"].to(f64)}
    if c["op"] == "int8":
        x = s["x"].to(f64)
        big = x.abs().amax(1, keepdim=True)
        x = torch.round(x * 127.0 / big.clamp(min=1e-300)) * (big / 127.0)
        if not c["experts"]:
            return x @ (s["w"].to(f64) * s["ws"].to(f64)[:, None]).t()
        x, w = x[s["rows"].long()], lambda e: s["w"][e].to(f64) * s["ws"][e].to(f64)[..., None]
    else:
        x = s["x"].to(f64)
        if c["op"] == "swiglu":
            x = x[s["rows"].long()]
        w = lambda e: s["w"][e].to(f64)  # noqa: E731
    gated = c["op"] == "swiglu" or (c["op"] == "int8" and c["swiglu"])
    n = c["d"] if c["op"] == "down" else c["inter"] if c["op"] == "swiglu" else c["n"]
    out = torch.zeros((s["out"].shape[0] if c["op"] == "down" else x.shape[0], n), dtype=f64, device="cuda")
    at = s["offsets"].tolist()
    for e, (lo, hi) in enumerate(zip(at, at[1:])):
        if lo < hi:
            we = w(e)
            out[lo:hi] = (torch.nn.functional.silu(x[lo:hi] @ we[0].t()) * (x[lo:hi] @ we[1].t()) if gated
                          else x[lo:hi] @ we.t())
    return out
