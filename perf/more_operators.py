"""Timing cases of the token-embedding, norm and routing operators.

The operators stand around a layer of experts: tokens are looked up in a table,
the residual stream is normalised on its way into the layer (in 8 bits for its
products), and a router chooses each token's experts.

  look       rows of a table by token, scaled
  lookgrad   the table's gradient: the tokens' gradients summed by row
  norm       residual added and the sum normalised by its root mean square, in the
             rows' own type or in e4m3 with a scale for each 128 columns
  normgrad   the norm's gradients, of the rows and of the weight
  route      experts by score, bias and group, and their weights
  routegrad  the gradient of the router's logits

Every case runs in a plain form (elementary torch operations, `own` false) or
through this framework's entry points (`own` true), on the same state.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16,
          "i32": torch.int32, "i64": torch.int64}
BLOCK = 128          # columns that share a scale
E4M3_MAX = 448.0     # largest finite e4m3 value
TINY = 2.0 ** -126   # smallest scale
EPS = 1e-6


def _bytes(dtype):
    return DTYPES[dtype].itemsize


def _blocks(n):
    return -(-n // BLOCK)


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # the tokens of four sequences being answered
        dict(name="look_token", kind="look", tokens=4, rows=50_000, width=1024, dtype="bf16",
             ids="i64", drop=0.0, scale=32.0),
        # a large training batch from a vocabulary of 131072
        dict(name="look_large", kind="look", tokens=131072, rows=131072, width=2048, dtype="bf16",
             ids="i32", drop=0.0, scale=1.0),
        # a small training batch whose sizes divide by nothing, with padding
        dict(name="lookgrad_ragged", kind="lookgrad", tokens=4097, rows=5003, width=1001,
             dtype="f16", out="f16", ids="i64", drop=0.1, scale=1.5),
        # a large training batch: a few tokens fill much of it, most rows get none
        dict(name="lookgrad_large", kind="lookgrad", tokens=65536, rows=131072, width=2048,
             dtype="bf16", out="bf16", ids="i32", drop=0.0, scale=1.0),
        # tokens being answered: the residual's sum, and 8 bits for the next product
        dict(name="norm_token", kind="norm", rows=4, width=1024, dtype="bf16", residual=True,
             out="fp8"),
        # an ordinary batch of odd width
        dict(name="norm_ragged", kind="norm", rows=4097, width=1001, dtype="f16", residual=False,
             out="f16"),
        # a large batch on its way into an 8-bit expert layer
        dict(name="norm_large", kind="norm", rows=65536, width=2048, dtype="bf16", residual=True,
             out="fp8"),
        # the same batch's training step
        dict(name="normgrad_large", kind="normgrad", rows=65536, width=2048, dtype="bf16",
             residual=True),
        # a few tokens being answered: two of sixteen experts
        dict(name="route_token", kind="route", tokens=4, experts=16, k=2, groups=1, top_groups=1,
             best=1, score="softmax", bias=False, renorm=True, scale=1.0, dtype="f32", masked=0.0),
        # a batch of 4096 bags; some experts closed to some tokens
        dict(name="route_batch", kind="route", tokens=4096, experts=64, k=4, groups=1,
             top_groups=1, best=1, score="softmax", bias=False, renorm=False, scale=1.0,
             dtype="bf16", masked=0.1),
        # a large batch: eight of 256 experts in four of eight groups, balanced by a bias
        dict(name="route_large", kind="route", tokens=65536, experts=256, k=8, groups=8,
             top_groups=4, best=2, score="sigmoid", bias=True, renorm=True, scale=2.5,
             dtype="f32", masked=0.0),
        # the same batch's training step
        dict(name="routegrad_large", kind="routegrad", tokens=65536, experts=256, k=8, groups=8,
             top_groups=4, best=2, score="sigmoid", bias=True, renorm=True, scale=2.5,
             dtype="f32", masked=0.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _some_width(rng, lo, hi):
    w = _log(rng, lo, hi)
    return max(lo, w - w % rng.choice([1, 8, 64]))


def draw(rng):
    kind = rng.choice(["look", "lookgrad", "norm", "normgrad", "route", "routegrad"])
    most = work(next(c for c in listed() if c["name"] == kind + "_large"))
    while True:
        dtype = rng.choice(["f16", "bf16", "f32"])
        if kind in ("look", "lookgrad"):
            c = dict(kind=kind, tokens=_log(rng, 1, 131072), rows=_log(rng, 1, 262144),
                     width=_some_width(rng, 8, 4096), dtype=dtype, ids=rng.choice(["i32", "i64"]),
                     drop=rng.choice([0.0, 0.05, 0.5]), scale=rng.choice([1.0, 0.5, 45.25]))
            if kind == "lookgrad":
                c["out"] = rng.choice([dtype, "f32"])
        elif kind == "norm":
            c = dict(kind=kind, rows=_log(rng, 1, 131072), width=_some_width(rng, 8, 8192),
                     dtype=dtype, residual=rng.random() < 0.5, out=rng.choice([dtype, "fp8"]))
        elif kind == "normgrad":
            c = dict(kind=kind, rows=_log(rng, 1, 131072), width=_some_width(rng, 8, 8192),
                     dtype=dtype, residual=rng.random() < 0.5)
        else:
            groups = rng.choice([1, 1, 2, 4, 8])
            size = _log(rng, 2, 512 // groups)
            top_groups = rng.randint(1, groups)
            bias, score = rng.random() < 0.5, rng.choice(["softmax", "sigmoid"])
            c = dict(kind=kind, tokens=_log(rng, 1, 131072), experts=groups * size,
                     k=rng.randint(1, min(8, top_groups * size)), groups=groups,
                     top_groups=top_groups, best=rng.choice([1, 2]), score=score, bias=bias,
                     renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]), dtype=dtype,
                     masked=rng.choice([0.0, 0.0, 0.2]))
        w = work(c)
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]:
            return c


def _distinct(tokens, rows):
    """Expected number of different rows among tokens of _token_ids."""
    r = torch.arange(1, rows + 1, dtype=torch.float64)
    p = torch.log1p(1 / r) / math.log(rows + 1)
    return float((1 - torch.exp(tokens * torch.log1p(-p.clamp(max=1 - 1e-12)))).sum())


def work(case):
    """Bytes read once and written once, and operations, of one pass."""
    c, kind = case, case["kind"]
    if kind in ("look", "lookgrad"):
        N, H, s, kept = c["tokens"], c["width"], _bytes(c["dtype"]), c["tokens"] * (1 - c["drop"])
        if kind == "look":
            return {"bytes": N * _bytes(c["ids"]) + (_distinct(kept, c["rows"]) + N) * H * s,
                    "flops": N * H}
        return {"bytes": N * _bytes(c["ids"]) + kept * H * s + c["rows"] * H * _bytes(c["out"]),
                "flops": 2 * kept * H}
    if kind == "norm":
        R, H, s = c["rows"], c["width"], _bytes(c["dtype"])
        out = H + 4 * _blocks(H) if c["out"] == "fp8" else H * s
        return {"bytes": R * ((3 if c["residual"] else 1) * H * s + out) + H * s,
                "flops": R * H * (6 if c["out"] == "fp8" else 5)}
    if kind == "normgrad":
        R, H, s = c["rows"], c["width"], _bytes(c["dtype"])
        return {"bytes": R * H * s * (4 if c["residual"] else 3) + H * (s + 4), "flops": 12 * R * H}
    N, E, k, s = c["tokens"], c["experts"], c["k"], _bytes(c["dtype"])
    if kind == "route":
        return {"bytes": N * E * s + 8 * N * k + (4 * E if c["bias"] else 0), "flops": 8 * N * E}
    # only softmax weights that are not normalised again have a gradient in every logit
    read = E if c["score"] == "softmax" and not c["renorm"] else k
    return {"bytes": N * (read * s + 8 * k + E * s), "flops": N * (8 * read + 8 * k)}


# --------------------------------------------------------------- the inputs

def _rand(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _fill(g, rows, cols, dtype):
    out = torch.empty(rows, cols, dtype=DTYPES[dtype], device="cuda")
    step = max(1, (1 << 27) // max(cols, 1))
    for r in range(0, rows, step):
        out[r:r + step] = _randn(g, min(step, rows - r), cols)
    return out


def _token_ids(c, g):
    """Tokens by Zipf's law, ranks scattered over the rows; -1 where there is padding."""
    u = torch.rand(c["tokens"], generator=g, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(c["rows"] + 1)).long() - 1).clamp(0, c["rows"] - 1)
    ids = (rank * 7919 + 13) % c["rows"]
    gone = _uniform(g, c["tokens"]) < c["drop"]
    return ids.masked_fill(gone, -1).to(DTYPES[c["ids"]])


def _logits(c, g):
    """A router's answers: some experts liked more than others, some closed (-inf)."""
    x = 1.5 * _randn(g, c["tokens"], c["experts"]) + 0.5 * _randn(g, c["experts"])
    closed = _uniform(g, c["tokens"], c["experts"]) < c["masked"]
    return x.to(DTYPES[c["dtype"]]).masked_fill(closed, float("-inf"))


def prepare(case, seed):
    c, g, kind = case, _rand(seed), case["kind"]
    s = {"kind": kind, "case": c}
    if kind == "look":
        return dict(s, ids=_token_ids(c, g), table=_fill(g, c["rows"], c["width"], c["dtype"]))
    if kind == "lookgrad":
        return dict(s, ids=_token_ids(c, g), dout=_fill(g, c["tokens"], c["width"], c["dtype"]))
    if kind in ("norm", "normgrad"):
        weight = (1 + 0.1 * _randn(g, c["width"])).to(DTYPES[c["dtype"]])
        s.update(weight=weight, x=_fill(g, c["rows"], c["width"], c["dtype"]),
                 other=_fill(g, c["rows"], c["width"], c["dtype"]) if c["residual"] else None)
        if kind == "normgrad":
            s["dy"] = _fill(g, c["rows"], c["width"], c["dtype"])
        return s
    s["logits"] = _logits(c, g)
    s["bias"] = 0.1 * _randn(g, c["experts"]) if c["bias"] else None
    if kind == "routegrad":  # the forward pass has left its choice
        s["ids"] = _route_plain(s)["ids"]
        s["dw"] = _randn(g, c["tokens"], c["k"])
    return s


# ----------------------------------------------------------- the plain forms

def _look_plain(s):
    ids, rows = s["ids"], s["table"].shape[0]
    on = (ids >= 0) & (ids < rows)
    out = s["table"][ids.clamp(0, rows - 1)].float() * s["case"]["scale"]
    return torch.where(on[:, None], out, 0.0).to(s["table"].dtype)


def _lookgrad_plain(s):
    c, ids = s["case"], s["ids"]
    kept = ((ids >= 0) & (ids < c["rows"])).nonzero()[:, 0]
    grad = torch.zeros(c["rows"], c["width"], device="cuda")
    grad.index_add_(0, ids[kept], s["dout"][kept].float())
    return (grad * c["scale"]).to(DTYPES[c["out"]])


def _quantize_plain(y):
    rows, cols = y.shape
    pad = torch.nn.functional.pad(y, (0, -cols % BLOCK)).view(rows, -1, BLOCK)
    scale = (pad.abs().amax(2) / E4M3_MAX).clamp_min(TINY)
    q = (pad / scale[..., None]).view(rows, -1)[:, :cols].to(torch.float8_e4m3fn)
    return q.contiguous(), scale


def _norm_plain(s):
    x, out = s["x"], {}
    if s["other"] is not None:
        x = out["h"] = (x.float() + s["other"].float()).to(x.dtype)
    h = x.float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["weight"].float()
    if s["case"]["out"] == "fp8":
        out["q"], out["scale"] = _quantize_plain(y)
    else:
        out["y"] = y.to(x.dtype)
    return out


def _normgrad_plain(s):
    h, dy, w = s["x"].float(), s["dy"].float(), s["weight"].float()
    r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    unit, dunit = h * r, dy * w
    dx = r * (dunit - unit * (dunit * unit).mean(1, keepdim=True))
    if s["other"] is not None:
        dx = dx + s["other"].float()
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * unit).sum(0)}


def _scores_plain(logits, score):
    """Scores in the logits' precision; zeros in rows where every expert is closed."""
    if score == "sigmoid":
        return torch.sigmoid(logits)
    top = logits.amax(1, keepdim=True).clamp_min(torch.finfo(logits.dtype).min)
    e = torch.exp(logits - top)
    return e / e.sum(1, keepdim=True).clamp_min(torch.finfo(logits.dtype).tiny)


def _route_plain(s):
    c, logits = s["case"], s["logits"]
    N, E = logits.shape
    # the choice is made in 64 bits: experts next to a border must not change places
    choice = _scores_plain(logits.double(), c["score"])
    if s["bias"] is not None:
        choice = choice + s["bias"].double()
    choice = choice.masked_fill(logits == float("-inf"), float("-inf"))
    if c["groups"] > 1:
        best = choice.view(N, c["groups"], -1).sort(2, descending=True).values[:, :, :c["best"]]
        some = best[:, :, 0] > float("-inf")
        best = best.masked_fill(best == float("-inf"), 0.0).sum(2).masked_fill(~some, float("-inf"))
        rank = best.sort(dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        chosen = torch.zeros_like(best, dtype=torch.bool).scatter_(1, rank, True)
        chosen = chosen[:, :, None].expand(-1, -1, E // c["groups"]).reshape(N, E)
        choice = choice.masked_fill(~chosen, float("-inf"))
    value, ids = choice.sort(dim=1, descending=True, stable=True)
    value, ids = value[:, :c["k"]], ids[:, :c["k"]]
    on = value > float("-inf")
    w = torch.where(on, _scores_plain(logits.float(), c["score"]).gather(1, ids), 0.0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-30)
    return {"ids": torch.where(on, ids, -1).to(torch.int32), "weights": w * c["scale"]}


def _routegrad_plain(s):
    c, ids = s["case"], s["ids"].long()
    on, at = ids >= 0, ids.clamp_min(0)
    scores = _scores_plain(s["logits"].float(), c["score"])
    p = torch.where(on, scores.gather(1, at), 0.0)
    d = torch.where(on, s["dw"] * c["scale"], 0.0)
    if c["renorm"]:
        total = p.sum(1, keepdim=True).clamp_min(1e-30)
        d = (d - (d * p).sum(1, keepdim=True) / total) / total
        if c["score"] == "softmax":  # the scores' own sum leaves no trace
            d, p = d * p, None
    if c["score"] == "sigmoid":
        d, p = d * p * (1 - p), None
    grad = torch.zeros_like(scores).scatter_add_(1, at, torch.where(on, d, 0.0))
    if p is not None:
        grad = scores * (grad - (d * p).sum(1, keepdim=True))
    return grad.to(s["logits"].dtype)


_PLAIN = {"look": _look_plain, "lookgrad": _lookgrad_plain, "norm": _norm_plain,
          "normgrad": _normgrad_plain, "route": _route_plain, "routegrad": _routegrad_plain}


# ------------------------------------------------- the framework's operators

def _run_own(s):
    import table_embedding_bag_gb300 as tbe
    c, kind = s["case"], s["kind"]
    if kind == "look":
        return tbe.tbe_embed(s["table"], s["ids"], c["scale"])
    if kind == "lookgrad":
        return tbe.tbe_embed_backward(s["dout"], s["ids"], c["rows"], c["scale"],
                                      out_dtype=DTYPES[c["out"]])
    if kind == "norm":
        names = ("q", "scale") if c["out"] == "fp8" else ("y",)
        call = tbe.tbe_rms_norm_fp8 if c["out"] == "fp8" else tbe.tbe_rms_norm
        got = call(s["x"], s["weight"], residual=s["other"], eps=EPS)
        got = got if isinstance(got, tuple) else (got,)
        return dict(zip(names + ("h",), got))
    if kind == "normgrad":
        dx, dw = tbe.tbe_rms_norm_backward(s["dy"], s["x"], s["weight"], grad_h=s["other"],
                                           eps=EPS)
        return {"dx": dx, "dw": dw}
    if kind == "route":
        ids, weights = tbe.tbe_expert_route(
            s["logits"], c["k"], bias=s["bias"], score=c["score"], groups=c["groups"],
            top_groups=c["top_groups"], group_best=c["best"], renormalize=c["renorm"],
            scale=c["scale"])
        return {"ids": ids, "weights": weights}
    return tbe.tbe_expert_route_backward(s["dw"], s["logits"], s["ids"], score=c["score"],
                                         renormalize=c["renorm"], scale=c["scale"])


def run(state):
    return _run_own(state) if own else _PLAIN[state["kind"]](state)


# ------------------------------------------------------- the values in 64 bits

def _route_exact(s):
    """Round after round the best expert that is left, in the groups that were taken likewise."""
    c, l = s["case"], s["logits"].double()
    N, E = l.shape
    closed = torch.isneginf(l)
    if c["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-l))
    else:
        score = torch.softmax(l, 1).nan_to_num(0.0)
    choice = score if s["bias"] is None else score + s["bias"].double()
    choice[closed] = -math.inf
    n = torch.arange(N, device="cuda")
    if c["groups"] > 1:
        left, worth = choice.clone(), torch.zeros(N, c["groups"], dtype=torch.float64, device="cuda")
        for i in range(c["best"]):
            v, at = left.view(N, c["groups"], -1).max(2)
            worth = worth + (v if i == 0 else torch.where(v == -math.inf, 0.0, v))
            left.view(N, c["groups"], -1).scatter_(2, at[:, :, None], -math.inf)
        size = E // c["groups"]
        open_ = torch.zeros(N, c["groups"], dtype=torch.bool, device="cuda")
        for _ in range(c["top_groups"]):
            v, at = worth.max(1)
            open_[n, at] |= v > -math.inf
            worth[n, at] = -math.inf
        choice[~open_.repeat_interleave(size, 1)] = -math.inf
    ids, w = [], []
    for _ in range(c["k"]):
        v, at = choice.max(1)
        on = v > -math.inf
        ids.append(torch.where(on, at, -1))
        w.append(torch.where(on, score[n, at], 0.0))
        choice[n, at] = -math.inf
    ids, w = torch.stack(ids, 1), torch.stack(w, 1)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return {"ids": ids.to(torch.int32), "weights": w * c["scale"]}


def _routegrad_exact(s):
    """By automatic differentiation of the weights in the logits."""
    c = s["case"]
    l = s["logits"].double().requires_grad_()
    on = s["ids"] >= 0
    chosen = torch.where(on, l.gather(1, s["ids"].clamp_min(0).long()), -math.inf)
    if c["renorm"]:
        logs = chosen if c["score"] == "softmax" else torch.nn.functional.logsigmoid(chosen)
        w = torch.exp(torch.where(on, logs, 0.0)) * on
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    elif c["score"] == "softmax":
        e = torch.exp(l)
        w = torch.exp(chosen) / e.sum(1, keepdim=True).clamp_min(1e-300)
    else:
        w = torch.sigmoid(chosen)
    loss = (torch.where(on, w, 0.0) * c["scale"] * s["dw"].double()).sum()
    return torch.autograd.grad(loss, l)[0].nan_to_num(0.0)


def exact(case, seed):
    c, s, kind = case, prepare(case, seed), case["kind"]
    if kind == "look":
        out = torch.zeros(c["tokens"], c["width"], dtype=torch.float64, device="cuda")
        kept = (s["ids"] >= 0).nonzero()[:, 0]
        out[kept] = s["table"][s["ids"][kept].long()].double() * c["scale"]
        return out
    if kind == "lookgrad":
        out = torch.zeros(c["rows"] + 1, c["width"], dtype=torch.float64, device="cuda")
        to = torch.where(s["ids"] >= 0, s["ids"], c["rows"]).long()
        step = 1 << 14
        for i in range(0, c["tokens"], step):
            out.index_put_((to[i:i + step],), s["dout"][i:i + step].double(), accumulate=True)
        return out[:-1] * c["scale"]
    if kind == "norm":
        h, out = s["x"].double(), {}
        if s["other"] is not None:  # the sum is held in the rows' type
            out["h"] = h + s["other"].double()
            h = (s["x"].float() + s["other"].float()).to(s["x"].dtype).double()
        y = h / torch.sqrt(h.square().sum(1, keepdim=True) / c["width"] + EPS)
        y = y * s["weight"].double()
        if c["out"] != "fp8":
            return dict(out, y=y)
        cols = torch.arange(c["width"], device="cuda") // BLOCK
        scale = torch.stack([p.abs().amax(1) for p in y.split(BLOCK, 1)], 1) / E4M3_MAX
        scale = scale.clamp_min(TINY)
        q = (y / scale[:, cols]).float().to(torch.float8_e4m3fn)
        return dict(out, q=q.double(), scale=scale)
    if kind == "normgrad":
        h = s["x"].double()
        n = torch.sqrt(h.square().sum(1, keepdim=True) / c["width"] + EPS)
        dy = s["dy"].double()
        g = dy * s["weight"].double()
        dx = g / n - h * ((g * h).sum(1, keepdim=True) / (c["width"] * n ** 3))
        if s["other"] is not None:
            dx += s["other"].double()
        return {"dx": dx, "dw": torch.einsum("rh,rh->h", dy, h / n)}
    return _route_exact(s) if kind == "route" else _routegrad_exact(s)
