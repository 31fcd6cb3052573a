"""Timing cases of the expert-layer and gradient-norm operators.

The operators follow the pooled embeddings into a layer of experts and close
its training step:

  move     assignments sorted by expert, the tokens' rows carried to their
           experts, the experts' rows weighted and summed back per token
  grad     the gradients of both: of the experts' rows and the weights, and of
           the tokens
  product  the experts' matrix products in 8-bit floating point, a scale for
           each 128 columns of a row and each 128 x 128 block of weights
  layer    tokens carried to their experts in 8 bits, then the product
  clip     global norm over many gradients, and the clipped gradients

Every case runs in a plain form (elementary torch operations in 32 bits,
`own` false) or through this framework's entry points (`own` true), on the
same state.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16,
          "i32": torch.int32, "i64": torch.int64}
BLOCK = 128          # columns that share a scale
E4M3_MAX = 448.0     # largest finite e4m3 value
TINY = 2.0 ** -126   # smallest scale


def _bytes(dtype):
    return DTYPES[dtype].itemsize


def _blocks(n):
    return -(-n // BLOCK)


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # a few tokens being answered: one row each, every launch counts
        dict(name="move_token", kind="move", tokens=4, k=2, experts=16, width=1024, dtype="bf16",
             ids="i32", drop=0.0),
        # one batch of 4096 bags; the assignments over their expert's capacity are dropped
        dict(name="move_batch", kind="move", tokens=4096, k=4, experts=64, width=1000, dtype="f16",
             ids="i64", drop=0.05),
        # the pooled output of eight tables of width 128 over 131072 bags, in its own type
        dict(name="move_pooled", kind="move", tokens=131072, k=2, experts=32, width=1024,
             dtype="f32", ids="i32", drop=0.0),
        # a training batch whose sizes divide by nothing
        dict(name="grad_ragged", kind="grad", tokens=4097, k=3, experts=10, width=1001,
             dtype="f16", ids="i32", drop=0.1),
        # a large training batch
        dict(name="grad_large", kind="grad", tokens=65536, k=4, experts=64, width=2048,
             dtype="bf16", ids="i32", drop=0.0),
        # tokens being answered: a handful of rows against many experts, the weights' bytes count
        dict(name="product_token", kind="product", rows=16, experts=64, n=2048, kdim=1024,
             out="bf16", used=1.0),
        # an ordinary batch with ends that fill no tile, summed further in 32 bits
        dict(name="product_ragged", kind="product", rows=5000, experts=8, n=1000, kdim=1008,
             out="f32", used=0.95),
        # one dense projection of a prompt
        dict(name="product_dense", kind="product", rows=2048, experts=1, n=4096, kdim=4096,
             out="bf16", used=1.0),
        # a large batch over sixteen experts
        dict(name="product_large", kind="product", rows=65536, experts=16, n=4096, kdim=2048,
             out="bf16", used=1.0),
        # the first half of an expert layer on a batch of 8192 pooled vectors
        dict(name="layer_batch", kind="layer", tokens=8192, k=4, experts=32, width=1024, n=2048,
             dtype="bf16", ids="i32", drop=0.02),
        # a small model's gradients, three types among them
        dict(name="clip_mixed", kind="clip", tensors=48, total=3_000_001, dtype="mixed", spread=2.5,
             max_norm=1.0),
        # a large model's gradients
        dict(name="clip_large", kind="clip", tensors=300, total=(1 << 29) + 77, dtype="bf16",
             spread=4.0, max_norm=1.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _odd_width(rng, lo, hi):
    w = _log(rng, lo, hi)
    w -= w % rng.choice([1, 8, 64])
    return max(lo, w if w != 3072 else 3064)


def draw(rng):
    kind = rng.choice(["move", "grad", "product", "layer", "clip"])
    top = {c["name"]: work(c) for c in listed()}
    while True:
        if kind in ("move", "grad"):
            experts = _log(rng, 2, 256)
            c = dict(kind=kind, tokens=_log(rng, 1, 131072), k=rng.randint(1, min(8, experts)),
                     experts=experts, width=_odd_width(rng, 8, 4096),
                     dtype=rng.choice(["f16", "bf16", "f32"]), ids=rng.choice(["i32", "i64"]),
                     drop=rng.choice([0.0, 0.03, 0.5]))
            most = top["move_pooled" if kind == "move" else "grad_large"]
        elif kind == "product":
            kdim, n = 16 * _log(rng, 4, 256), _odd_width(rng, 16, 4096)
            c = dict(kind=kind, rows=_log(rng, 1, 65536), experts=_log(rng, 1, 64), n=n,
                     kdim=kdim if kdim != 3072 else 3088, out=rng.choice(["f16", "bf16", "f32"]),
                     used=rng.choice([1.0, 0.9]))
            most = top["product_large"]
        elif kind == "layer":
            experts, width = _log(rng, 2, 64), 16 * _log(rng, 4, 128)
            c = dict(kind=kind, tokens=_log(rng, 1, 16384), k=rng.randint(1, min(8, experts)),
                     experts=experts, width=width, n=_odd_width(rng, 16, 4096),
                     dtype=rng.choice(["f16", "bf16", "f32"]), ids=rng.choice(["i32", "i64"]),
                     drop=rng.choice([0.0, 0.05]))
            most = top["product_large"]
        else:
            tensors = _log(rng, 1, 400)
            c = dict(kind=kind, tensors=tensors, total=_log(rng, 64 * tensors, 1 << 28),
                     dtype=rng.choice(["f32", "bf16", "f16", "mixed"]),
                     spread=round(rng.uniform(0.5, 4.0), 2), max_norm=rng.choice([0.5, 1.0, 1e6]))
            most = top["clip_large"]
        w = work(c)
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]:
            return c


def work(case):
    """Bytes read once and written once, and operations, of one pass."""
    c, kind = case, case["kind"]
    if kind in ("move", "grad"):
        A, N, H, s = c["tokens"] * c["k"], c["tokens"], c["width"], _bytes(c["dtype"])
        if kind == "move":  # ids, plan, x -> rows, y -> out with weights
            return {"bytes": A * (_bytes(c["ids"]) + 8 + 4) + 2 * (N + A) * H * s,
                    "flops": 2 * A * H}
        # dout, y -> dy, dw with plan and weights; drows -> dx
        return {"bytes": (N + 2 * A) * H * s + 12 * A + (A + N) * H * s, "flops": 4 * A * H}
    if kind == "product":
        rows, N, K, E = c["rows"], c["n"], c["kdim"], c["experts"]
        read = rows * (K + 4 * _blocks(K)) + min(rows, E) * (N * K + 4 * _blocks(N) * _blocks(K))
        return {"bytes": read + rows * N * _bytes(c["out"]),
                "flops": 2 * int(rows * c["used"]) * N * K}
    if kind == "layer":
        A, N, H, s = c["tokens"] * c["k"], c["tokens"], c["width"], _bytes(c["dtype"])
        w = min(A, c["experts"]) * (c["n"] * H + 4 * _blocks(c["n"]) * _blocks(H))
        return {"bytes": N * H * s + 4 * A + w + A * c["n"] * s, "flops": 2 * A * c["n"] * H}
    sizes, types = _tensor_list(c)
    return {"bytes": 2 * sum(n * t.itemsize for n, t in zip(sizes, types)), "flops": 3 * c["total"]}


# --------------------------------------------------------------- the inputs

def _rand(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _routing(c, g):
    """Distinct experts per token, some experts liked more than others; dropped assignments hold -1."""
    logits = _randn(g, c["tokens"], c["experts"]) + _randn(g, c["experts"])
    val, ids = logits.topk(c["k"], dim=1)
    gone = torch.rand(ids.shape, generator=g, device="cuda") < c["drop"]
    return ids.masked_fill(gone, -1).to(DTYPES[c["ids"]]), torch.softmax(val, 1)


def _fill(g, rows, cols, dtype):
    out = torch.empty(rows, cols, dtype=DTYPES[dtype], device="cuda")
    step = max(1, (1 << 27) // max(cols, 1))
    for r in range(0, rows, step):
        out[r:r + step] = _randn(g, min(step, rows - r), cols)
    return out


def _tensor_list(c):
    """Sizes of the gradients (log-normal, `spread` octaves, exact total) and their types."""
    r = random.Random("%d %d" % (c["tensors"], c["total"]))
    raw = [2.0 ** r.gauss(0, c["spread"]) for _ in range(c["tensors"])]
    sizes = [max(1, int(c["total"] * v / sum(raw))) for v in raw]
    most = max(range(len(sizes)), key=sizes.__getitem__)
    sizes[most] += c["total"] - sum(sizes)
    names = ["f32", "bf16", "f16"] if c["dtype"] == "mixed" else [c["dtype"]]
    return sizes, [DTYPES[names[i % len(names)]] for i in range(len(sizes))]


def _quantized_weights(g, experts, n, k):
    q, s = [], []
    for _ in range(experts):
        w = _randn(g, n, k) / math.sqrt(k)
        pad = torch.nn.functional.pad(w, (0, -k % BLOCK, 0, -n % BLOCK))
        tiles = pad.view(_blocks(n), BLOCK, _blocks(k), BLOCK)
        sc = (tiles.abs().amax((1, 3)) / E4M3_MAX).clamp_min(TINY)
        q.append((tiles / sc[:, None, :, None]).view(pad.shape)[:n, :k].to(torch.float8_e4m3fn))
        s.append(sc)
    return torch.stack(q), torch.stack(s)


def prepare(case, seed):
    c, g = case, _rand(seed)
    kind = c["kind"]
    if kind in ("move", "grad", "layer"):
        ids, w = _routing(c, g)
        s = {"kind": kind, "experts": c["experts"], "ids": ids}
        x = _fill(g, c["tokens"], c["width"], c["dtype"])
        if kind == "layer":
            wq, ws = _quantized_weights(g, c["experts"], c["n"], c["width"])
            s.update(x=x, wq=wq, ws=ws)
        else:
            y = _fill(g, ids.numel(), c["width"], c["dtype"])
            s.update(w=w, y=y, **({"x": x} if kind == "move" else {"dout": x}))
        if kind != "move":  # the forward pass has left its plan
            s["offsets"], s["source"], s["position"] = _sort_plain(ids, c["experts"])
            s["sizes"] = s["offsets"].diff().tolist()
        if kind == "grad":
            s["drows"] = _fill(g, ids.numel(), c["width"], c["dtype"])
        return s
    if kind == "product":
        p = torch.softmax(_randn(g, c["experts"]), 0)
        of = torch.multinomial(p, int(c["rows"] * c["used"]), replacement=True, generator=g)
        sizes = torch.bincount(of, minlength=c["experts"])
        offsets = torch.nn.functional.pad(sizes.cumsum(0), (1, 0)).to(torch.int32)
        # activations: rows of different loudness
        x = _fill(g, c["rows"], c["kdim"], "f32") * torch.exp(_randn(g, c["rows"], 1))
        q, scale = _quantize_plain(x)
        wq, ws = _quantized_weights(g, c["experts"], c["n"], c["kdim"])
        return {"kind": kind, "q": q, "scale": scale, "wq": wq, "ws": ws, "offsets": offsets,
                "sizes": sizes.tolist(), "out": DTYPES[c["out"]]}
    sizes, types = _tensor_list(c)
    loud = torch.exp(_randn(g, len(sizes)) * 1.5 - 6).tolist()
    grads = [(_randn(g, n) * a).to(t) for n, t, a in zip(sizes, types, loud)]
    # clipped gradients go to one flat buffer per type, every tensor on a 64-element boundary
    room, place = {}, []
    for n, t in zip(sizes, types):
        place.append(room.get(t, 0))
        room[t] = place[-1] + -(-n // 64) * 64
    flat = {t: torch.zeros(n, dtype=t, device="cuda") for t, n in room.items()}
    out = [flat[t][at:at + n] for n, t, at in zip(sizes, types, place)]
    return {"kind": kind, "grads": grads, "out": out, "flat": list(flat.values()),
            "max_norm": c["max_norm"]}


# ----------------------------------------------------------- the plain forms

def _sort_plain(ids, experts):
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < experts), flat, experts).to(torch.int32)
    sorted_key, order = torch.sort(key, stable=True)
    kept = sorted_key < experts
    source = torch.where(kept, order, -1).to(torch.int32)
    place = torch.arange(key.numel(), device=key.device, dtype=torch.int32)
    position = torch.empty_like(place)
    position[order] = torch.where(kept, place, -1)
    edges = torch.arange(experts + 1, device=key.device, dtype=torch.int32)
    offsets = torch.searchsorted(sorted_key, edges).to(torch.int32)
    return offsets, source, position.view(ids.shape)


def _carry_plain(x, source, k):
    rows = x[source.clamp_min(0) // k]
    return torch.where((source >= 0)[:, None], rows, torch.zeros((), dtype=x.dtype, device=x.device))


def _pool_plain(y, position, w):
    rows = torch.where((position >= 0)[..., None], y[position.clamp_min(0)].float(), 0.0)
    return (rows if w is None else rows * w[..., None]).sum(1).to(y.dtype)


def _quantize_plain(x):
    rows, cols = x.shape
    pad = torch.nn.functional.pad(x.float(), (0, -cols % BLOCK)).view(rows, -1, BLOCK)
    scale = (pad.abs().amax(2) / E4M3_MAX).clamp_min(TINY)
    q = (pad / scale[..., None]).view(rows, -1)[:, :cols].to(torch.float8_e4m3fn)
    return q.contiguous(), scale


def _widen(q, scale, rows_per_scale):
    s = scale.repeat_interleave(BLOCK, 1)[:, :q.shape[1]]
    if rows_per_scale > 1:
        s = s.repeat_interleave(rows_per_scale, 0)[:q.shape[0]]
    return q.float() * s


def _product_plain(q, scale, wq, ws, sizes, dtype):
    a = _widen(q, scale, 1)
    parts = torch.split(a, sizes + [q.shape[0] - sum(sizes)])
    outs = [p @ _widen(wq[e], ws[e], BLOCK).T for e, p in enumerate(parts[:-1]) if len(p)]
    rest = torch.zeros(parts[-1].shape[0], wq.shape[1], device=q.device)
    return torch.cat(outs + [rest]).to(dtype)


def _grad_plain(s):
    source, position, w = s["source"], s["position"], s["w"]
    k = position.shape[1]
    kept = (source >= 0)[:, None]
    token, flat = source.clamp_min(0) // k, source.clamp_min(0).long()
    dout = s["dout"].float()[token]
    dy = torch.where(kept, dout * w.reshape(-1)[flat][:, None], 0.0).to(s["y"].dtype)
    dots = (dout * s["y"].float()).sum(1)
    dw = torch.where(position >= 0, dots[position.clamp_min(0)], 0.0)
    return {"dy": dy, "dw": dw, "dx": _pool_plain(s["drows"], position, None)}


def _clip_plain(s):
    norm = torch.stack([g.float().square().sum() for g in s["grads"]]).sum().sqrt()
    c = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    [o.copy_(g.float() * c) for o, g in zip(s["out"], s["grads"])]
    return {"norm": norm, "out": s["flat"]}


def _run_plain(s):
    kind = s["kind"]
    if kind == "move":
        offsets, source, position = _sort_plain(s["ids"], s["experts"])
        return {"offsets": offsets, "source": source, "position": position,
                "rows": _carry_plain(s["x"], source, position.shape[1]),
                "out": _pool_plain(s["y"], position, s["w"])}
    if kind == "grad":
        return _grad_plain(s)
    if kind == "product":
        return _product_plain(s["q"], s["scale"], s["wq"], s["ws"], s["sizes"], s["out"])
    if kind == "layer":
        rows = _carry_plain(s["x"], s["source"], s["position"].shape[1])
        q, scale = _quantize_plain(rows)
        return _product_plain(q, scale, s["wq"], s["ws"], s["sizes"], s["x"].dtype)
    return _clip_plain(s)


# ------------------------------------------------- the framework's operators

def _run_own(s):
    import table_embedding_bag_gb300 as tbe
    kind = s["kind"]
    if kind == "move":
        offsets, source, position = tbe.tbe_expert_sort(s["ids"], s["experts"])
        return {"offsets": offsets, "source": source, "position": position,
                "rows": tbe.tbe_expert_dispatch(s["x"], offsets, position),
                "out": tbe.tbe_expert_combine(s["y"], position, s["w"])}
    if kind == "grad":
        dy, dw = tbe.tbe_expert_combine_backward(s["dout"], s["y"], s["offsets"], s["position"],
                                                 s["w"])
        return {"dy": dy, "dw": dw,
                "dx": tbe.tbe_expert_dispatch_backward(s["drows"], s["position"])}
    if kind == "product":
        return tbe.tbe_expert_product(s["q"], s["scale"], s["wq"], s["ws"], s["offsets"],
                                      out_dtype=s["out"])
    if kind == "layer":
        q, scale = tbe.tbe_expert_dispatch_fp8(s["x"], s["offsets"], s["position"])
        return tbe.tbe_expert_product(q, scale, s["wq"], s["ws"], s["offsets"],
                                      out_dtype=s["x"].dtype)
    norm = tbe.tbe_grad_clip(s["grads"], s["max_norm"], out=s["out"])
    return {"norm": norm, "out": s["flat"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------- the values in 64 bits

def _plan_exact(ids, experts):
    """Places by counting: a running count per expert instead of a sort."""
    flat = ids.reshape(-1).long()
    kept = (flat >= 0) & (flat < experts)
    hot = torch.zeros(flat.numel(), experts, dtype=torch.int32, device=flat.device)
    hot[kept.nonzero()[:, 0], flat[kept]] = 1
    seen = hot.cumsum(0, dtype=torch.int32)
    offsets = torch.cat([seen.new_zeros(1), seen[-1].cumsum(0).to(torch.int32)])
    rank = seen.gather(1, flat.clamp(0, experts - 1)[:, None])[:, 0] - 1
    position = torch.where(kept, offsets[flat.clamp(0, experts - 1)] + rank, -1)
    source = torch.full_like(position, -1)
    source[position[kept].long()] = kept.nonzero()[:, 0].to(source.dtype)
    return offsets, source, position.view(ids.shape)


def _pool_exact(y, position, w):
    out = torch.zeros(position.shape[0], y.shape[1], dtype=torch.float64, device=y.device)
    for j in range(position.shape[1]):
        n = (position[:, j] >= 0).nonzero()[:, 0]
        rows = y[position[n, j].long()].double()
        out[n] += rows if w is None else rows * w[n, j].double()[:, None]
    return out


def _product_exact(q, scale, wq, ws, offsets):
    out = torch.zeros(q.shape[0], wq.shape[1], dtype=torch.float64, device=q.device)
    K, at = q.shape[1], offsets.tolist()
    for e in range(wq.shape[0]):
        if at[e + 1] > at[e]:
            col = torch.arange(K, device=q.device) // BLOCK
            row = torch.arange(wq.shape[1], device=q.device) // BLOCK
            w = wq[e].double() * ws[e].double()[row][:, col]
            a = q[at[e]:at[e + 1]].double() * scale[at[e]:at[e + 1]].double()[:, col]
            out[at[e]:at[e + 1]] = torch.mm(a, w.t())
    return out


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "product":
        return _product_exact(s["q"], s["scale"], s["wq"], s["ws"], s["offsets"])
    if kind == "clip":
        norm = math.sqrt(sum(float(g.double().pow(2).sum()) for g in s["grads"]))
        c = min(1.0, case["max_norm"] / (norm + 1e-6))
        flat = [torch.zeros(f.shape, dtype=torch.float64, device=f.device) for f in s["flat"]]
        for o, g in zip(s["out"], s["grads"]):
            k = next(i for i, f in enumerate(s["flat"]) if f.dtype == g.dtype)
            flat[k][o.storage_offset():o.storage_offset() + o.numel()] = g.double() * c
        return {"norm": norm, "out": flat}
    offsets, source, position = _plan_exact(s["ids"], case["experts"])
    kept = (source >= 0).nonzero()[:, 0]
    token = source[kept].long() // case["k"]
    if kind == "move":
        rows = torch.zeros(source.numel(), case["width"], dtype=torch.float64, device="cuda")
        rows[kept] = s["x"][token].double()
        return {"offsets": offsets, "source": source, "position": position, "rows": rows,
                "out": _pool_exact(s["y"], position, s["w"])}
    if kind == "grad":
        dy = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros(position.numel(), dtype=torch.float64, device="cuda")
        step = 1 << 15
        for i in range(0, kept.numel(), step):
            r, a, t = kept[i:i + step], source[kept[i:i + step]].long(), token[i:i + step]
            dout = s["dout"][t].double()
            dy[r] = dout * s["w"].reshape(-1)[a].double()[:, None]
            dw[a] = torch.einsum("rh,rh->r", dout, s["y"][r].double())
        return {"dy": dy, "dw": dw.view(position.shape), "dx": _pool_exact(s["drows"], position, None)}
    # layer: the 8-bit values are part of the definition, so they are formed as it says
    x = torch.zeros(source.numel(), case["width"], device="cuda")
    x[kept] = s["x"][token].float()
    q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(x.shape[0], _blocks(case["width"]), device="cuda")
    for b in range(scale.shape[1]):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        scale[:, b] = torch.maximum(part.abs().max(1).values / E4M3_MAX,
                                    torch.tensor(TINY, device="cuda"))
        q[:, b * BLOCK:(b + 1) * BLOCK] = (part / scale[:, b:b + 1]).to(torch.float8_e4m3fn)
    return _product_exact(q, scale, s["wq"], s["ws"], offsets)
