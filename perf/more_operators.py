"""The operators around the expert layer, case by case: what they take, what
they compute and what each cannot do without.

Three operators of a mixture-of-experts training step:

* norm   - the joint between two blocks: the norm after a block, its gate, the
           scaled residual sum and the norm before the next block, and the
           gradients of all of it;
* router - the choice of the experts from the router's logits, the counts per
           expert, a balance loss and a loss on the logits' size, and the
           gradient for the logits;
* clip   - the global norm of many gradient tensors, and their clipping.

``own`` false computes them in elementary torch operations, true by this
package's operators.
"""
import math
import random

import torch

own = False

EPS = 1e-5
CLIP_EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token of one sequence between two blocks: latency
        dict(name="norm_token", kind="norm", tokens=1, width=768, stream="fp32", dtype="bf16", join=True, after=True,
             gate="channel", before=True, res_scale=1.0, out_scale=1.0, padded=0),
        # between two blocks of a training microbatch of 32 x 1024 tokens
        dict(name="norm_step", kind="norm", tokens=32768, width=768, stream="fp32", dtype="bf16", join=True, after=True,
             gate="channel", before=True, res_scale=1.0, out_scale=0.25, padded=0),
        # the same microbatch's gradients
        dict(name="norm_step_grad", kind="norm_grad", tokens=32768, width=768, stream="fp32", dtype="bf16", join=True,
             after=True, gate="channel", before=True, res_scale=1.0, out_scale=0.25, padded=0),
        # a padded batch of odd sizes, a gate for every element, fp32 throughout
        dict(name="norm_odd_grad", kind="norm_grad", tokens=1537, width=1001, stream="fp32", dtype="fp32", join=True,
             after=True, gate="full", before=True, res_scale=0.5, out_scale=1.0, padded=100),
        # the router of a single token
        dict(name="router_token", kind="router", tokens=1, experts=16, top_k=2, dtype="fp32", renormalize=True,
             masked=0.0, closed=0),
        # a microbatch's router
        dict(name="router_step", kind="router", tokens=32768, experts=16, top_k=2, dtype="fp32", renormalize=True,
             masked=0.0, closed=0),
        # its gradient
        dict(name="router_step_grad", kind="router_grad", tokens=32768, experts=16, top_k=2, dtype="fp32",
             renormalize=True, masked=0.0, closed=0),
        # the tokens of a whole update of 16 microbatches over many experts, some tokens padding
        dict(name="router_top8", kind="router", tokens=131072, experts=64, top_k=8, dtype="bf16", renormalize=False,
             masked=0.1, closed=0),
        # the gradients of a small model's few tensors: latency
        dict(name="clip_small", kind="clip", tensors="model", vocab=256, width=64, layers=2, heads=64, experts=4,
             ffn=128, dtype="fp32", packed=False, max_norm=1.0, scale=1.0),
        # one by one, the gradient tensors of every layer of a 219M-parameter model
        dict(name="clip_model", kind="clip", tensors="model", vocab=32000, width=768, layers=8, heads=768, experts=16,
             ffn=512, dtype="fp32", packed=False, max_norm=1.0, scale=0.0625),
        # many ragged bf16 tensors, packed one behind the other without alignment
        dict(name="clip_ragged", kind="clip", tensors="ragged", count=500, total=20000000, sizes=1,
             dtype="bf16", packed=True, max_norm=1.0, scale=1.0),
    ]


def _spread(rng, lo, hi):
    """A whole number spread over the logarithm of lo..hi, odd ones among them."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["norm", "norm", "norm_grad", "norm_grad", "router", "router_grad", "clip"])
    if kind in ("norm", "norm_grad"):
        width = _spread(rng, 16, 8192)
        if rng.random() < 0.7:
            width = -(-width // 8) * 8
        tokens = _spread(rng, 1, max(1, min(65536, (32768 * 768) // width)))
        stream, dtype = rng.choice([("fp32", "bf16"), ("fp32", "bf16"), ("bf16", "bf16"), ("fp32", "fp32")])
        join = rng.random() < 0.8
        return dict(kind=kind, tokens=tokens, width=width, stream=stream, dtype=dtype, join=join,
                    after=join and rng.random() < 0.7, gate=rng.choice(["none", "channel", "token", "full"]) if join else "none",
                    before=not join or rng.random() < 0.8, res_scale=rng.choice([1.0, 0.75]) if join else 1.0,
                    out_scale=rng.choice([1.0, 0.25]) if join else 1.0,
                    padded=rng.choice([0, 0, rng.randint(0, tokens)]))
    if kind in ("router", "router_grad"):
        experts = rng.randint(2, 64)
        top_k = rng.randint(1, min(8, experts))
        tokens = _spread(rng, 1, 131072)
        return dict(kind=kind, tokens=tokens, experts=experts, top_k=top_k, dtype=rng.choice(["fp32", "bf16"]),
                    renormalize=rng.random() < 0.7, masked=rng.choice([0.0, 0.0, 0.3]),
                    closed=rng.choice([0, 0, rng.randint(0, experts - 1)]))
    return dict(kind="clip", tensors="ragged", count=_spread(rng, 1, 500), total=_spread(rng, 1000, 100000000),
                sizes=rng.randint(0, 1 << 30), dtype=rng.choice(["fp32", "bf16"]), packed=rng.random() < 0.5,
                max_norm=rng.choice([1.0, 1e9]), scale=rng.choice([1.0, 0.125]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(gen, shape, std, dtype=torch.float32, mean=0.0):
    return (torch.randn(shape, generator=gen, device=gen.device) * std + mean).to(dtype)


def _hidden(gen, shape, dtype):
    """Hidden rows: unit normal, a few channels several times larger."""
    gain = 1.0 + 4.0 * (torch.rand(shape[-1], generator=gen, device=gen.device) < 0.01).float()
    return (torch.randn(shape, generator=gen, device=gen.device) * gain).to(dtype)


def _shapes(case):
    """The shapes of a gradient set."""
    if case["tensors"] == "model":
        v, d, hq, e, f = (case[k] for k in ("vocab", "width", "heads", "experts", "ffn"))
        layer = [(d,), (3 * hq, d), (d, hq), (d,), (e, d), (e, f, d), (e, f, d), (e, d, f)]
        return [(v, d)] + layer * case["layers"] + [(d,), (v, d)]
    rng = random.Random(case["sizes"])
    share = [math.exp(rng.uniform(0.0, 8.0)) for _ in range(case["count"])]
    per = case["total"] / sum(share)
    return [(max(1, int(per * s)),) for s in share]


def _set_of(shapes, packed, dtype, dev):
    """A buffer and its parts of these shapes: one behind the other, or each on a boundary of 64 elements."""
    sizes = [math.prod(x) for x in shapes]
    room = [n if packed else -(-n // 64) * 64 for n in sizes]
    flat = torch.zeros(sum(room), dtype=dtype, device=dev)
    return flat, [g[:n].view(sh) for g, n, sh in zip(flat.split(room), sizes, shapes)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev, kind = gen.device, case["kind"]
    dt = TYPES[case["dtype"]]
    s = {"case": case}
    if kind in ("norm", "norm_grad"):
        t, d, st = case["tokens"], case["width"], TYPES[case["stream"]]
        s["y"] = _normal(gen, (t, d), 0.5, dt) if case["join"] else None
        s["after"] = _normal(gen, (d,), 0.1, mean=1.0) if case["after"] else None
        s["before"] = _normal(gen, (d,), 0.1, mean=1.0) if case["before"] else None
        gate = case["gate"]
        s["gate"] = None if gate == "none" else _normal(gen, (d,), 0.3) if gate == "channel" else \
            torch.sigmoid(_normal(gen, (t, 1), 1.0)) if gate == "token" else torch.sigmoid(_normal(gen, (t, d), 1.0)).to(dt)
        s["n_rows"] = torch.tensor([t - case["padded"]], dtype=torch.int32, device=dev) if case["padded"] else None
        s["x" if kind == "norm" else "h"] = _hidden(gen, (t, d), st)
        if kind == "norm":
            s["h"] = torch.zeros((t, d), dtype=st, device=dev)
            s["r"] = torch.zeros((t, d), dtype=dt, device=dev)
        else:
            s["dr"] = _normal(gen, (t, d), 1e-3, dt) if case["before"] else None
            s["dh"] = _normal(gen, (t, d), 1e-3, st)
            s["dx"] = torch.zeros((t, d), dtype=st, device=dev)
            s["dy"] = torch.zeros((t, d), dtype=dt, device=dev) if case["join"] else None
            s["dgate"] = torch.zeros_like(s["gate"]) if s["gate"] is not None else None
    elif kind in ("router", "router_grad"):
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        z = torch.randn((t, e), generator=gen, device=dev) + 0.5 * torch.randn(e, generator=gen, device=dev)
        z[:, torch.randperm(e, generator=gen, device=dev)[:case["closed"]]] = -math.inf
        s["z"] = z.to(dt)
        s["mask"] = torch.rand(t, generator=gen, device=dev) >= case["masked"] if case["masked"] else None
        if kind == "router_grad":
            s["idx"], _, s["counts"], _ = _choose(s["z"], k, s["mask"], case["renormalize"])
            s["dw"] = _normal(gen, (t, k), 1e-3)
            s["dlosses"] = torch.tensor([1e-2, 1e-3], device=dev)
    else:
        shapes = _shapes(case)
        std = 0.02 * 2.0 ** _normal(gen, (len(shapes),), 1.0).cpu()
        s["flat"], s["out"] = _set_of(shapes, case["packed"], dt, dev)
        s["grads"] = [g.copy_(_normal(gen, g.shape, float(x))) for g, x in zip(_set_of(shapes, case["packed"], dt, dev)[1], std)]
    return s


# ---------------------------------------------------------------------------
# the operators' plain forms, in 32 bits
# ---------------------------------------------------------------------------
def _inv_rms(v):
    return torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)


def _rows(v, into, n_rows):
    """The rows of v below n_rows in `into`'s type, its own rows behind them."""
    v = v.to(into.dtype)
    if n_rows is None:
        return v
    return torch.where(torch.arange(v.shape[0], device=v.device)[:, None] < n_rows, v, into)


def _softmax(z, live):
    """Probabilities and logs of the sums of exponentials; zeros in rows that take no part."""
    top = torch.where(live, z.amax(1), 0.0)[:, None]
    ex = torch.where(live[:, None], torch.exp(z - top), 0.0)
    total = torch.where(live, ex.sum(1), 1.0)
    return ex / total[:, None], torch.where(live, top[:, 0] + torch.log(total), 0.0)


def _choose(z, top_k, mask, renormalize):
    z = z.float() + 0.0
    n, e = z.shape
    live = z.amax(1) > -math.inf
    if mask is not None:
        live = live & mask
    p, lse = _softmax(z, live)
    by = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :top_k]
    open_ = live[:, None] & (z.gather(1, by) > -math.inf)
    idx = torch.where(open_, by, -1)
    w = torch.where(open_, p.gather(1, by), 0.0)
    if renormalize:
        top = torch.where(live, z.amax(1), 0.0)[:, None]
        ex = torch.where(open_, torch.exp(z.gather(1, by) - top), 0.0)
        w = ex / torch.where(live, ex.sum(1), 1.0)[:, None]
    counts = (idx.reshape(-1, 1) == torch.arange(e, device=z.device)).sum(0)
    tokens = live.sum()
    many = tokens.clamp(min=1).double()
    mean_p = p.sum(0, dtype=torch.float64) / many
    balance = e / (top_k * many) * (counts * mean_p).sum()
    size = (lse.double() ** 2).sum() / many
    return (idx.to(torch.int32), w, torch.cat([counts, tokens[None]]).to(torch.int32),
            torch.stack([balance, size]).float())


def _choose_grad(z, idx, counts, dw, dlosses, mask, renormalize):
    zf = z.float()
    n, e = zf.shape
    top_k = idx.shape[1]
    live = zf.amax(1) > -math.inf
    if mask is not None:
        live = live & mask
    p, lse = _softmax(zf, live)
    chosen = idx >= 0
    at = idx.clamp(min=0).long()
    dw = torch.where(chosen, dw, 0.0)
    w = torch.where(chosen, p.gather(1, at), 0.0)
    if renormalize:
        top = torch.where(live, zf.amax(1), 0.0)[:, None]
        ex = torch.where(chosen, torch.exp(zf.gather(1, at) - top), 0.0)
        w = ex / torch.where(live, ex.sum(1), 1.0)[:, None]
    own_part = torch.zeros_like(zf).scatter_add_(1, at, w * dw)
    dot = (w * dw).sum(1, keepdim=True)
    if renormalize:
        dz = own_part - torch.zeros_like(zf).scatter_add_(1, at, w) * dot
    else:
        dz = own_part - p * dot
    many = counts[-1].clamp(min=1).float()
    c = counts[:-1].float()
    dz = dz + (dlosses[0] * e / (top_k * many * many)) * p * (c - (p * c).sum(1, keepdim=True))
    dz = dz + (dlosses[1] * 2.0 / many) * lse[:, None] * p
    return torch.where(live[:, None], dz, 0.0).to(z.dtype)


def run(state):
    """One pass."""
    if own:
        return _run_own(state)
    c, s = state["case"], state
    kind = c["kind"]
    if kind == "norm":
        h = s["x"].float()
        if c["join"]:
            n = s["y"].float()
            if c["after"]:
                n = n * _inv_rms(n) * s["after"]
            if s["gate"] is not None:
                n = n * s["gate"].float()
            h = c["res_scale"] * h + c["out_scale"] * n
        out = {"h": _rows(h, s["h"], s["n_rows"]) if c["join"] else None}
        out["r"] = _rows(h * _inv_rms(h) * s["before"], s["r"], s["n_rows"]) if c["before"] else None
        return out
    if kind == "norm_grad":
        live = None if s["n_rows"] is None else torch.arange(c["tokens"], device=s["h"].device)[:, None] < s["n_rows"]
        cut = lambda v: v if live is None else torch.where(live, v, 0.0)        # noqa: E731
        g, h = s["dh"].float(), s["h"].float()
        out = dict.fromkeys(("dx", "dy", "dafter", "dgate", "dbefore"))
        if c["before"]:
            ir, dr = _inv_rms(h), s["dr"].float()
            u, hn = dr * s["before"], h * _inv_rms(h)
            g = g + ir * (u - hn * (u * hn).mean(1, keepdim=True))
            out["dbefore"] = cut(dr * hn).sum(0)
        out["dx"] = _rows(c["res_scale"] * g, s["dx"], s["n_rows"])
        if not c["join"]:
            return out
        g, y = c["out_scale"] * g, s["y"].float()
        ir = _inv_rms(y) if c["after"] else None
        n = y * ir * s["after"] if c["after"] else y
        if s["gate"] is not None:
            dgate = g * n
            out["dgate"] = cut(dgate).sum(0) if c["gate"] == "channel" else \
                _rows(dgate.sum(1, keepdim=True) if c["gate"] == "token" else dgate, s["dgate"], s["n_rows"])
            g = g * s["gate"].float()
        if c["after"]:
            yn = y * ir
            out["dafter"] = cut(g * yn).sum(0)
            u = g * s["after"]
            g = ir * (u - yn * (u * yn).mean(1, keepdim=True))
        out["dy"] = _rows(g, s["dy"], s["n_rows"])
        return out
    if kind == "router":
        idx, w, counts, losses = _choose(s["z"], c["top_k"], s["mask"], c["renormalize"])
        return {"idx": idx, "w": w, "counts": counts, "losses": losses}
    if kind == "router_grad":
        return _choose_grad(s["z"], s["idx"], s["counts"], s["dw"], s["dlosses"], s["mask"], c["renormalize"])
    total = torch.stack([(g.float() ** 2).sum(dtype=torch.float64) for g in s["grads"]]).sum()
    norm = abs(c["scale"]) * total.sqrt()
    coef = (c["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)
    by = (c["scale"] * coef).float()
    for g, o in zip(s["grads"], s["out"]):
        o.copy_(g.float() * by)
    return {"stats": torch.stack([norm, coef]).float(), "grads": s["flat"]}     # `out` is its parts


def _run_own(state):
    """The calls of a program that keeps its buffers (made at its first step)."""
    from adamw_persistent_sm_gb300 import block_ops as ops
    c, s = state["case"], state
    kind = c["kind"]
    if kind == "norm":
        h, r = ops.block_norm(s["x"], s["y"], after=s["after"], gate=s["gate"], before=s["before"],
                              res_scale=c["res_scale"], out_scale=c["out_scale"], eps=EPS, n_rows=s["n_rows"],
                              h=s["h"] if c["join"] else None, r=s["r"] if c["before"] else None)
        return {"h": h if c["join"] else None, "r": r}
    kept = s.get("kept")
    if kind == "norm_grad":
        if kept is None:
            kept = s["kept"] = [None if v is None else torch.empty_like(v) for v in (s["after"], s["before"])]
        g = ops.block_norm_bwd(s["dr"], s["dh"], s["h"], s["y"], after=s["after"], gate=s["gate"], before=s["before"],
                               res_scale=c["res_scale"], out_scale=c["out_scale"], eps=EPS, n_rows=s["n_rows"],
                               dx=s["dx"], dy=s["dy"], dgate=s["dgate"], dafter=kept[0], dbefore=kept[1])
        return {"dx": g.dx, "dy": g.dy, "dafter": g.dafter, "dgate": g.dgate, "dbefore": g.dbefore}
    if kind == "router":
        a = s["kept"] = ops.choose(s["z"], c["top_k"], mask=s["mask"], renormalize=c["renormalize"], out=kept)
        return {"idx": a.idx, "w": a.w, "counts": a.counts, "losses": a.losses}
    if kind == "router_grad":
        dz = s["kept"] = ops.choose_bwd(s["z"], s["idx"], s["counts"], s["dw"], s["dlosses"], mask=s["mask"],
                                        renormalize=c["renormalize"], out=kept)
        return dz
    if kept is None:
        kept = s["kept"] = ops.GradSet(s["grads"], out=s["out"])
    return {"stats": kept.clip(c["max_norm"], eps=CLIP_EPS, scale=c["scale"]), "grads": s["flat"]}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    kind = case["kind"]
    size = lambda what: 4 if case[what] == "fp32" else 2        # noqa: E731
    if kind in ("norm", "norm_grad"):
        t, d = case["tokens"] - case["padded"], case["width"]
        es, eo = size("stream"), size("dtype")
        full = eo if case["gate"] == "full" else 0
        if kind == "norm":
            # x and y in, h and r out
            per = es + (es + eo + full if case["join"] else 0) + (eo if case["before"] else 0)
            return {"bytes": t * d * per + 12 * d, "flops": 12.0 * t * d}
        # h, dh, y and dr in, dx and dy out
        per = 3 * es + (eo if case["before"] else 0) + (2 * eo + 2 * full if case["join"] else 0)
        return {"bytes": t * d * per + 24 * d, "flops": 30.0 * t * d}
    if kind in ("router", "router_grad"):
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        # logits in, choices and weights out; or logits, choices and weights' gradients in, logits' gradients out
        rows = t * e * size("dtype") * (1 if kind == "router" else 2)
        return {"bytes": rows + t * k * 8 + (t if case["masked"] else 0), "flops": 8.0 * t * e}
    n = sum(math.prod(x) for x in _shapes(case))
    return {"bytes": n * size("dtype") * 2, "flops": 3.0 * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, written apart from the plain forms
# ---------------------------------------------------------------------------
def _norm_exact(v, gain):
    return v / torch.sqrt((v ** 2).sum(1, keepdim=True) / v.shape[1] + EPS) * gain


def _through_norm(v, gain, dout):
    """Gradients of _norm_exact for v and for gain."""
    d = v.shape[1]
    rms = torch.sqrt((v ** 2).sum(1, keepdim=True) / d + EPS)
    inner = (dout * gain * v).sum(1, keepdim=True)
    return dout * gain / rms - v * inner / (d * rms ** 3), (dout * v / rms).sum(0)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("norm", "norm_grad"):
        n = case["tokens"] - case["padded"]
        up = lambda k: s[k].double()[:n]                            # noqa: E731
        whole = lambda v: torch.cat([v, v.new_zeros(case["padded"], v.shape[1])])       # noqa: E731
        gate = None
        if s["gate"] is not None:
            gate = s["gate"].double() if case["gate"] == "channel" else up("gate")
        if kind == "norm":
            out, h = {"h": None, "r": None}, up("x")
            if case["join"]:
                b = up("y")
                b = _norm_exact(b, s["after"].double()) if case["after"] else b
                b = b if gate is None else gate * b
                h = case["res_scale"] * h + case["out_scale"] * b
                out["h"] = whole(h)
            if case["before"]:
                out["r"] = whole(_norm_exact(h, s["before"].double()))
            return out
        out = dict.fromkeys(("dx", "dy", "dafter", "dgate", "dbefore"))
        g = up("dh")
        if case["before"]:
            back, out["dbefore"] = _through_norm(up("h"), s["before"].double(), up("dr"))
            g = g + back
        out["dx"] = whole(case["res_scale"] * g)
        if case["join"]:
            g = case["out_scale"] * g
            if gate is not None:
                b = _norm_exact(up("y"), s["after"].double()) if case["after"] else up("y")
                out["dgate"] = (g * b).sum(0) if case["gate"] == "channel" else \
                    whole((g * b).sum(1, keepdim=True) if case["gate"] == "token" else g * b)
                g = g * gate
            if case["after"]:
                g, out["dafter"] = _through_norm(up("y"), s["after"].double(), g)
            out["dy"] = whole(g)
        return out
    if kind in ("router", "router_grad"):
        z, e, k = s["z"].double(), case["experts"], case["top_k"]
        rank = torch.zeros_like(z)
        for j in range(e):
            col = z[:, j:j + 1]
            rank += (col > z) | ((col == z) & (j < torch.arange(e, device=z.device)))
        part = (z > -math.inf).any(1)
        if s["mask"] is not None:
            part &= s["mask"]
        taken = (rank < k) & (z > -math.inf) & part[:, None]
        n = max(1, int(part.sum()))
        zl = z[part]
        lse = torch.logsumexp(zl, 1)
        p = torch.zeros_like(z)
        p[part] = torch.exp(zl - lse[:, None])
        load = taken.sum(0).double()
        weight = torch.where(taken, p, 0.0)
        if case["renormalize"]:
            weight = weight / weight.sum(1, keepdim=True).clamp(min=1e-300)
        if kind == "router":
            w = torch.zeros((z.shape[0], k), dtype=z.dtype, device=z.device)
            r, c = torch.nonzero(taken, as_tuple=True)
            w[r, rank[r, c].long()] = weight[r, c]
            losses = torch.stack([e / (k * n * n) * (load * p.sum(0)).sum(), (lse ** 2).sum() / n])
            return {"idx": None, "w": w, "counts": None, "losses": losses}
        dw = torch.zeros_like(z)
        r, c = torch.nonzero(taken, as_tuple=True)
        dw[r, c] = s["dw"].double()[r, rank[r, c].long()]
        mean = (weight * dw).sum(1, keepdim=True)
        dz = weight * dw - (weight if case["renormalize"] else p) * mean
        l0, l1 = s["dlosses"].double().unbind()
        dz += l0 * e / (k * n * n) * (p * load - p * (p @ load)[:, None])
        dz[part] += l1 * 2 / n * lse[:, None] * p[part]
        return dz
    norm = abs(case["scale"]) * math.sqrt(math.fsum(float((g.double() ** 2).sum()) for g in s["grads"]))
    coef = min(1.0, case["max_norm"] / (norm + CLIP_EPS))
    return {"stats": torch.tensor([norm, coef], dtype=torch.float64, device="cuda"),
            "grads": torch.cat([torch.nn.functional.pad(g.double().reshape(-1) * (case["scale"] * coef), (0, 0 if case["packed"] else -g.numel() % 64))
                                for g in s["grads"]])}
