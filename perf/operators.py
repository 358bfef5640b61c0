"""The expert layer's stand-alone operators, case by case: what they take, what
they compute and what each cannot do without.

Three operators of a mixture-of-experts training step:

* route   - assignments (token, slot) sorted by expert into 128-row segments,
            the rows moved there and back with the routing weights applied,
            and the gradients of both moves;
* product - C = A B^T with A and B held in 8-bit floating point (e4m3), one
            power-of-two scale for each block of 128: dense, by expert over
            ragged rows, and as weight gradients reduced over ragged rows;
* swiglu  - the expert nonlinearity, its result quantised for the next product
            and its inputs kept as 8-bit checkpoints, and the backward pass
            that reads them.

``own`` false computes them in elementary torch operations, true by this
package's operators.
"""
import math

import torch

own = False

BLOCK = 128
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token of one sequence through the router's order, there and back: latency
        dict(name="route_token", kind="route", tokens=1, top_k=2, experts=16, width=768, dtype="bf16", skew=0.0, dropped=0.0),
        # the forward moves of a training microbatch of 32 x 1024 tokens
        dict(name="route_step", kind="route", tokens=32768, top_k=2, experts=16, width=768, dtype="bf16", skew=0.0, dropped=0.0),
        # the same microbatch's gradients
        dict(name="route_step_grad", kind="route_grad", tokens=32768, top_k=2, experts=16, width=768, dtype="bf16", skew=0.0, dropped=0.0),
        # many slots over many experts, a few of which take most tokens; fp32 rows
        dict(name="route_top8", kind="route", tokens=4096, top_k=8, experts=32, width=768, dtype="fp32", skew=1.1, dropped=0.0),
        # a padded batch: a third of the tokens go nowhere; odd counts and widths
        dict(name="route_odd_grad", kind="route_grad", tokens=1537, top_k=3, experts=7, width=100, dtype="fp32", skew=0.0, dropped=0.3),
        # the qkv projection of a single token
        dict(name="product_token", kind="product", rows=1, n=2304, k=768, top_k=1, experts=0, dtype="bf16", out="bf16", skew=0.0),
        # the output head over 2 x 1024 tokens
        dict(name="product_head", kind="product", rows=2048, n=32000, k=768, top_k=1, experts=0, dtype="bf16", out="bf16", skew=0.0),
        # gate and up projections of 16 experts over a microbatch, rows gathered from the tokens
        dict(name="product_experts", kind="product", rows=32768, n=1024, k=768, top_k=2, experts=16, dtype="bf16", out="bf16", skew=0.0),
        # the weight gradient of the same product, from the saved 8-bit rows
        dict(name="product_experts_grad", kind="wgrad", rows=32768, m=1024, n=768, top_k=2, experts=16, dtype="bf16", skew=0.0),
        # a single token's two expert rows, nothing saved
        dict(name="swiglu_token", kind="swiglu", rows=2, width=512, dtype="bf16", save=False),
        # a microbatch's expert rows with checkpoints
        dict(name="swiglu_step", kind="swiglu", rows=65536, width=512, dtype="bf16", save=True),
        # its backward pass from the checkpoints
        dict(name="swiglu_step_grad", kind="swiglu_grad", rows=65536, width=512, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number spread over the logarithm of lo..hi, odd ones among them."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["route", "route_grad", "product", "product", "wgrad", "swiglu", "swiglu_grad"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if kind in ("route", "route_grad"):
        top_k = rng.randint(1, 8)
        width = _spread(rng, 16, 1024)
        tokens = _spread(rng, 1, max(1, min(32768, (16384 * 768 * 2) // (top_k * width))))
        return dict(kind=kind, tokens=tokens, top_k=top_k, experts=rng.randint(top_k, 64), width=width, dtype=dtype,
                    skew=rng.choice([0.0, 1.1]), dropped=rng.choice([0.0, 0.0, 0.3]))
    if kind == "product":
        experts = rng.choice([0, 0, rng.randint(2, 32)])
        top_k = rng.randint(1, min(8, experts)) if experts else 1
        n = _spread(rng, 8, 2048 if experts else 32000)
        k = _spread(rng, 16, 2304)
        rows = _spread(rng, 1, max(1, min(32768, (1 << 34) // (n * k * top_k), (1 << 26) // (max(n, k) * top_k))))
        return dict(kind=kind, rows=rows, n=n, k=k, top_k=top_k, experts=experts, dtype=dtype,
                    out=rng.choice(["bf16", "fp32"]), skew=rng.choice([0.0, 0.5]) if experts else 0.0)
    if kind == "wgrad":
        experts = rng.randint(1, 32)
        top_k = rng.randint(1, min(8, experts))
        m, n = _spread(rng, 16, 1536), _spread(rng, 16, 1536)
        rows = _spread(rng, 1, max(1, min(32768, (1 << 34) // (m * n * top_k), (1 << 26) // ((m + n) * top_k))))
        return dict(kind=kind, rows=rows, m=m, n=n, top_k=top_k, experts=experts, dtype=dtype,
                    skew=rng.choice([0.0, 0.5]))
    width = 16 * _spread(rng, 1, 128)
    rows = _spread(rng, 1, max(1, min(65536, (32768 * 512) // width)))
    if kind == "swiglu":
        return dict(kind=kind, rows=rows, width=width, dtype=dtype, save=rng.choice([True, False]))
    return dict(kind=kind, rows=rows, width=width, dtype=dtype)


# ---------------------------------------------------------------------------
# the operators' plain forms, in 32 bits
# ---------------------------------------------------------------------------
def _rows_max(assignments, experts):
    """Rows that any routing of so many assignments fits in, segments padded to 128."""
    return -(-(assignments + experts * (BLOCK - 1)) // BLOCK) * BLOCK


def _order(idx, experts):
    """Segment starts, the assignment at each row (-1: none), the row of each assignment (-1: none)."""
    a = idx.reshape(-1).to(torch.int32)
    hit = a == torch.arange(experts, device=a.device, dtype=torch.int32)[:, None]
    rank = hit.to(torch.int32).cumsum(1, dtype=torch.int32)
    padded = (rank[:, -1] + (BLOCK - 1)) // BLOCK * BLOCK
    offs = torch.zeros(experts + 1, dtype=torch.int32, device=a.device)
    offs[1:] = padded.cumsum(0, dtype=torch.int32)
    kept = a >= 0
    row = torch.where(kept, offs[a.clamp(min=0)] + (rank * hit).sum(0, dtype=torch.int32) - 1, -1)
    rows = _rows_max(a.numel(), experts)
    perm = torch.full((rows + 1,), -1, dtype=torch.int32, device=a.device)
    perm[torch.where(kept, row, rows).long()] = torch.arange(a.numel(), dtype=torch.int32, device=a.device)
    return offs, perm[:rows].contiguous(), row.reshape(idx.shape)


def _dispatch(x, perm, top_k):
    return torch.where((perm >= 0)[:, None], x[(perm.clamp(min=0) // top_k).long()], torch.zeros((), dtype=x.dtype, device=x.device))


def _combine(y, row, w):
    g = y[row.clamp(min=0).long()].float()
    if w is not None:
        g = g * w[:, :, None]
    return torch.where((row >= 0)[:, :, None], g, 0.0).sum(1).to(y.dtype)


def _exponents(amax):
    """The least e >= -126 with amax <= 448 * 2^e; 0 for a block of zeros."""
    m, ex = torch.frexp(amax)
    e = (ex - 9 + (m > 0.875).to(ex.dtype)).clamp(min=-126)
    return torch.where(amax > 0, e, 0)


def _two(e):
    """2^e for whole e of -126..127, as fp32."""
    return ((e + 127).to(torch.int32) << 23).view(torch.float32)


def _codes(x, e):
    """e4m3 codes of x [..., 128] under one exponent for the last axis, as numbers."""
    return (x * _two(-e)[..., None]).to(torch.float8_e4m3fn)


def _blocks(x, axis_pad):
    """The last axis padded with zeros to whole blocks of 128 and split."""
    short = -x.shape[-1] % BLOCK
    if short and axis_pad:
        x = torch.nn.functional.pad(x, (0, short))
    return x.unflatten(-1, (-1, BLOCK))


def _values(x):
    """What x holds after quantisation in blocks of 1 x 128 along its last axis."""
    b = _blocks(x.float(), True)
    e = _exponents(b.abs().amax(-1))
    v = _codes(b, e).float() * _two(e)[..., None]
    return v.flatten(-2)[..., :x.shape[-1]]


def _restored(codes, scales, cols):
    """The values that 8-bit codes [..., R, ld] with scale bytes [..., R, blocks] stand for."""
    v = _blocks(codes[..., :cols].view(torch.float8_e4m3fn).float(), True)
    v = v * _two(scales.to(torch.int32) - 127)[..., None]
    return v.flatten(-2)[..., :cols]


def _restored_weights(codes, scales, cols):
    """The same for weights [E, N, ld] with one scale byte for each 128 x 128 block."""
    per_row = scales.repeat_interleave(BLOCK, dim=-2)[..., :codes.shape[-2], :]
    return _restored(codes, per_row, cols)


def _by_expert(offs, longest, rows):
    """Row numbers [E, longest] of the segments, and which of them are inside."""
    at = offs[:-1, None].long() + torch.arange(longest, device=offs.device)
    inside = at < offs[1:, None]
    return torch.where(inside, at, rows), inside


def _swiglu(g, u):
    return g * torch.sigmoid(g) * u


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(gen, shape, std, dtype=torch.float32):
    return (torch.randn(shape, generator=gen, device=gen.device, dtype=torch.float32) * std).to(dtype)


def _choices(gen, tokens, top_k, experts, skew, dropped):
    """Distinct experts per token, best first: scores plus noise; a share of the tokens go nowhere (-1)."""
    score = -skew * torch.log(torch.arange(1, experts + 1, device=gen.device, dtype=torch.float32))
    u = torch.rand((tokens, experts), generator=gen, device=gen.device).clamp(1e-9, 1 - 1e-7)
    idx = (score - torch.log(-torch.log(u))).topk(top_k, dim=1).indices.to(torch.int32)
    if dropped:
        idx = torch.where(torch.rand((tokens, 1), generator=gen, device=gen.device) < dropped, -1, idx)
    return idx.contiguous()


def _hidden(gen, shape, dtype):
    """Normalised hidden rows: unit normal, a few channels several times larger."""
    gain = 1.0 + 4.0 * (torch.rand(shape[-1], generator=gen, device=gen.device) < 0.01).float()
    return (torch.randn(shape, generator=gen, device=gen.device) * gain).to(dtype)


def _held(x):
    """x [R, C] as 8-bit codes [R, C up to 16] and scale bytes [R, blocks], as a program holds it."""
    b = _blocks(x.float(), True)
    e = _exponents(b.abs().amax(-1))
    q = _codes(b, e).view(torch.uint8).flatten(-2)
    return q[..., :-(-x.shape[-1] // 16) * 16].contiguous(), (e + 127).to(torch.uint8)


def _held_weights(w):
    """w [E, N, K] as 8-bit codes [E, N, K up to 16] and one scale byte for each 128 x 128 block."""
    experts, n, k = w.shape
    p = torch.nn.functional.pad(w, (0, -k % BLOCK, 0, -n % BLOCK)).unflatten(2, (-1, BLOCK)).unflatten(1, (-1, BLOCK))
    e = _exponents(p.abs().amax((2, 4)))
    q = (p * _two(-e)[:, :, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    q = q.flatten(3).flatten(1, 2)[:, :n, :-(-k // 16) * 16].contiguous()
    return q, (e + 127).to(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev, kind = gen.device, case["kind"]
    dt = TYPES[case["dtype"]]
    s = {"case": case}
    if kind in ("route", "route_grad"):
        t, k, e, d = case["tokens"], case["top_k"], case["experts"], case["width"]
        rows = _rows_max(t * k, e)
        s["idx"] = _choices(gen, t, k, e, case["skew"], case["dropped"])
        s["w"] = torch.softmax(torch.randn((t, k), generator=gen, device=dev), 1)
        s["y"] = _normal(gen, (rows, d), 0.5, dt)
        if kind == "route":
            s["x"] = _hidden(gen, (t, d), dt)
            s["xs"] = torch.zeros((rows, d), dtype=dt, device=dev)
        else:
            s["offs"], s["perm"], s["row"] = _order(s["idx"], e)
            s["dout"] = _normal(gen, (t, d), 1e-3, dt)
            s["dxs"] = _normal(gen, (rows, d), 1e-3, dt)
            s["dy"] = torch.zeros((rows, d), dtype=dt, device=dev)
    elif kind == "product":
        t, n, k, e = case["rows"], case["n"], case["k"], case["experts"]
        s["x"] = _hidden(gen, (t, k), dt)
        s["b"], s["b_scales"] = _held_weights(_normal(gen, (max(1, e), n, k), 0.02))
        rows = t
        if e:
            idx = _choices(gen, t, case["top_k"], e, case["skew"], 0.0)
            s["offs"], s["perm"], s["row"] = _order(idx, e)
            s["longest"] = int((s["offs"][1:] - s["offs"][:-1]).max())
            rows = s["perm"].numel()
        s["c"] = torch.zeros((rows, n), dtype=TYPES[case["out"]], device=dev)
    elif kind == "wgrad":
        idx = _choices(gen, case["rows"], case["top_k"], case["experts"], case["skew"], 0.0)
        s["offs"], perm, _ = _order(idx, case["experts"])
        s["longest"] = int((s["offs"][1:] - s["offs"][:-1]).max())
        real = (perm >= 0).float()[:, None]
        s["dy"] = (_normal(gen, (perm.numel(), case["m"]), 1e-3) * real).to(dt)
        s["x"], s["x_scales"] = _held(_hidden(gen, (perm.numel(), case["n"]), torch.float32) * real)
        s["c"] = torch.zeros((case["experts"], case["m"], case["n"]), dtype=torch.float32, device=dev)
    else:
        r, f = case["rows"], case["width"]
        gu = _normal(gen, (r, 2 * f), 1.0, dt)
        if kind == "swiglu":
            s["gu"] = gu
        else:
            (qg, sg), (qu, su) = _held(gu[:, :f]), _held(gu[:, f:])
            s["saved"], s["saved_scales"] = torch.cat([qg, qu], 1), torch.cat([sg, su], 1)
            s["dact"] = _normal(gen, (r, f), 1e-3, dt)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    kind = c["kind"]
    if kind == "route":
        offs, perm, row = _order(state["idx"], c["experts"])
        xs = _dispatch(state["x"], perm, c["top_k"])
        return {"offs": offs, "perm": perm, "row": row, "xs": xs, "out": _combine(state["y"], row, state["w"])}
    if kind == "route_grad":
        perm, row, w, dout = state["perm"], state["row"], state["w"], state["dout"]
        at = (perm.clamp(min=0) // c["top_k"]).long()
        dy = torch.where((perm >= 0)[:, None], w.reshape(-1)[perm.clamp(min=0).long()][:, None] * dout[at].float(), 0.0)
        dw = (dout.float()[:, None, :] * state["y"][row.clamp(min=0).long()].float()).sum(-1)
        return {"dy": dy.to(dout.dtype), "dw": torch.where(row >= 0, dw, 0.0), "dx": _combine(state["dxs"], row, None)}
    if kind == "product":
        b = _restored_weights(state["b"], state["b_scales"], c["k"])
        x = _values(state["x"])
        if not c["experts"]:
            return (x @ b[0].T).to(TYPES[c["out"]])
        xs = _dispatch(x, state["perm"], c["top_k"])
        rows = xs.shape[0]
        at, inside = _by_expert(state["offs"], state["longest"], rows)
        part = torch.where(inside[:, :, None], xs[at.clamp(max=rows - 1)], 0.0) @ b.transpose(1, 2)
        full = torch.zeros((rows + 1, c["n"]), device=part.device)
        full[at.reshape(-1)] = part.reshape(-1, c["n"])
        full[rows] = 0.0
        return full[:rows].to(TYPES[c["out"]])
    if kind == "wgrad":
        rows = state["dy"].shape[0]
        dy = _values(state["dy"].float().T.contiguous())
        x = _values(_restored(state["x"], state["x_scales"], c["n"]).T.contiguous())
        at, inside = _by_expert(state["offs"], state["longest"], rows)
        at = at.clamp(max=rows - 1)
        a = torch.where(inside, dy[:, at], 0.0).permute(1, 0, 2)
        b = torch.where(inside, x[:, at], 0.0).permute(1, 2, 0)
        return a @ b
    f = c["width"]
    if kind == "swiglu":
        g, u = state["gu"][:, :f].float(), state["gu"][:, f:].float()
        out = {"act": _values(_swiglu(g, u)).to(torch.bfloat16)}
        if c["save"]:
            out["saved"] = torch.cat([_values(g), _values(u)], 1).to(torch.bfloat16)
        return out
    blocks = state["saved_scales"].shape[1] // 2
    g = _restored(state["saved"][:, :f], state["saved_scales"][:, :blocks], f)
    u = _restored(state["saved"][:, f:], state["saved_scales"][:, blocks:], f)
    sig, da = torch.sigmoid(g), state["dact"].float()
    dgu = torch.cat([da * u * sig * (1 + g * (1 - sig)), da * g * sig], 1)
    return {"dgu": dgu.to(state["dact"].dtype), "act": (g * sig * u).to(state["dact"].dtype)}


def _run_own(state):
    """The calls of a program that keeps its buffers (made at its first step)."""
    from adamw_persistent_sm_gb300 import expert_ops as ops
    c = state["case"]
    kind = c["kind"]
    kept = state.get("kept")
    if kind == "route":
        if kept is None:
            kept = state["kept"] = (ops.Route(c["tokens"], c["top_k"], c["experts"], "cuda"), torch.empty_like(state["x"]))
        r, out = kept
        r.order(state["idx"])
        r.dispatch(state["x"], out=state["xs"])
        r.combine(state["y"], state["w"], out=out)
        return {"offs": r.offs, "perm": r.perm, "row": r.row, "xs": state["xs"], "out": out}
    if kind == "route_grad":
        if kept is None:
            r = ops.Route.of(state["offs"], state["perm"], state["row"])
            kept = state["kept"] = (r, torch.empty_like(state["w"]), torch.empty_like(state["dout"]))
        r, dw, dx = kept
        r.combine_bwd(state["dout"], state["y"], state["w"], dy=state["dy"], dw=dw)
        r.dispatch_bwd(state["dxs"], out=dx)
        return {"dy": state["dy"], "dw": dw, "dx": dx}
    if kind == "product":
        if kept is None:
            b = ops.Tensor8(state["b"], state["b_scales"], c["k"], 128)
            r = ops.Route.of(state["offs"], state["perm"], state["row"]) if c["experts"] else None
            kept = state["kept"] = (r, ops.empty8(state["c"].shape[0], c["k"], "cuda"), b if r else b[0])
        r, a, b = kept
        if r is None:
            ops.quant8(state["x"], out=a)
            return ops.gemm8(a, b, out=state["c"])
        r.dispatch8(state["x"], out=a)
        return ops.gemm8(a, b, out=state["c"], offs=r.offs)
    if kind == "wgrad":
        if kept is None:
            rows = state["dy"].shape[0]
            x = ops.Tensor8(state["x"], state["x_scales"], c["n"], 1)
            kept = state["kept"] = (x, ops.empty8(c["m"], rows, "cuda"), ops.empty8(c["n"], rows, "cuda"))
        x, dyt, xt = kept
        ops.quant8_t(state["dy"], out=dyt, n_rows=state["offs"][-1:])
        ops.quant8_t(x, out=xt, n_rows=state["offs"][-1:])
        return ops.gemm8_reduce(dyt, xt, out=state["c"], offs=state["offs"])
    r, f = c["rows"], c["width"]
    if kind == "swiglu":
        if kept is None:
            save = (ops.empty8(r, 2 * f, "cuda", halves=True), torch.empty((r, 2 * f), dtype=torch.bfloat16, device="cuda")) if c["save"] else (None, None)
            kept = state["kept"] = (ops.empty8(r, f, "cuda"), torch.empty((r, f), dtype=torch.bfloat16, device="cuda"), *save)
        act8, act, saved8, saved = kept
        ops.swiglu8(state["gu"], act=act8, saved=saved8)
        out = {"act": ops.dequant8(act8, out=act)}
        if saved is not None:
            out["saved"] = ops.dequant8(saved8, out=saved)
        return out
    if kept is None:
        saved8 = ops.Tensor8(state["saved"], state["saved_scales"], 2 * f, 1, halves=True)
        kept = state["kept"] = (saved8, torch.empty((r, 2 * f), dtype=state["dact"].dtype, device="cuda"), torch.empty_like(state["dact"]))
    saved8, dgu, act = kept
    ops.swiglu8_bwd(state["dact"], saved8, dgu=dgu, act=act)
    return {"dgu": dgu, "act": act}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    kind = case["kind"]
    es = 4 if case["dtype"] == "fp32" else 2
    if kind in ("route", "route_grad"):
        t, k, d = case["tokens"], case["top_k"], case["width"]
        r = t * k * (1.0 - case["dropped"])
        if kind == "route":
            # choices in; starts, assignments and rows out; x in, its copies out; y in, weights in, sums out
            return {"bytes": t * k * 4 + _rows_max(t * k, case["experts"]) * 4 + t * k * 8 + es * d * (2 * t + 2 * r), "flops": 2 * r * d}
        return {"bytes": t * k * 16 + es * d * (2 * t + 3 * r), "flops": 4 * r * d}
    if kind == "product":
        t, n, k, e = case["rows"], case["n"], case["k"], case["experts"]
        r = t * case["top_k"]
        # x in, weights in, C out (the 8-bit rows between the two steps need not reach memory)
        return {"bytes": es * t * k + max(1, e) * n * k + (4 if case["out"] == "fp32" else 2) * r * n, "flops": 2.0 * r * n * k}
    if kind == "wgrad":
        r = case["rows"] * case["top_k"]
        return {"bytes": r * (es * case["m"] + case["n"]) + 4 * case["experts"] * case["m"] * case["n"], "flops": 2.0 * r * case["m"] * case["n"]}
    r, f = case["rows"], case["width"]
    if kind == "swiglu":
        # g and u in; 8-bit results out and restored as bf16
        held = r * f * (3 if case["save"] else 1)
        return {"bytes": 2 * r * f * es + held + 2 * held, "flops": 8.0 * r * f}
    return {"bytes": r * f * (es + 2 + 3 * es), "flops": 16.0 * r * f}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, written apart from the plain forms
# ---------------------------------------------------------------------------
def _power(e):
    """2^e for whole doubles e, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _e4m3(v):
    """Nearest e4m3 value, ties to even, of doubles within +-448: steps of 2^(exponent - 3), 2^-9 at the bottom."""
    _, ex = torch.frexp(v)
    step = _power((ex - 1).clamp(min=-6) - 3)
    return torch.round(v / step) * step


def _held_exact(v):
    """Values of v [R, C] (double) after quantisation in 1 x 128 blocks along C."""
    rows, cols = v.shape
    out = torch.empty_like(v)
    for c0 in range(0, cols, BLOCK):
        b = v[:, c0:c0 + BLOCK]
        top = b.abs().max(1, keepdim=True).values
        e = torch.ceil(torch.log2(torch.where(top > 0, top, 448.0) / 448.0))
        e = torch.where(top > 448.0 * _power(e), e + 1, e)
        e = torch.where(top <= 448.0 * _power(e - 1), e - 1, e).clamp(min=-126.0)
        scale = _power(torch.where(top > 0, e, 0.0))
        out[:, c0:c0 + BLOCK] = _e4m3(b / scale) * scale
    return out


def _unheld(codes, scales, cols, block_rows=1):
    """Doubles that e4m3 codes [R, ld] with scale bytes stand for."""
    b = codes[:, :cols].to(torch.int64)
    ex, m = (b >> 3) & 15, (b & 7).double()
    v = torch.where(ex > 0, (8 + m) * _power(ex - 10), m * 2.0 ** -9)
    v = torch.where(b >= 128, -v, v)
    r = torch.arange(codes.shape[0], device=b.device) // block_rows
    c = torch.arange(cols, device=b.device) // BLOCK
    return v * _power(scales.to(torch.int64)[r][:, c] - 127)


def _order_exact(idx, experts):
    a = idx.reshape(-1).long()
    n = torch.stack([(a == e).sum() for e in range(experts)]).tolist()
    offs = [0]
    for e in range(experts):
        offs.append(offs[-1] + -(-n[e] // BLOCK) * BLOCK)
    row = torch.full_like(a, -1)
    perm = torch.full((_rows_max(a.numel(), experts),), -1, dtype=torch.int64, device=a.device)
    for e in range(experts):
        at = torch.nonzero(a == e)[:, 0]
        row[at] = torch.arange(n[e], device=a.device) + offs[e]
        perm[offs[e]:offs[e] + n[e]] = at
    return offs, perm, row.reshape(idx.shape)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("route", "route_grad"):
        offs, perm, row = _order_exact(s["idx"], case["experts"])
        real, k = perm >= 0, case["top_k"]
        token = perm[real] // k
        move = torch.zeros(s["y"].shape, dtype=torch.float64, device=perm.device)
        w = s["w"].double()
        back = torch.zeros((case["tokens"], case["width"]), dtype=torch.float64, device=perm.device)
        if kind == "route":
            move[real] = s["x"].double()[token]
            back.index_add_(0, token, s["y"].double()[real] * w.reshape(-1)[perm[real]][:, None])
            return {"offs": None, "perm": None, "row": None, "xs": move, "out": back}
        move[real] = s["dout"].double()[token] * w.reshape(-1)[perm[real]][:, None]
        dw = torch.zeros(w.numel(), dtype=torch.float64, device=perm.device)
        dw[perm[real]] = (s["dout"].double()[token] * s["y"].double()[real]).sum(1)
        back.index_add_(0, token, s["dxs"].double()[real])
        return {"dy": move, "dw": dw.reshape(w.shape), "dx": back}
    if kind == "product":
        x = _held_exact(s["x"].double())
        out = torch.zeros(s["c"].shape, dtype=torch.float64, device=x.device)
        if not case["experts"]:
            out.copy_(x @ _unheld(s["b"][0], s["b_scales"][0], case["k"], BLOCK).T)
            return out
        offs, perm = s["offs"].tolist(), s["perm"].long()
        for e in range(case["experts"]):
            b = _unheld(s["b"][e], s["b_scales"][e], case["k"], BLOCK)
            p = perm[offs[e]:offs[e + 1]]
            rows = torch.nonzero(p >= 0)[:, 0]
            out[offs[e] + rows] = x[p[rows] // case["top_k"]] @ b.T
        return out
    if kind == "wgrad":
        offs = s["offs"].tolist()
        dy = _held_exact(s["dy"].double().T.contiguous())
        x = _held_exact(_unheld(s["x"], s["x_scales"], case["n"]).T.contiguous())
        return torch.stack([dy[:, a:b] @ x[:, a:b].T for a, b in zip(offs, offs[1:])])
    f = case["width"]
    if kind == "swiglu":
        g, u = s["gu"][:, :f].double(), s["gu"][:, f:].double()
        out = {"act": _held_exact(g / (1 + torch.exp(-g)) * u)}
        if case["save"]:
            out["saved"] = torch.cat([_held_exact(g), _held_exact(u)], 1)
        return out
    nb = s["saved_scales"].shape[1] // 2
    g = _unheld(s["saved"][:, :f], s["saved_scales"][:, :nb], f)
    u = _unheld(s["saved"][:, f:], s["saved_scales"][:, nb:], f)
    da, p = s["dact"].double(), 1 / (1 + torch.exp(-g))
    return {"dgu": torch.cat([da * u * (p + g * p * (1 - p)), da * g * p], 1), "act": g * p * u}
