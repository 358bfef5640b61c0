"""The operators around the expert layer on the GPU against their definitions in
float64 (tests/block_ref.py), within bounds derived there from the order of the
kernels' additions (U = 2^-24 per fp32 operation), half a step for the rounding to
the output type."""
import math

import numpy as np
import pytest
import torch

import block_ref as R

pytestmark = pytest.mark.gpu

U = R.U
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
EPS = 1e-5


@pytest.fixture(scope="module")
def ops():
    from adamw_persistent_sm_gb300 import block_ops
    return block_ops


def as64(t):
    return t.detach().cpu().double().numpy()


def rnd(seed, *shape, std=1.0, mean=0.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std + mean).to(dtype).cuda()


def strided(t, pad, shift=0):
    """t as a view of a wider buffer: rows `pad` elements further apart, starting `shift` in."""
    buf = torch.full((t.shape[0], t.shape[1] + pad + shift), float("nan"), dtype=t.dtype, device=t.device)
    v = buf[:, shift:shift + t.shape[1]]
    v.copy_(t)
    return v


def close(got, want, bound, what=""):
    dtype, got = got.dtype, as64(got)
    # a value beyond the type is infinite there: the square of the lowest logit is (3.4e38)^2 = 1.2e77 > 3.4e38
    want = np.where(np.abs(want) > torch.finfo(dtype).max, np.copysign(np.inf, want), want)
    assert np.array_equal(np.isnan(want), np.isnan(got)) and np.array_equal(np.isinf(want), np.isinf(got)), what
    f = np.isfinite(want)
    # half a step of the output, at the value or at what the bound lets it be
    lim = np.broadcast_to(bound, want.shape)[f] * 1.01 + HALF[dtype] * np.abs(want[f]) * 1.01 + 1e-44
    off = np.abs(got[f] - want[f])
    bad = off > lim
    assert not bad.any(), (what, int(bad.sum()), float(off[bad].max()), np.argwhere(f)[bad][:4].tolist(), got[f][bad][:4], want[f][bad][:4])


# ---------------------------------------------------------------------------
# the joint
# ---------------------------------------------------------------------------
def make_gate(kind, t, d, dtype, seed=9):
    return {"none": None, "channel": rnd(seed, d, std=0.5), "token": rnd(seed, t, 1), "full": rnd(seed, t, d, dtype=dtype)}[kind]


def as_row(v, kind=None):
    """A vector or gate for the definition, which broadcasts."""
    return None if v is None else as64(v).reshape(1, -1) if v.dim() == 1 else as64(v)


def joint_inputs(t, d, stream, dtype, gate, after=True, before=True):
    st, dt = DT[stream], DT[dtype]
    return dict(x=rnd(1, t, d, dtype=st), y=rnd(2, t, d, std=0.5, dtype=dt), gate=make_gate(gate, t, d, dt),
                after=rnd(3, d, std=0.2, mean=1.0) if after else None, before=rnd(4, d, std=0.2, mean=1.0) if before else None)


def check_joint(ops, p, a, b, **kw):
    h, r = ops.block_norm(p["x"], p["y"], after=p["after"], gate=p["gate"], before=p["before"], res_scale=a, out_scale=b,
                          eps=EPS, **kw)
    want = R.joint(as64(p["x"]), as64(p["y"]), as_row(p["after"]), as_row(p["gate"]), as_row(p["before"]), a, b, EPS)
    close(h, want[0], want[2], "h")
    if r is not None:
        close(r, want[1], want[3], "r")
    return h, r


def check_joint_grad(ops, p, dr, dh, h, a, b, **kw):
    got = ops.block_norm_bwd(dr, dh, h, p["y"], after=p["after"], gate=p["gate"], before=p["before"], res_scale=a,
                             out_scale=b, eps=EPS, **kw)
    want = R.joint_grad(None if dr is None else as64(dr), None if dh is None else as64(dh), as64(h),
                        None if p["y"] is None else as64(p["y"]), as_row(p["after"]), as_row(p["gate"]), as_row(p["before"]), a, b, EPS)
    for name in ("dx", "dy", "dgate", "dafter", "dbefore"):
        g = getattr(got, name)
        if name not in want:
            assert g is None, name
            continue
        v, e = want[name]
        if g.dim() == 1:
            v, e = R.row_sum(v, e)
        elif g.shape[1] == 1 and v.shape[1] > 1:
            v, e = v.sum(1, keepdims=True), e.sum(1, keepdims=True) + R.D * U * np.abs(v).sum(1, keepdims=True)
        close(g, v, e, name)
    return got


TYPES = [("fp32", "bf16"), ("bf16", "bf16"), ("fp32", "fp32")]
WIDTHS = [1, 7, 8, 33, 100, 256, 264, 768, 1001, 1024, 1032, 2048, 2056, 4095, 4096, 4104, 8191, 8192]


@pytest.mark.parametrize("stream,dtype", TYPES)
@pytest.mark.parametrize("d", WIDTHS)
def test_joint_widths(ops, d, stream, dtype):
    for t, gate in ((1, "channel"), (37, "none"), (5, "full")):
        p = joint_inputs(t, d, stream, dtype, gate)
        h, _ = check_joint(ops, p, 1.0, 0.5)
        dr, dh = rnd(5, t, d, std=0.01, dtype=DT[dtype]), rnd(6, t, d, std=0.01, dtype=DT[stream])
        check_joint_grad(ops, p, dr, dh, h, 1.0, 0.5)


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("after,before", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("t,d", [(1, 768), (700, 768), (2000, 264), (310, 2304), (40, 5000), (333, 101)])
def test_joint_forms(ops, t, d, after, before, gate):
    """Every part present or not, rows enough for several per group of warps."""
    p = joint_inputs(t, d, "fp32", "bf16", gate, after, before)
    h, _ = check_joint(ops, p, 0.75, 1.25)
    dr = rnd(5, t, d, std=0.01, dtype=torch.bfloat16) if before else None
    check_joint_grad(ops, p, dr, rnd(6, t, d, std=0.01), h, 0.75, 1.25)
    if before:
        check_joint_grad(ops, p, dr, None, h, 0.75, 1.25)


@pytest.mark.parametrize("stream,dtype", TYPES)
@pytest.mark.parametrize("t,d", [(1, 768), (900, 768), (3, 4104), (50, 77)])
def test_norm_before_the_first_block(ops, t, d, stream, dtype):
    x, w = rnd(1, t, d, dtype=DT[stream]), rnd(4, d, mean=1.0)
    h, r = ops.block_norm(x, before=w, eps=EPS, dtype=DT[dtype])
    assert h is x and r.dtype is DT[dtype]
    _, want, _, bound = R.joint(as64(x), None, None, None, as_row(w), 1.0, 1.0, EPS)
    close(r, want, bound)
    p = dict(x=x, y=None, gate=None, after=None, before=w)
    check_joint_grad(ops, p, rnd(5, t, d, dtype=DT[dtype]), rnd(6, t, d, dtype=DT[stream]), x, 1.0, 1.0)


@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (3, 0), (0, 1), (4, 4)])
@pytest.mark.parametrize("d", [768, 104])
def test_joint_views(ops, d, pad, shift):
    """Rows of any stride and alignment, in and out; what lies between them stays."""
    t = 70
    p = joint_inputs(t, d, "fp32", "bf16", "full")
    v = {k: strided(q, pad, shift) if q is not None and q.dim() == 2 else q for k, q in p.items()}
    outs = [strided(torch.zeros(t, d, dtype=q, device="cuda"), pad, shift) for q in (torch.float32, torch.bfloat16)]
    h, r = check_joint(ops, v, 1.0, 0.5, h=outs[0], r=outs[1])
    assert h is outs[0] and r is outs[1]
    dr, dh = strided(rnd(5, t, d, dtype=torch.bfloat16), pad, shift), strided(rnd(6, t, d), pad, shift)
    grads = [strided(torch.zeros(t, d, dtype=q, device="cuda"), pad, shift) for q in (torch.float32, torch.bfloat16, torch.bfloat16)]
    check_joint_grad(ops, v, dr, dh, h, 1.0, 0.5, dx=grads[0], dy=grads[1], dgate=grads[2])
    for q in outs + grads:
        if pad + shift:
            rest = torch.ones(q._base.shape[1], dtype=torch.bool)
            rest[shift:shift + d] = False
            assert q._base[:, rest.cuda()].isnan().all()


def test_gains_off_their_boundary(ops):
    t, d = 9, 256
    p = joint_inputs(t, d, "fp32", "bf16", "channel")
    for k in ("after", "before", "gate"):
        q = dict(p)
        q[k] = torch.cat([p[k][:1], p[k]])[1:]
        h, _ = check_joint(ops, q, 1.0, 1.0)
        check_joint_grad(ops, q, rnd(5, t, d, dtype=torch.bfloat16), None, h, 1.0, 1.0)


@pytest.mark.parametrize("gate", ["channel", "token", "full"])
@pytest.mark.parametrize("live", [-3, 0, 1, 29, 200, 1 << 30])
@pytest.mark.parametrize("d", [100, 768, 1500])
def test_rows_behind_the_last_are_left(ops, d, live, gate):
    t = 200
    n = min(max(live, 0), t)
    p = joint_inputs(t, d, "fp32", "bf16", gate)
    for k in ("x", "y"):
        p[k][n:] = float("nan")
    lim = torch.tensor([live], dtype=torch.int32, device="cuda")
    h, r = torch.full((t, d), 7.0, device="cuda"), torch.full((t, d), 7.0, dtype=torch.bfloat16, device="cuda")
    ops.block_norm(p["x"], p["y"], after=p["after"], gate=p["gate"], before=p["before"], h=h, r=r, n_rows=lim)
    cut = {k: v[:n] if v is not None and v.dim() == 2 else v for k, v in p.items()}
    assert (h[n:] == 7).all() and (r[n:] == 7).all()
    dr, dh = rnd(5, t, d, dtype=torch.bfloat16), rnd(6, t, d)
    dr[n:], dh[n:] = float("nan"), float("nan")
    out = dict(dx=torch.full((t, d), 7.0, device="cuda"), dy=torch.full((t, d), 7.0, dtype=torch.bfloat16, device="cuda"))
    if gate != "channel":
        out["dgate"] = torch.full_like(p["gate"], 7.0)
    got = ops.block_norm_bwd(dr, dh, h, p["y"], after=p["after"], gate=p["gate"], before=p["before"], n_rows=lim, **out)
    assert all((v[n:] == 7).all() for v in out.values())
    if n == 0:
        assert (got.dafter == 0).all() and (got.dbefore == 0).all() and (gate != "channel" or (got.dgate == 0).all())
        return
    h2, r2 = ops.block_norm(cut["x"], cut["y"], after=p["after"], gate=cut["gate"], before=p["before"])
    assert torch.equal(h[:n], h2) and torch.equal(r[:n], r2)
    check_joint_grad(ops, cut, dr[:n].contiguous(), dh[:n].contiguous(), h2, 1.0, 1.0)
    want = ops.block_norm_bwd(dr[:n].contiguous(), dh[:n].contiguous(), h2, cut["y"], after=p["after"], gate=cut["gate"], before=p["before"])
    assert torch.equal(got.dx[:n], want.dx) and torch.equal(got.dy[:n], want.dy)
    R_, B_ = R.row_sum(*[np.abs(v) for v in R.joint_grad(as64(dr[:n]), as64(dh[:n]), as64(h2), as64(cut["y"]), as_row(p["after"]),
                                                         as_row(cut["gate"]), as_row(p["before"]), 1.0, 1.0, EPS)["dbefore"]])
    assert (np.abs(as64(got.dbefore) - as64(want.dbefore)) <= 2 * B_).all()


def test_no_rows(ops):
    p = joint_inputs(0, 64, "fp32", "bf16", "channel")
    h, r = ops.block_norm(p["x"], p["y"], after=p["after"], gate=p["gate"], before=p["before"])
    assert h.shape == r.shape == (0, 64)
    g = ops.block_norm_bwd(r, h, h, p["y"], after=p["after"], gate=p["gate"], before=p["before"])
    assert all((v == 0).all() for v in (g.dafter, g.dgate, g.dbefore))
    held = [torch.full((64,), 2.0, device="cuda") for _ in range(3)]
    ops.block_norm_bwd(r, h, h, p["y"], after=p["after"], gate=p["gate"], before=p["before"], dafter=held[0], dgate=held[1],
                       dbefore=held[2], accumulate=True)
    assert all((v == 2).all() for v in held)
    for gate in ("token", "full"):
        q = joint_inputs(0, 64, "fp32", "bf16", gate)
        h, r = ops.block_norm(q["x"], q["y"], gate=q["gate"], before=q["before"])
        ops.block_norm_bwd(r, h, h, q["y"], gate=q["gate"], before=q["before"])


def test_joint_accumulates(ops):
    t, d = 400, 768
    p = joint_inputs(t, d, "fp32", "bf16", "channel")
    h, _ = check_joint(ops, p, 1.0, 1.0)
    dr, dh = rnd(5, t, d, dtype=torch.bfloat16), rnd(6, t, d)
    kw = dict(after=p["after"], gate=p["gate"], before=p["before"])
    once = ops.block_norm_bwd(dr, dh, h, p["y"], **kw)
    held = {k: rnd(20 + i, d) for i, k in enumerate(("dafter", "dgate", "dbefore"))}
    before = {k: v.clone() for k, v in held.items()}
    got = ops.block_norm_bwd(dr, dh, h, p["y"], **kw, **held, accumulate=True)
    for k in held:
        assert getattr(got, k) is held[k] and torch.equal(held[k], before[k] + getattr(once, k))
    with pytest.raises(ValueError):
        ops.block_norm_bwd(dr, dh, h, p["y"], **kw, dafter=held["dafter"], dbefore=held["dbefore"], accumulate=True)


@pytest.mark.parametrize("d", [64, 768, 1001, 4104])
def test_few_rows_accumulate_and_end_early(ops, d):
    """As few rows as one CTA takes: sums added to what is there, rows behind the last left as they were."""
    t = 2
    p = joint_inputs(t, d, "fp32", "bf16", "channel")
    kw = dict(after=p["after"], gate=p["gate"], before=p["before"])
    h, _ = check_joint(ops, p, 1.0, 1.0)
    dr, dh = rnd(5, t, d, dtype=torch.bfloat16), rnd(6, t, d)
    once = ops.block_norm_bwd(dr, dh, h, p["y"], **kw)
    for live in (0, 1, 2, 5):
        lim = torch.tensor([live], dtype=torch.int32, device="cuda")
        n = min(live, t)
        cut = {k: v[:n] if v is not None and v.dim() == 2 else v for k, v in p.items()}
        want = ops.block_norm_bwd(dr[:n], dh[:n], h[:n], cut["y"], **kw) if n else None
        held = {k: rnd(20 + i, d) for i, k in enumerate(("dafter", "dgate", "dbefore"))}
        before = {k: v.clone() for k, v in held.items()}
        dx, dy = torch.full((t, d), 7.0, device="cuda"), torch.full((t, d), 7.0, dtype=torch.bfloat16, device="cuda")
        got = ops.block_norm_bwd(dr, dh, h, p["y"], **kw, **held, dx=dx, dy=dy, accumulate=True, n_rows=lim)
        assert (dx[n:] == 7).all() and (dy[n:] == 7).all() and torch.equal(dx[:n], once.dx[:n]) and torch.equal(dy[:n], once.dy[:n])
        for k in held:
            assert torch.equal(getattr(got, k), before[k] + (getattr(want, k) if n else 0.0))


def test_joint_of_very_many_narrow_rows(ops):
    t, d = 300001, 40
    x, y, w = rnd(1, t, d), rnd(2, t, d, dtype=torch.bfloat16), rnd(3, d, std=0.1, mean=1.0)
    h, r = ops.block_norm(x, y, after=w, before=w)
    rms = lambda v: v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)        # noqa: E731
    want = x.double() + rms(y.double()) * w.double()
    assert float((h.double() - want).abs().max()) < 100 * U * float(want.abs().max())
    assert float((r.double() - rms(want) * w.double()).abs().max()) < 2.0 ** -8 * 1.1 * float(r.abs().max())
    g = ops.block_norm_bwd(r, x, h, y, after=w, before=w)
    hn = rms(h.double())
    ref = (r.double() * hn).sum(0)
    assert float((g.dbefore.double() - ref).abs().max()) <= (t / 100 + 200) * U * float((r.double() * hn).abs().sum(0).max())


def test_joint_in_place(ops):
    for d in (768, 101, 4104):
        t = 300
        p = joint_inputs(t, d, "fp32", "bf16", "channel")
        kw = dict(after=p["after"], gate=p["gate"], before=p["before"])
        h, r = ops.block_norm(p["x"], p["y"], **kw)
        dr, dh = rnd(5, t, d, dtype=torch.bfloat16), rnd(6, t, d)
        want = ops.block_norm_bwd(dr, dh, h, p["y"], **kw)
        x = p["x"].clone()
        h2, r2 = ops.block_norm(x, p["y"], **kw, h=x)
        assert h2 is x and torch.equal(h, x) and torch.equal(r, r2)
        got = ops.block_norm_bwd(dr, dh, h, p["y"], **kw, dx=dh)
        assert got.dx is dh and all(torch.equal(a, b) for a, b in zip(got, want))


def test_joint_rows_that_are_zero_or_not_finite(ops):
    """Rows of zeros have finite gradients; infinities and NaN spoil their own row, and the sums over rows."""
    t, d = 40, 768
    p = joint_inputs(t, d, "fp32", "bf16", "channel")
    p["x"][3], p["y"][3], p["y"][5] = 0.0, 0.0, 0.0
    h, _ = check_joint(ops, p, 1.0, 1.0)
    dr, dh = rnd(5, t, d, dtype=torch.bfloat16), rnd(6, t, d)
    check_joint_grad(ops, p, dr, dh, h, 1.0, 1.0)
    q = {k: None if v is None else v.clone() for k, v in p.items()}
    q["x"][7, 5], q["y"][9, 700], q["x"][11, 0] = float("nan"), float("inf"), float("-inf")
    h2, r2 = ops.block_norm(q["x"], q["y"], after=q["after"], gate=q["gate"], before=q["before"])
    ok = torch.ones(t, dtype=torch.bool, device="cuda")
    ok[[7, 9, 11]] = False
    assert torch.equal(h2[ok], h[ok]) and r2[~ok].isnan().any(1).all() and h2[ok].isfinite().all() and r2[ok].isfinite().all()
    g = ops.block_norm_bwd(dr, dh, h2, q["y"], after=q["after"], gate=q["gate"], before=q["before"])
    assert g.dx[ok].isfinite().all() and g.dy[ok].isfinite().all() and g.dbefore.isnan().any()


def test_joint_of_tiny_rows_and_eps(ops):
    """Rows of zeros and of 1e-12 under an eps of 1e-26: the cube of 1 / rms is beyond
    fp32, the gradients are not."""
    t, d = 12, 768
    x = rnd(1, t, d) * 1e-12
    x[3] = 0.0
    w = rnd(4, d, std=0.1, mean=1.0)
    _, r = ops.block_norm(x, before=w, eps=1e-26)
    _, want, _, bound = R.joint(as64(x), None, None, None, as_row(w), 1.0, 1.0, 1e-26)
    close(r, want, bound)
    dr = rnd(5, t, d)
    got = ops.block_norm_bwd(dr, None, x, before=w, eps=1e-26)
    ref = R.joint_grad(as64(dr), None, as64(x), None, None, None, as_row(w), 1.0, 1.0, 1e-26)
    close(got.dx, *ref["dx"])
    close(got.dbefore, *R.row_sum(*ref["dbefore"]))
    y = x.clone()
    got = ops.block_norm_bwd(None, dr, x, y, after=w, eps=1e-26)
    ref = R.joint_grad(None, as64(dr), as64(x), as64(y), as_row(w), None, None, 1.0, 1.0, 1e-26)
    close(got.dy, *ref["dy"])


def test_rows_far_apart(ops):
    """Row strides of 2^26 elements: offsets beyond 32 bits."""
    t, d = 40, 264
    far = lambda dt: torch.empty(t << 26, dtype=dt, device="cuda").view(t, 1 << 26)[:, :d]      # noqa: E731
    p = joint_inputs(t, d, "fp32", "bf16", "full")
    x, h = far(torch.float32), far(torch.float32)
    y = far(torch.bfloat16)
    x.copy_(p["x"])
    y.copy_(p["y"])
    q = dict(p, x=x, y=y)
    check_joint(ops, q, 1.0, 0.5, h=h)
    want = ops.block_norm(p["x"], p["y"], after=p["after"], gate=p["gate"], before=p["before"], out_scale=0.5)
    assert torch.equal(h, want[0])
    dr, dh = rnd(5, t, d, dtype=torch.bfloat16), rnd(6, t, d)
    a = ops.block_norm_bwd(dr, dh, want[0], p["y"], after=p["after"], gate=p["gate"], before=p["before"])
    x.copy_(dh)
    b = ops.block_norm_bwd(dr, x, h, y, after=p["after"], gate=p["gate"], before=p["before"], dx=x)
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    z = rnd(7, t, 16)
    h[:, :16] = z
    c, c2 = ops.choose(z, 2), ops.choose(h[:, :16], 2)
    assert all(torch.equal(u, v) for u, v in zip(c[:4], c2[:4]))
    want = ops.choose_bwd(z, c.idx, c.counts, c.w, c.losses)
    assert torch.equal(ops.choose_bwd(h[:, :16], c.idx, c.counts, c.w, c.losses, out=x[:, :16]), want)


def test_joint_refusals(ops):
    p = joint_inputs(6, 64, "fp32", "bf16", "channel")
    x, y, w = p["x"], p["y"], p["after"]
    bad = [lambda: ops.block_norm(x, y.float().double(), before=w), lambda: ops.block_norm(x, y[:5], before=w),
           lambda: ops.block_norm(x, y, after=w[:-1]), lambda: ops.block_norm(x, y, after=w.bfloat16()),
           lambda: ops.block_norm(x, y, gate=w.bfloat16()), lambda: ops.block_norm(x, y, gate=torch.ones(6, 1, device="cuda", dtype=torch.bfloat16)),
           lambda: ops.block_norm(x, y, gate=torch.ones(6, 64, device="cuda")), lambda: ops.block_norm(x), lambda: ops.block_norm(x, before=w, after=w),
           lambda: ops.block_norm(x, before=w, res_scale=2.0), lambda: ops.block_norm(x, y, r=y), lambda: ops.block_norm(x, y, before=w, dtype=torch.float32),
           lambda: ops.block_norm(x, y, before=w, h=torch.empty(6, 64, device="cuda", dtype=torch.bfloat16)),
           lambda: ops.block_norm(x, y, before=w, n_rows=torch.ones(1, device="cuda")), lambda: ops.block_norm(x.t(), y, before=w),
           lambda: ops.block_norm(x[0], y, before=w), lambda: ops.block_norm(x, before=w, dtype=torch.float16),
           lambda: ops.block_norm_bwd(None, None, x, y, after=w), lambda: ops.block_norm_bwd(y, x, x, y, after=w),
           lambda: ops.block_norm_bwd(None, x, x, y, before=w), lambda: ops.block_norm_bwd(y, x.bfloat16(), x, y, before=w),
           lambda: ops.block_norm_bwd(x, x, x, y, before=w), lambda: ops.block_norm_bwd(y, x, x, y, before=w, dafter=w),
           lambda: ops.block_norm_bwd(y, x, x, None, before=w, dy=y), lambda: ops.block_norm_bwd(y, x, x, y, before=w, dgate=w),
           lambda: ops.block_norm_bwd(y, x, x, y, before=w, accumulate=True)]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            f()
            pytest.fail(f"call {i} was not refused")
    with pytest.raises(RuntimeError):
        ops.block_norm(x, y, before=w, eps=0.0)
    with pytest.raises(RuntimeError):
        ops.block_norm(x.bfloat16(), y.float(), before=w)
    with pytest.raises(RuntimeError):
        ops.block_norm(torch.zeros(1, 8200, device="cuda"), before=torch.ones(8200, device="cuda"))


def test_joint_of_many_rows(ops):
    """A microbatch of 32 x 1024 tokens: rows against float64 on the device, the
    sums over rows within a rounding for each of their additions."""
    t, d = 32768, 768
    p = joint_inputs(t, d, "fp32", "bf16", "channel")
    dr, dh = rnd(5, t, d, std=1e-3, dtype=torch.bfloat16), rnd(6, t, d, std=1e-3)
    kw = dict(after=p["after"], gate=p["gate"], before=p["before"])
    h, r = ops.block_norm(p["x"], p["y"], **kw)
    g = ops.block_norm_bwd(dr, dh, h, p["y"], **kw)
    some = torch.randint(0, t, (200,), generator=torch.Generator().manual_seed(0)).cuda()
    sub = {k: v[some] if v is not None and v.dim() == 2 else v for k, v in p.items()}
    want = R.joint(as64(sub["x"]), as64(sub["y"]), as_row(p["after"]), as_row(p["gate"]), as_row(p["before"]), 1.0, 1.0, EPS)
    close(h[some], want[0], want[2])
    close(r[some], want[1], want[3])
    wg = R.joint_grad(as64(dr), as64(dh), as64(h), as64(p["y"]), as_row(p["after"]), as_row(p["gate"]), as_row(p["before"]), 1.0, 1.0, EPS)
    close(g.dx, *wg["dx"])
    close(g.dy, *wg["dy"])
    for name in ("dgate", "dafter", "dbefore"):
        close(getattr(g, name), *R.row_sum(*wg[name]))
    again = ops.block_norm_bwd(dr, dh, h, p["y"], **kw)
    assert all(torch.equal(a, b) for a, b in zip(g, again))


# ---------------------------------------------------------------------------
# the router's choice
# ---------------------------------------------------------------------------
def logits(seed, t, e, how, dtype=torch.float32):
    z = rnd(seed, t, e) + rnd(seed + 1, e)
    if how == "ties":
        z = (z * 2).round() / 2
    elif how == "equal":
        z = torch.zeros_like(z)
    elif how == "closed":                        # some experts for all tokens, all experts for some
        z[:, ::3] = float("-inf")
        z[::5] = float("-inf")
        z[torch.rand(t, e, generator=torch.Generator().manual_seed(3)).cuda() < 0.3] = float("-inf")
    elif how == "lowest":
        z[torch.rand(t, e, generator=torch.Generator().manual_seed(3)).cuda() < 0.7] = torch.finfo(dtype).min
        z[::7] = torch.finfo(dtype).min
    elif how == "wide":
        z = z * 40
    elif how == "zeros":
        z = torch.where(z > 0, 0.0, -0.0)
    elif how == "bad":
        z[3 % t, e // 2], z[(t - 1), 0], z[t // 2] = float("nan"), float("inf"), float("-inf")
    return z.to(dtype)


def check_choice(ops, z, k, mask, renormalize):
    c = ops.choose(z, k, mask, renormalize)
    m = None if mask is None else mask.cpu().numpy().astype(bool)
    z64 = as64(z)
    idx, w, counts, losses, p, lse, live = R.choose(z64, k, m, renormalize)
    assert np.array_equal(c.idx.cpu().numpy(), idx)
    assert np.array_equal(c.counts.cpu().numpy(), counts)
    # exponentials: U |z - max| of the argument, 2 ulp of expf; 64 additions; the division
    # (of those within 110 of the largest: others vanish)
    top = np.where(np.isfinite(z64), z64, -np.inf).max(1, keepdims=True)
    near = np.isfinite(z64) & (z64 > top - 110)
    span = np.where(near, np.where(near, top, 0.0) - np.where(near, z64, 0.0), 0.0).max(1)
    rel = (span[:, None] + 80) * U
    close(c.w, w, rel * np.nan_to_num(w) + 1e-37, "w")
    worst = float(rel.max()) if rel.size else 0.0
    total = (worst + (z.shape[0] / 100 + 80) * U) * 2
    bound = np.array([total * np.nan_to_num(losses[0]), 0.0])
    if live.any():
        el = np.nan_to_num(np.abs(lse[live]) * 3 * U + 80 * U)
        bound[1] = (2 * np.nan_to_num(np.abs(lse[live])) * el + el * el).sum() / live.sum() + total * np.nan_to_num(losses[1])
    close(c.losses, losses, bound, "losses")
    return c, worst


SHAPES = [(1, 1, 1), (1, 16, 2), (3, 2, 2), (33, 7, 3), (64, 8, 8), (200, 16, 2), (130, 17, 8), (77, 32, 8), (100, 33, 4), (129, 64, 8)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("how", ["plain", "ties", "equal", "closed", "lowest", "wide", "zeros", "bad"])
@pytest.mark.parametrize("t,e,k", SHAPES)
def test_choice_and_its_gradient(ops, t, e, k, how, dtype):
    z = logits(t + e, t, e, how, DT[dtype])
    for renormalize in (True, False):
        for mask in (None, torch.rand(t, generator=torch.Generator().manual_seed(5)).cuda() < 0.6):
            c, rel = check_choice(ops, z, k, mask, renormalize)
            dw, dl = rnd(8, t, k), torch.tensor([0.7, 0.03], device="cuda")
            m = None if mask is None else mask.cpu().numpy()
            for a, b in ((dw, dl), (dw, None), (None, dl)):
                got = ops.choose_bwd(z, c.idx, c.counts, a, b, mask, renormalize)
                want, mag = R.choose_grad(as64(z), c.idx.cpu().numpy(), c.counts.cpu().numpy().astype(np.int64),
                                          None if a is None else as64(a), None if b is None else as64(b), m, renormalize)
                close(got, want, (3 * rel + 30 * U) * mag + 1e-36, (renormalize, mask is not None))


def test_choice_of_all_masked_and_of_no_tokens(ops):
    z = rnd(1, 50, 16)
    c = ops.choose(z, 2, torch.zeros(50, dtype=torch.bool, device="cuda"))
    assert (c.idx == -1).all() and (c.w == 0).all() and (c.counts == 0).all() and (c.losses == 0).all()
    assert (ops.choose_bwd(z, c.idx, c.counts, rnd(2, 50, 2), torch.ones(2, device="cuda"), torch.zeros(50, dtype=torch.bool, device="cuda")) == 0).all()
    c = ops.choose(z[:0], 2)
    assert c.idx.shape == (0, 2) and (c.counts == 0).all() and (c.losses == 0).all()
    assert ops.choose_bwd(z[:0], c.idx, c.counts, c.w).shape == (0, 16)


@pytest.mark.parametrize("t,e,k", [(1023, 16, 2), (1024, 16, 2), (1025, 64, 8), (5000, 8, 2), (9000, 30, 5), (32768, 16, 2)])
def test_choice_over_many_tokens(ops, t, e, k):
    """Sizes around and above those that one CTA takes; the same results again bit for bit."""
    z = logits(4, t, e, "plain")
    mask = torch.rand(t, generator=torch.Generator().manual_seed(5)).cuda() < 0.8
    c, rel = check_choice(ops, z, k, mask, True)
    again = ops.choose(z, k, mask, True)
    assert all(torch.equal(a, b) for a, b in zip(c[:4], again[:4]))
    dw, dl = rnd(8, t, k), torch.tensor([0.7, 0.03], device="cuda")
    want, mag = R.choose_grad(as64(z), c.idx.cpu().numpy(), c.counts.cpu().numpy().astype(np.int64), as64(dw), as64(dl), mask.cpu().numpy(), True)
    close(ops.choose_bwd(z, c.idx, c.counts, dw, dl, mask), want, (3 * rel + 30 * U) * mag + 1e-36)


TILED = [(50000, 17, 8), (60000, 24, 6), (45000, 32, 8), (101000, 33, 3), (38000, 63, 8), (40000, 64, 8)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("how", ["plain", "ties", "equal", "closed", "lowest", "wide", "zeros", "bad"])
@pytest.mark.parametrize("t,e,k", TILED)
def test_choice_by_tiles(ops, t, e, k, how, dtype):
    """More choices than the lanes' kernel takes: the same as its own, which the
    other tests hold to the definition, over slices that it takes."""
    z = logits(t, t, e, how, DT[dtype])
    mask = torch.rand(t, generator=torch.Generator().manual_seed(5)).cuda() < 0.8
    for renormalize, m in ((True, mask), (False, None)):
        assert t * k > 300000
        c = ops.choose(z, k, m, renormalize)
        n = 300000 // k
        parts = [ops.choose(z[i:i + n], k, None if m is None else m[i:i + n], renormalize) for i in range(0, t, n)]
        assert torch.equal(c.idx, torch.cat([p.idx for p in parts]))
        assert torch.equal(c.counts, sum(p.counts for p in parts))
        w = torch.cat([p.w for p in parts])
        # sums of up to 64 exponentials in another order
        assert torch.equal(c.w.isnan(), w.isnan())       # NaN meets no bound: compared apart
        w = w.nan_to_num(0.0)
        assert ((c.w.nan_to_num(0.0) - w).abs() <= 130 * U * w).all()
        spoiled = ~(z < float("inf")).all(1)
        if m is not None:
            spoiled &= m                         # a masked row spoils nothing
        assert bool(c.losses.isnan().all()) == bool(spoiled.any()) == bool(c.losses.isnan().any())
        if spoiled.any():
            continue
        if how == "lowest":                      # squares of the lowest logit: beyond fp32
            assert c.losses[1] == float("inf")
        many = torch.stack([p.counts[-1] for p in parts]).double()
        size = float((torch.stack([p.losses[1] for p in parts]).double() * many).sum() / many.sum())
        assert how == "lowest" or abs(float(c.losses[1]) - size) <= 1000 * U * size
        live = torch.ones(t, dtype=torch.bool, device="cuda") if m is None else m
        live = live & (z.float().amax(1) > -float("inf"))
        p = torch.softmax(z[live].double(), 1).mean(0)
        balance = float(e * (c.counts[:-1].double() / (k * int(c.counts[-1])) * p).sum())
        assert abs(float(c.losses[0]) - balance) <= 1000 * U * balance
        again = ops.choose(z, k, m, renormalize)
        assert all(torch.equal(a, b) for a, b in zip(c[:3], again[:3])) and torch.equal(c.losses, again.losses)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_choice_by_tiles_against_the_definition(ops, dtype):
    z = logits(3, 40000, 64, "closed", DT[dtype])
    check_choice(ops, z, 8, torch.rand(40000, generator=torch.Generator().manual_seed(5)).cuda() < 0.8, True)
    check_choice(ops, strided(z[:, :61].contiguous(), 3, 1), 8, None, False)


def test_choice_of_views_and_given_outputs(ops):
    z = strided(rnd(1, 300, 16), 3, 1)
    a, _ = check_choice(ops, z, 2, None, True)
    c = ops.choose(z, 2)
    for v in c:
        v.fill_(77)
    c2 = ops.choose(z, 2, out=c)
    assert all(x is y for x, y in zip(c, c2)) and all(torch.equal(x, y) for x, y in zip(a[:4], c[:4]))
    out = strided(torch.zeros(300, 16, device="cuda"), 5, 2)
    want = ops.choose_bwd(z.contiguous(), c.idx, c.counts, rnd(8, 300, 2))
    got = ops.choose_bwd(z, c.idx, c.counts, rnd(8, 300, 2), out=out)
    assert got is out and (got - want).abs().max() <= 1e-6 and out._base[:, :2].isnan().all() and out._base[:, 18:].isnan().all()


def test_choice_gradient_of_strange_indices(ops):
    """Indices outside the experts add nothing; an expert named twice gets both gradients."""
    z, dw = rnd(1, 4, 8), rnd(2, 4, 3)
    idx = torch.tensor([[0, 0, 3], [-1, 9, 2], [5, -7, 5], [-1, -1, -1]], dtype=torch.int32, device="cuda")
    for renormalize in (True, False):
        want, mag = R.choose_grad(as64(z), idx.cpu().numpy(), np.zeros(9, np.int64), as64(dw), None, None, renormalize)
        close(ops.choose_bwd(z, idx, dw=dw, renormalize=renormalize), want, 400 * U * mag + 1e-36)


@pytest.mark.parametrize("t,e,k", [(1000003, 16, 2), (300001, 40, 8)])
def test_choice_over_very_many_tokens(ops, t, e, k):
    z = rnd(1, t, e)
    c = ops.choose(z, k)
    want = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(c.idx.long(), want)
    load = torch.bincount(want.reshape(-1), minlength=e)
    assert torch.equal(c.counts[:-1].long(), load) and int(c.counts[-1]) == t
    p = torch.softmax(z.double(), 1)
    balance = float(e * (load.double() / (k * t) * p.mean(0)).sum())
    size = float((torch.logsumexp(z.double(), 1) ** 2).mean())
    assert abs(float(c.losses[0]) - balance) < 1e-5 and abs(float(c.losses[1]) - size) < 1e-5 * size
    w = p.gather(1, want)
    assert float((c.w.double() - w / w.sum(1, keepdim=True)).abs().max()) < 1e-6


def test_masks_of_bytes(ops):
    """Any byte but 0 lets a token take part."""
    z = rnd(1, 300, 16)
    m = torch.tensor([0, 1, 2, 255] * 75, dtype=torch.uint8, device="cuda")
    a, b = ops.choose(z, 2, m), ops.choose(z, 2, m != 0)
    assert all(torch.equal(u, v) for u, v in zip(a[:4], b[:4]))
    dw = rnd(2, 300, 2)
    assert torch.equal(ops.choose_bwd(z, a.idx, a.counts, dw, a.losses, m), ops.choose_bwd(z, a.idx, a.counts, dw, a.losses, m != 0))


def test_choice_refusals(ops):
    z, i = rnd(1, 6, 8), torch.zeros(6, 2, dtype=torch.int32, device="cuda")
    dw, dl = rnd(2, 6, 2), torch.ones(2, device="cuda")
    c = ops.choose(z, 2)
    bad = [lambda: ops.choose(z.double(), 2), lambda: ops.choose(z[0], 2), lambda: ops.choose(z, 2, mask=torch.ones(6, device="cuda")),
           lambda: ops.choose(z, 2, mask=torch.ones(5, dtype=torch.bool, device="cuda")), lambda: ops.choose(z, 3, out=c), lambda: ops.choose(z[:5], 2, out=c),
           lambda: ops.choose_bwd(z, i), lambda: ops.choose_bwd(z, i, dlosses=dl), lambda: ops.choose_bwd(z, i.long(), dw=dw),
           lambda: ops.choose_bwd(z, i, dw=dw[:, :1]), lambda: ops.choose_bwd(z, i, c.counts, dlosses=dl.double()),
           lambda: ops.choose_bwd(z, i, c.counts[:-1], dlosses=dl), lambda: ops.choose_bwd(z, i, dw=dw, out=z.bfloat16()), lambda: ops.choose_bwd(z, i[0], dw=dw)]
    for f in bad:
        with pytest.raises((ValueError, TypeError)):
            f()
    for f in (lambda: ops.choose(z, 9), lambda: ops.choose(z, 0), lambda: ops.choose(rnd(1, 4, 65), 2)):
        with pytest.raises(RuntimeError):
            f()


# ---------------------------------------------------------------------------
# the gradient norm
# ---------------------------------------------------------------------------
# sums of at most 64 squares and eight places in 32 bits; the norm is their root, rounded
NORM = 40 * U


def check_clip(ops, ts, max_norm, scale=1.0, eps=1e-6, out=None):
    vals = [as64(t) for t in ts]
    with np.errstate(over="ignore"):
        norm = abs(scale) * math.sqrt(math.fsum(float((v * v).sum()) for v in vals)) if all(np.isfinite(v).all() for v in vals) else math.inf
    s = ops.GradSet(ts, out)
    got = s.norm(scale)
    stats = s.clip(max_norm, eps, scale)
    coef = min(1.0, max_norm / (norm + eps)) if norm < math.inf else 0.0
    for n in (float(got), float(stats[0])):
        assert n == norm or abs(n - norm) <= NORM * norm + 1e-45, (n, norm)
    assert abs(float(stats[1]) - coef) <= (NORM + U) * coef
    for v, o in zip(vals, ts if out is None else out):
        f = scale * coef
        want = v * f
        assert o.shape == v.shape
        close(o, want, (NORM + 3 * U) * np.abs(want) + 1e-44 if coef < 1 else 2 * U * np.abs(want) + 1e-44)
    return stats


SETS = [[1], [8], [7, 9], [1000, 3, 0, 8192], [8193, 8191, 16384], [100000, 1, 250000], [5] * 40, [33, 4097] * 150, [3] * 1500 + [70000]]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "mixed"])
@pytest.mark.parametrize("sizes", SETS, ids=lambda s: f"{len(s)}x{sum(s)}")
def test_clip_of_sets(ops, sizes, dtype):
    for max_norm, scale in ((0.5, 1.0), (1e9, 1.0), (0.5, -0.25)):
        ts = [rnd(i, n, dtype=DT[dtype] if dtype != "mixed" else list(DT.values())[i % 2]) for i, n in enumerate(sizes)]
        before = [t.clone() for t in ts]
        out = [torch.full_like(t, 5.0) for t in ts]
        check_clip(ops, ts, max_norm, scale, out=out)
        assert all(torch.equal(a, b) for a, b in zip(ts, before))
        check = [t.clone() for t in ts]
        stats = ops.clip_grads(check, max_norm, scale=scale)
        assert all(torch.equal(a, b) for a, b in zip(check, out))
        assert torch.equal(stats, ops.clip_grads(ts, max_norm, scale=scale, out=out))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_clip_of_packed_views(ops, dtype):
    """Tensors one behind the other in a buffer, off every boundary; outputs on other boundaries than the inputs."""
    sizes = [1, 2, 3, 5, 17, 1001, 9999, 40001]
    flat = rnd(1, sum(sizes), dtype=DT[dtype])
    for shift in (0, 1, 4, 8):
        buf = torch.full((shift + flat.numel() + 9,), 7.0, dtype=flat.dtype, device="cuda")
        out = list(buf[shift:shift + flat.numel()].split(sizes))
        check_clip(ops, list(flat.split(sizes)), 1.0, out=out)
        assert (buf[:shift] == 7).all() and (buf[shift + flat.numel():] == 7).all()
    g = flat.clone()
    ops.clip_grads(list(g.split(sizes)), 1.0)
    assert torch.equal(g, buf[8:8 + flat.numel()])


def test_clip_of_any_dense_shape(ops):
    ts = [rnd(1, 3, 4).t(), rnd(2, 2, 3, 5).permute(2, 0, 1), rnd(3, 1)[0], rnd(4, 0, 3), rnd(5, 4, 4)[:, :, None]]
    check_clip(ops, ts, 1.0, out=[torch.empty_like(t) for t in ts])
    ops.clip_grads(ts, 1.0)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("size", [1e38, 1e30, 1e17, 1e-12, 1e-17, 1e-25, 1e-38, 3e-41])
def test_norms_at_the_ends_of_the_range(ops, size, dtype):
    """Squares that 32 bits do not hold, alone and among others."""
    for n in (8, 33, 5000):
        ts = [rnd(1, n, std=1.0).mul(size / 4).to(DT[dtype])]
        vals = as64(ts[0])
        norm = math.sqrt(float((vals * vals).sum()))
        got = float(ops.grad_norm(ts))
        want = np.float32(norm) if norm < 3.4e38 else np.inf
        assert got == want or abs(got - norm) <= NORM * norm + 1e-45, (got, norm)
        mixed = ts + [rnd(2, 1000)]
        total = math.sqrt(norm ** 2 + float((as64(mixed[1]) ** 2).sum()))
        got = float(ops.grad_norm(mixed))
        assert got == np.inf and total > 3.4e38 or abs(got - total) <= NORM * total
    sc = 1.0 / size if size < 1e38 else 1e-30
    assert abs(float(ops.grad_norm(ts, sc)) - sc * norm) <= NORM * sc * norm


def test_norms_that_are_not_finite(ops):
    for where in (0, 4, 4095, 9000):
        t = rnd(1, 9001)
        t[where] = float("inf")
        u = t.clone()
        stats = ops.clip_grads([u], 1.0)
        assert float(stats[0]) == math.inf and float(stats[1]) == 0.0
        assert u[where].isnan() and (u.nan_to_num(0.0) == 0).all()
        t[where] = float("nan")
        stats = ops.clip_grads([t], 1.0)
        assert stats.isnan().all() and t.isnan().all()


def test_clip_leaves_small_sets_alone(ops):
    """In place and under the limit nothing is written (scale 1); no tensors at all have a norm of zero."""
    t = [rnd(1, 5000, std=1e-3), torch.zeros(9, device="cuda")]
    want = [v.clone() for v in t]
    stats = ops.clip_grads(t, 10.0)
    assert float(stats[1]) == 1.0 and all(torch.equal(a, b) for a, b in zip(t, want))
    z = ops.GradSet([], device="cuda")
    assert float(z.norm()) == 0.0 and z.clip(1.0).tolist() == [0.0, 1.0]
    z = ops.GradSet([torch.zeros(100, device="cuda"), torch.zeros(0, device="cuda")])
    assert float(z.norm()) == 0.0 and z.clip(1.0, eps=0.0).tolist() == [0.0, 1.0]


def test_sets_keep_their_memory(ops):
    """A set is of the memory its tensors had, whatever they are given later; the values are those of the call."""
    a, b = rnd(1, 1000), rnd(2, 500)
    was = a.detach()
    s = ops.GradSet([a, b])
    want = float(torch.cat([a, b]).double().norm())
    a.data = rnd(3, 1000) * 10
    torch.cuda.synchronize()
    assert abs(float(s.norm()) - want) < 1e-4
    was.mul_(3.0)
    assert abs(float(s.norm()) - float(torch.cat([was, b]).double().norm())) < 1e-3
    del was, a, b
    filler = [torch.full((1000,), 1e9, device="cuda") for _ in range(50)]
    assert float(s.norm()) < 1e4 and filler


def test_clip_refusals(ops):
    a, b = rnd(1, 100), rnd(2, 100)
    bad = [lambda: ops.GradSet([a, a]), lambda: ops.GradSet([a, a[50:]]), lambda: ops.GradSet([a.double()]), lambda: ops.GradSet([a.half()]),
           lambda: ops.GradSet([a[::2]]), lambda: ops.GradSet([a.expand(3, 100)]), lambda: ops.GradSet([a, b], [a]),
           lambda: ops.GradSet([a, b], [b, a]), lambda: ops.GradSet([a, b], [a, b[:50]]), lambda: ops.GradSet([a[:50], b[:50]], [a[25:75], b[50:]]),
           lambda: ops.GradSet([a], [b.bfloat16()]), lambda: ops.GradSet([a.view(10, 10)], [b.view(10, 10).t()]), lambda: ops.GradSet([a], [b.cpu()])]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    for kw in (dict(max_norm=0.0), dict(max_norm=float("nan")), dict(max_norm=1.0, eps=-1.0), dict(max_norm=1.0, scale=float("inf"))):
        before = a.clone()
        with pytest.raises(RuntimeError):
            ops.clip_grads([a], **kw)
        assert torch.equal(a, before)


def test_clip_of_a_tensor_beyond_32_bits(ops):
    """2^31 and some elements in one tensor, and a few behind it."""
    n = (1 << 31) + 4099
    big, small = torch.zeros(n, dtype=torch.bfloat16, device="cuda"), torch.ones(1001, device="cuda")
    for i in (0, 12345, (1 << 31) - 1, 1 << 31, n - 1):
        big[i] = 3.0
    s = ops.clip_grads([big, small], 1.0)
    norm = math.sqrt(5 * 9 + 1001)
    assert abs(float(s[0]) - norm) <= NORM * norm
    want = torch.tensor(3.0 * (1.0 / (norm + 1e-6))).bfloat16()
    for i in (0, 12345, (1 << 31) - 1, 1 << 31, n - 1):
        assert float((big[i].float() - want.float()).abs()) <= 2.0 ** -8 * float(want)
    assert int(torch.count_nonzero(big)) == 5


def test_norm_of_a_large_set(ops):
    """200 million elements over a few tensors: several rounds of every thread."""
    ts = [torch.randn(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(n)) for n in (120_000_003, 5, 80_000_001)]
    want = math.sqrt(sum(float((t.double() ** 2).sum()) for t in ts))
    outs = [torch.empty_like(t) for t in ts]
    s = ops.GradSet(ts, outs).clip(1.0)
    assert abs(float(s[0]) - want) <= NORM * want
    f = 1.0 / (want + 1e-6)
    for t, o in zip(ts, outs):
        assert float(((o.double() - t.double() * f).abs() - (NORM + 3 * U) * f * t.double().abs()).max()) <= 0
