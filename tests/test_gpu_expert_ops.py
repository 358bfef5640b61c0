"""The stand-alone expert operators on the GPU against their definitions in
float64 on the host (tests/expert_ref.py), with bounds derived from the
roundings each operator makes: U32 = 2^-24 per fp32 operation, half a step for
the rounding to the output type."""
import numpy as np
import pytest
import torch

import expert_ref as R

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
HALF_STEP = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}     # of the output's rounding (fp32: counted in U32)


@pytest.fixture(scope="module")
def ops():
    from adamw_persistent_sm_gb300 import expert_ops
    yield expert_ops
    expert_ops.check()


def rnd(seed, *shape, std=1.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def strided(t, pad, shift=0):
    """t as a view of a wider buffer: rows `pad` elements further apart, starting `shift` in."""
    buf = torch.full((t.shape[0], t.shape[1] + pad + shift), float("nan"), dtype=t.dtype, device=t.device)
    v = buf[:, shift:shift + t.shape[1]]
    v.copy_(t)
    return v


def close(got, want, bound, what=""):
    got = R.as64(got) if isinstance(got, torch.Tensor) else got
    assert np.array_equal(np.isfinite(want), np.isfinite(got)), what
    f = np.isfinite(want)
    bad = np.abs(got - want)[f] > np.broadcast_to(bound, want.shape)[f]
    assert not bad.any(), (what, int(bad.sum()), float(np.abs(got - want)[f][bad].max()))


# ---------------------------------------------------------------------------
# route
# ---------------------------------------------------------------------------
def choices(seed, t, k, e, how):
    g = np.random.default_rng(seed)
    idx = np.stack([g.permutation(e)[:k] for _ in range(t)]).astype(np.int32) if t else np.zeros((0, k), np.int32)
    if how == "dropped":
        idx[g.random(t) < 0.4] = -1
        idx[g.random((t, k)) < 0.1] = -1
    elif how == "none":
        idx[:] = -1
    elif how == "one":
        idx[:] = e - 1                   # every slot of every token names the same expert
    elif how == "skewed":
        idx = (g.random((t, k)) ** 4 * e).astype(np.int32)
    return idx


ROUTES = [(0, 2, 4, "even"), (1, 1, 1, "even"), (1, 2, 16, "even"), (1, 2, 16, "none"), (5, 8, 8, "even"),
          (127, 1, 3, "one"), (128, 2, 2, "even"), (129, 4, 5, "dropped"), (1000, 3, 7, "skewed"),
          (1024, 8, 64, "even"), (1025, 8, 64, "dropped"), (8193, 1, 33, "one"), (4097, 2, 16, "dropped"),
          (5000, 2, 16, "none"), (20000, 8, 64, "skewed"), (32768, 2, 16, "even"), (40001, 8, 64, "dropped")]


@pytest.mark.parametrize("t,k,e,how", ROUTES)
def test_route_order(ops, t, k, e, how):
    idx = choices(t + k, t, k, e, how)
    r = ops.Route(t, k, e)
    for b in (r.offs, r.perm, r.row):
        b.fill_(12345)
    r.order(torch.from_numpy(idx).cuda())
    offs, perm, row = R.order(idx, e)
    assert np.array_equal(r.offs.cpu().numpy(), offs)
    assert np.array_equal(r.perm.cpu().numpy(), perm)
    assert np.array_equal(r.row.cpu().numpy(), row)
    ops.check()


@pytest.mark.parametrize("n", [31, 33, 1023, 4095, 4096, 4097, 16385, 65535, 65536, 65537, 98305, 262145])
@pytest.mark.parametrize("how", ["dropped", "one"])
def test_route_order_at_the_kernels_limits(ops, n, how):
    """Sizes around those where one CTA, a cluster and a grid take over."""
    test_route_order(ops, n, 1, 5, how)


def test_route_order_of_many_tokens(ops):
    """Three million assignments (a grid of CTAs with long chunks), against a
    stable sort on the device."""
    t, k, e = 400001, 8, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    idx = (torch.rand(t, k, generator=g, device="cuda") ** 2 * e).to(torch.int32)
    idx[torch.rand(t, generator=g, device="cuda") < 0.1] = -1
    r = ops.Route(t, k, e).order(idx)
    a = idx.reshape(-1).long()
    counts = torch.stack([(a == i).sum() for i in range(e)])
    offs = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), ((counts + 127) // 128 * 128).cumsum(0)])
    assert torch.equal(r.offs.long(), offs)
    kept = torch.nonzero(a >= 0)[:, 0]
    by = kept[torch.sort(a[kept], stable=True).indices]
    first = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), counts.cumsum(0)])[:-1]
    at = offs[a[by]] + torch.arange(by.numel(), device="cuda") - first[a[by]]
    perm = torch.full((r.rows,), -1, dtype=torch.long, device="cuda")
    perm[at] = by
    row = torch.full_like(a, -1)
    row[by] = at
    assert torch.equal(r.perm.long(), perm) and torch.equal(r.row.reshape(-1).long(), row)
    ops.check()


@pytest.mark.parametrize("t", [10, 9000, 140000])
def test_route_order_reports_bad_indices(ops, t):
    idx = choices(1, t, 2, 8, "even")
    bad = idx.copy()
    bad[3, 0], bad[t - 1, 1], bad[5, 0] = 8, -2, 2 ** 31 - 1
    r = ops.Route(t, 2, 8).order(torch.from_numpy(bad).cuda())
    from adamw_persistent_sm_gb300.trainer import StatusError
    with pytest.raises(StatusError, match="out of range"):
        ops.check()
    ops.check()                                        # reported once
    bad[3, 0] = bad[t - 1, 1] = bad[5, 0] = -1
    for got, want in zip((r.offs, r.perm, r.row), R.order(bad, 8)):
        assert np.array_equal(got.cpu().numpy(), want)


MOVES = [(1, 2, 16, "even", 768), (7, 3, 5, "dropped", 1), (40, 8, 8, "even", 100), (300, 2, 4, "one", 7),
         (257, 4, 9, "skewed", 264), (64, 1, 64, "even", 1000), (33, 2, 3, "none", 128), (90, 5, 6, "dropped", 2050)]


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("layout", ["plain", "wide", "shifted"])
@pytest.mark.parametrize("t,k,e,how,width", MOVES)
def test_moves(ops, t, k, e, how, width, layout, dt):
    """dispatch, dispatch8, combine and their gradients; rows behind the last
    segment and rows that no slot names are NaN and must reach nothing."""
    dtype = DT[dt]
    pad, shift = {"plain": (0, 0), "wide": (8, 0), "shifted": (3, 1)}[layout]
    idx = choices(t, t, k, e, how)
    r = ops.Route(t, k, e).order(torch.from_numpy(idx).cuda())
    offs, perm, row = R.order(idx, e)
    n = perm.size
    x, dout = (strided(rnd(i, t, width, dtype=dtype), pad, shift) for i in (1, 2))
    w = rnd(3, t, k)
    y = rnd(4, n, width, dtype=dtype)
    y[torch.from_numpy(perm < 0).cuda()] = float("nan")
    y = strided(y, pad, shift)
    ww = R.as64(w).copy()
    live = perm >= 0

    out = strided(torch.full((n, width), 7.0, dtype=dtype, device="cuda"), pad, shift)
    xs = R.as64(r.dispatch(x, out=out))
    want = np.zeros((n, width))
    want[live] = R.as64(x)[perm[live] // k]
    want[offs[-1]:] = 7.0
    assert np.array_equal(xs, want)

    t8 = ops.empty8(n, width)
    t8.codes.fill_(0x55)
    t8.scales.fill_(0x33)
    r.dispatch8(x, out=t8)
    codes, scales = R.quant(want[:offs[-1]])
    assert np.array_equal(t8.codes.cpu().numpy()[:offs[-1], :width], codes)
    assert np.array_equal(t8.scales.cpu().numpy()[:offs[-1]], scales)
    assert (t8.codes[offs[-1]:] == 0x55).all() and (t8.scales[offs[-1]:] == 0x33).all()

    yy = np.where(live[:, None], R.as64(y), 0.0)
    for weights in (w, None):
        got = r.combine(y, weights)
        wk = ww if weights is not None else np.ones_like(ww)
        term = np.where((row >= 0)[:, :, None], yy[np.maximum(row, 0)] * wk[:, :, None], 0.0)
        ref = term.sum(1)
        close(got, ref, (k + 1) * U32 * np.abs(term).sum(1) + HALF_STEP[dtype] * np.abs(ref) * (1 + 1e-3), "combine")

    dy = strided(torch.full((n, width), 7.0, dtype=dtype, device="cuda"), pad, shift)
    dy, dw = r.combine_bwd(dout, y, w, dy=dy)
    dd = R.as64(dout)
    ref = np.zeros((n, width))
    ref[live] = dd[perm[live] // k] * ww.reshape(-1)[perm[live]][:, None]
    ref[offs[-1]:] = 7.0
    close(dy, ref, (U32 + HALF_STEP[dtype] * (1 + 1e-3)) * np.abs(ref), "dy")
    prod = np.where((row >= 0)[:, :, None], dd[:, None, :] * yy[np.maximum(row, 0)], 0.0)
    close(dw, prod.sum(-1), (width + 1) * U32 * np.abs(prod).sum(-1), "dw")
    ops.check()


def test_move_gradients_by_differences(ops):
    """d<combine(dispatch-like y, w), g>/dy and /dw against central differences
    of the operator itself (fp32; the map is linear in y and in w, so the
    difference quotient has rounding error alone: 2 eps terms / step)."""
    t, k, e, width = 9, 2, 4, 12
    r = ops.Route(t, k, e).order(torch.from_numpy(choices(5, t, k, e, "dropped")).cuda())
    y, w, g = rnd(1, r.rows, width), rnd(2, t, k), rnd(3, t, width)
    dy, dw = r.combine_bwd(g, y, w, dy=torch.zeros(r.rows, width, device="cuda"))
    f = lambda yy, ww: float((r.combine(yy, ww).double() * g.double()).sum())  # noqa: E731
    h = 0.5
    scale = float((g.abs().sum() * (y.abs().max() + h) * (w.abs().max() + h)))
    tol = 2 * 4 * U32 * scale / (2 * h)
    for i in (int(r.row[r.row >= 0][0]), int(r.row.max())):
        d = torch.zeros_like(y)
        d[i, 5] = h
        assert abs((f(y + d, w) - f(y - d, w)) / (2 * h) - float(dy[i, 5])) <= tol
    for i in range(t):
        d = torch.zeros_like(w)
        d[i, 1] = h
        assert abs((f(y, w + d) - f(y, w - d)) / (2 * h) - float(dw[i, 1])) <= tol
    x, gs = rnd(4, t, width), rnd(5, r.rows, width)
    dx = r.dispatch_bwd(gs)
    d = torch.zeros_like(x)
    d[4] = h
    q = ((r.dispatch(x + d, out=torch.zeros_like(gs)) - r.dispatch(x - d, out=torch.zeros_like(gs))).double()
         * gs.double()).sum() / (2 * h)
    assert abs(float(q) - float(dx[4].double().sum())) <= tol


# ---------------------------------------------------------------------------
# 8 bits and back
# ---------------------------------------------------------------------------
def specials(rows, cols, seed=0):
    """Values across the range of fp32, with borders, subnormals, zeros, infinities and NaN."""
    g = np.random.default_rng(seed)
    x = (g.normal(size=(rows, cols)) * 2.0 ** g.integers(-40, 40, (rows, 1))).astype(np.float32)
    x[0] = 0
    if rows > 6:
        x[1, ::2] = 448.0
        x[2] = np.float32(448.0) * (1 + 2.0 ** -23)
        x[3] = 2.0 ** -140                       # subnormal: the exponent stops at -126
        x[4, 0], x[4, -1] = np.inf, np.nan
        x[5] = -np.inf
        x[6] = 3.0e38 * np.sign(x[6])
    return x


QUANT = [(1, 1), (1, 768), (7, 100), (128, 128), (130, 264), (300, 1000), (33, 2050)]


def codes_equal(t, want, what):
    codes, scales = want
    assert np.array_equal(t.scales.cpu().numpy(), scales), what
    assert np.array_equal(t.codes.cpu().numpy()[:, :t.cols], codes), what


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,cols", QUANT)
def test_quant_codes(ops, rows, cols, dt):
    """Every code and scale byte, straight and transposed, over plain and
    strided rows; and the values read back."""
    x = torch.from_numpy(specials(rows, cols)).to(DT[dt]).cuda()
    x64 = R.as64(x)
    for v in (x, strided(x, 8), strided(x, 3, 1)):
        codes_equal(ops.quant8(v), R.quant(x64), "rows")
        codes_equal(ops.quant8(v, block_rows=128), R.quant(x64, 128), "blocks")
        codes_equal(ops.quant8_t(v), R.quant(x64.T), "columns")
        codes_equal(ops.quant8_t(v, block_rows=128), R.quant(x64.T, 128), "blocks transposed")
    t = ops.quant8(x)
    val = R.value8(t)
    assert np.array_equal(R.as64(ops.dequant8(t, torch.float32)), val, equal_nan=True)
    out = strided(torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda"), 3, 1)
    assert np.array_equal(R.as64(ops.dequant8(t, out=out)), R.rounded(val, torch.bfloat16), equal_nan=True)
    # a saved matrix transposed: quantised again from its values
    codes_equal(ops.quant8_t(t), R.quant(np.where(np.isnan(val), np.nan, val).T), "from 8 bits")
    codes_equal(ops.quant8_t(t, block_rows=128), R.quant(val.T, 128), "from 8 bits, blocks")


@pytest.mark.parametrize("cols", [2, 200, 256, 514, 1024])
def test_quant_halves(ops, cols):
    x = torch.from_numpy(specials(20, cols, 1)).cuda()
    t = ops.quant8(x, halves=True)
    codes_equal(t, R.quant(R.as64(x), halves=True), cols)
    assert np.array_equal(R.as64(ops.dequant8(t, torch.float32)), R.value8(t), equal_nan=True)


@pytest.mark.parametrize("shape", [(3, 100, 200), (2, 128, 128), (1, 1, 5), (4, 257, 96)])
def test_quant_stacks(ops, shape):
    x = rnd(1, *shape)
    x64 = R.as64(x)
    for t, tr in ((ops.quant8(x), False), (ops.quant8(x, 128), False), (ops.quant8_t(x), True), (ops.quant8_t(x, 128), True)):
        for i in range(shape[0]):
            codes_equal(t[i], R.quant(x64[i].T if tr else x64[i], t.block_rows), (i, tr))


@pytest.mark.parametrize("limit", [-5, 0, 128, 384, 1000])
def test_row_limits(ops, limit):
    """Only rows below the device's count are written, in every operator that takes one."""
    rows, cols = 500, 272
    n = torch.tensor([limit], dtype=torch.int32, device="cuda")
    m = min(max(limit, 0), rows)
    x = rnd(2, rows, cols)
    a = ops.empty8(rows, cols)
    b = ops.empty8(cols, rows)
    c = ops.empty8(rows, cols // 2)
    s = ops.empty8(rows, cols, halves=True)
    for t in (a, b, c, s):
        t.codes.fill_(0x55)
        t.scales.fill_(0x33)
    ops.quant8(x, out=a, n_rows=n)
    ops.quant8_t(x, out=b, n_rows=n)
    ops.swiglu8(x, act=c, saved=s, n_rows=n)
    want, wt = R.quant(R.as64(x)), R.quant(R.as64(x).T)
    assert np.array_equal(a.codes.cpu().numpy()[:m, :cols], want[0][:m]) and (a.codes[m:] == 0x55).all()
    assert np.array_equal(a.scales.cpu().numpy()[:m], want[1][:m]) and (a.scales[m:] == 0x33).all()
    assert np.array_equal(b.codes.cpu().numpy()[:, :m], wt[0][:, :m]) and (b.codes[:, m:] == 0x55).all()
    mb = -(-m // 128)
    assert np.array_equal(b.scales.cpu().numpy()[:, :mb], wt[1][:, :mb]) and (b.scales[:, mb:] == 0x33).all()
    for t in (c, s):
        assert (t.codes[m:] == 0x55).all() and (t.scales[m:] == 0x33).all()
    codes, scales = R.quant(R.as64(x), halves=True)
    assert np.array_equal(s.codes.cpu().numpy()[:m, :cols], codes[:m])
    full = ops.quant8(x, halves=True)
    d = torch.full((rows, cols), 7.0, device="cuda")
    ops.dequant8(full, out=d, n_rows=n)
    assert (d[m:] == 7).all() and np.array_equal(R.as64(d[:m]), R.value8(full)[:m])
    d.fill_(7.0)
    ops.swiglu8_bwd(x[:, :cols // 2], full, dgu=d, n_rows=n)
    assert (d[m:] == 7).all() and not (d[:m] == 7).any()


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------
def product_close(got, a, b, dtype, k, extra=0.0):
    """Sums of k exact products: at most k roundings (of up to a whole step, 2 U32) of partial sums no
    larger than the sum of magnitudes."""
    ref, mag = a @ b.T + extra, np.abs(a) @ np.abs(b).T + np.abs(extra)
    close(got, ref, (k + 2) * 2 * U32 * mag + HALF_STEP[dtype] * np.abs(ref) * (1 + 1e-3))


PRODUCTS = [(1, 1, 1), (1, 2304, 768), (2, 8, 16), (100, 72, 130), (128, 256, 128), (129, 257, 129), (300, 1000, 777),
            (700, 640, 512), (1000, 2000, 200), (513, 64, 2300)]


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_gemm_dense(ops, m, n, k, block_rows, dt):
    a = ops.quant8(rnd(1, m, k))
    b = ops.quant8(rnd(2, n, k, std=0.02), block_rows=block_rows)
    av, bv = R.value8(a), R.value8(b)
    product_close(ops.gemm8(a, b, dtype=DT[dt]), av, bv, DT[dt], k)
    for pad, shift in ((8, 0), (3, 1)):
        buf = torch.full((m, n + pad + shift), 7.0, dtype=DT[dt], device="cuda")
        product_close(ops.gemm8(a, b, out=buf[:, shift:shift + n]), av, bv, DT[dt], k)
        assert (buf[:, :shift] == 7).all() and (buf[:, shift + n:] == 7).all()
        if dt == "fp32":
            buf[:, shift:shift + n] = rnd(5, m, n)
            before = R.as64(buf[:, shift:shift + n])
            product_close(ops.gemm8(a, b, out=buf[:, shift:shift + n], accumulate=True), av, bv, DT[dt], k, before)
            assert (buf[:, :shift] == 7).all() and (buf[:, shift + n:] == 7).all()
    ops.check()


SEGMENTS = [[0, 128], [0, 0, 0], [0, 128, 128, 384], [0, 0, 256, 256, 640, 640], [0, 1280]]


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("offs", SEGMENTS)
@pytest.mark.parametrize("n,k", [(72, 130), (264, 256), (1024, 100)])
def test_gemm_by_expert(ops, offs, n, k, block_rows, dt):
    rows, e = 1280, len(offs) - 1
    a = ops.quant8(rnd(1, rows, k))
    a.codes[offs[-1]:] = 0x7F                          # behind the last segment: NaN
    b = ops.quant8(rnd(2, e, n, k, std=0.02), block_rows=block_rows)
    out = torch.full((rows, n), 7.0, dtype=DT[dt], device="cuda")
    ops.gemm8(a, b, out=out, offs=torch.tensor(offs, dtype=torch.int32, device="cuda"))
    av, bv = R.value8(a), R.value8(b)
    for i in range(e):
        product_close(out[offs[i]:offs[i + 1]], av[offs[i]:offs[i + 1]], bv[i], DT[dt], k)
    assert (out[offs[-1]:] == 7).all()
    ops.check()


@pytest.mark.parametrize("offs", SEGMENTS + [[0, 1152, 1280]])
@pytest.mark.parametrize("m,n", [(16, 40), (130, 257), (256, 768), (33, 1000)])
def test_gemm_reduce(ops, offs, m, n):
    p, e = 1280, len(offs) - 1
    a, b = ops.quant8_t(rnd(1, p, m)), ops.quant8_t(rnd(2, p, n))
    a.codes[:, offs[-1]:] = 0x7F
    o = torch.tensor(offs, dtype=torch.int32, device="cuda")
    av, bv = R.value8(a), R.value8(b)
    for pad, shift in ((0, 0), (3, 1)):
        buf = torch.full((e, m, n + pad + shift), 7.0, device="cuda")
        out = buf[:, :, shift:shift + n]
        for acc in (False, True):
            before = R.as64(out) if acc else np.zeros((e, m, n))
            ops.gemm8_reduce(a, b, o, out=out, accumulate=acc)
            for i in range(e):
                s = slice(offs[i], offs[i + 1])
                product_close(out[i], av[:, s], bv[:, s], torch.float32, offs[i + 1] - offs[i], before[i])
        assert (buf[:, :, :shift] == 7).all() and (buf[:, :, shift + n:] == 7).all()
    ops.check()


@pytest.mark.parametrize("p", [1, 100, 300, 1263])
def test_gemm_reduce_of_lengths_off_blocks(ops, p):
    """The last segment ends at the length rounded up to 128: its last block is
    a part of one."""
    end = -(-p // 128) * 128
    a, b = ops.quant8_t(rnd(1, p, 70)), ops.quant8_t(rnd(2, p, 200))
    av, bv = R.value8(a), R.value8(b)
    for offs in ([0, end], [0, end - 128, end], [0, 0, end, end]):
        out = ops.gemm8_reduce(a, b, torch.tensor(offs, dtype=torch.int32, device="cuda"))
        for i in range(len(offs) - 1):
            s = slice(offs[i], min(offs[i + 1], p))
            product_close(out[i], av[:, s], bv[:, s], torch.float32, max(s.stop - s.start, 0))
    ops.check()


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("lo,hi", [(0, 2), (1, 3), (2, 5), (4, 5), (1, 2)])
def test_gemm_by_some_of_the_experts(ops, lo, hi, dt):
    """A run of consecutive experts of a routing: their rows alone are written."""
    offs, n, k = [0, 256, 256, 640, 1152, 1280], 264, 200
    a, b = ops.quant8(rnd(1, 1300, k)), ops.quant8(rnd(2, 5, n, k, std=0.02), 128)
    o = torch.tensor(offs, dtype=torch.int32, device="cuda")
    some = ops.Tensor8(b.codes[lo:hi], b.scales[lo:hi], k, 128)
    out = torch.full((1300, n), 7.0, dtype=DT[dt], device="cuda")
    ops.gemm8(a, some, out=out, offs=o[lo:hi + 1])
    want = ops.gemm8(a, b, dtype=DT[dt], offs=o)
    s = slice(offs[lo], offs[hi])
    assert torch.equal(out[s], want[s]) and (out[:s.start] == 7).all() and (out[s.stop:] == 7).all()
    ops.check()


def product64(got, a, b, k, dtype, before=None):
    """product_close on the device, for sizes that the host takes too long for."""
    av, bv = (torch.from_numpy(R.value8(t)).cuda() for t in (a, b))
    ref, mag = av @ bv.T, av.abs() @ bv.abs().T
    if before is not None:
        ref, mag = ref + before, mag + before.abs()
    bound = (k + 2) * 2 * U32 * mag + HALF_STEP[dtype] * ref.abs() * (1 + 1e-3)
    bad = (got.double() - ref).abs() > bound
    assert not bad.any(), (int(bad.sum()), float((got.double() - ref).abs().max()))


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("m,n,k", [(2500, 4100, 300), (2560, 4096, 640), (5000, 2049, 129)])
def test_gemm_wide_tiles(ops, m, n, k, block_rows, dt):
    """Products large enough for 256-column tiles, edges on both sides."""
    a = ops.quant8(rnd(1, m, k))
    b = ops.quant8(rnd(2, n, k, std=0.02), block_rows=block_rows)
    product64(ops.gemm8(a, b, dtype=DT[dt]), a, b, k, DT[dt])
    buf = torch.full((m, n + 4), 7.0, dtype=DT[dt], device="cuda")
    product64(ops.gemm8(a, b, out=buf[:, 3:3 + n]), a, b, k, DT[dt])
    assert (buf[:, :3] == 7).all() and (buf[:, 3 + n:] == 7).all()
    if dt == "fp32":
        c = rnd(3, m, n)
        before = c.double()
        product64(ops.gemm8(a, b, out=c, accumulate=True), a, b, k, DT[dt], before)
    ops.check()


@pytest.mark.parametrize("m,n,k", [(1, 70, 4097), (130, 300, 9000), (3000, 4200, 4500)])
def test_gemm_long_sums(ops, m, n, k):
    """Reductions beyond the 4096 that tensor memory sums: rounded fp32 additions
    join the parts, so all of them stay within 2^-21 of the sum of magnitudes (the
    parts' cut-off sums: 128 additions of at most 2^-23 each on a growing sum)."""
    a, b = ops.quant8(rnd(1, m, k) + 0.5), ops.quant8(rnd(2, n, k) + 0.5, block_rows=1)
    c = ops.gemm8(a, b, dtype=torch.float32).double()
    av, bv = (torch.from_numpy(R.value8(t)).cuda() for t in (a, b))
    assert ((c - av @ bv.T).abs() <= 128 * 2.0 ** -23 / 2 * (av.abs() @ bv.abs().T)).all()
    ops.check()


def test_gemm_reduce_long_segments_and_many(ops):
    """Segments of zero to 20000 columns and sixty-four of them."""
    p, m, n, e = 40960, 260, 300, 64
    g = np.random.default_rng(1)
    blocks = g.multinomial(320 - 157, [1.0 / e] * e)
    blocks[5], blocks[9] = 0, blocks[9] + 157
    offs = np.concatenate([[0], np.cumsum(blocks)]) * 128
    a, b = ops.quant8_t(rnd(1, p, m)), ops.quant8_t(rnd(2, p, n))
    out = ops.gemm8_reduce(a, b, torch.from_numpy(offs.astype(np.int32)).cuda())
    av, bv = (torch.from_numpy(R.value8(t)).cuda() for t in (a, b))
    for i in range(e):
        s = slice(int(offs[i]), int(offs[i + 1]))
        ref, mag = av[:, s] @ bv[:, s].T, av[:, s].abs() @ bv[:, s].abs().T
        assert ((out[i].double() - ref).abs() <= (s.stop - s.start + 2) * 2 * U32 * mag).all(), i
    ops.check()


def test_gemm_by_expert_wide(ops):
    """Many rows over sixteen experts, some without any, in wide tiles."""
    g = np.random.default_rng(2)
    e, n, k = 16, 1030, 200
    blocks = g.integers(0, 14, e)
    blocks[3] = blocks[15] = 0
    offs = np.concatenate([[0], np.cumsum(blocks)]) * 128
    rows = int(offs[-1]) + 300
    a = ops.quant8(rnd(1, rows, k))
    a.codes[int(offs[-1]):] = 0x7F
    b = ops.quant8(rnd(2, e, n, k, std=0.02), 128)
    out = torch.full((rows, n), 7.0, device="cuda")
    ops.gemm8(a, b, out=out, offs=torch.from_numpy(offs.astype(np.int32)).cuda())
    for i in range(e):
        s = slice(int(offs[i]), int(offs[i + 1]))
        if s.stop > s.start:
            product64(out[s], a.part(s.start, s.stop), b[i], k, torch.float32)
    assert (out[int(offs[-1]):] == 7).all()
    ops.check()


def test_gemm_scale_rows_of_any_stride(ops):
    """Scale bytes whose rows start anywhere (read by bytes) and by words agree."""
    a, b = ops.quant8(rnd(1, 300, 900)), ops.quant8(rnd(2, 200, 900))
    want = ops.gemm8(a, b, dtype=torch.float32)
    for t in (0, 1):
        m = (a, b)[t]
        buf = torch.empty(m.rows * 9 + 1, dtype=torch.uint8, device="cuda")
        odd = buf[1:].view(m.rows, 9)[:, :8]
        odd.copy_(m.scales)
        o = ops.Tensor8(m.codes, odd, m.cols)
        got = ops.gemm8(o if t == 0 else a, o if t else b, dtype=torch.float32)
        assert torch.equal(got, want)
    ops.check()


def test_gemm_keeps_nan_and_large_scales_in_their_rows(ops):
    x = rnd(1, 200, 300)
    x[17, 5] = float("nan")
    x[60] *= 2.0 ** 100
    x[61] *= 2.0 ** -60
    w = rnd(2, 90, 300, std=2.0 ** -30)
    a, b = ops.quant8(x), ops.quant8(w, block_rows=128)
    c = ops.gemm8(a, b, dtype=torch.float32)
    assert torch.isnan(c[17]).all() and torch.isfinite(torch.cat([c[:17], c[18:]])).all()
    keep = np.arange(200) != 17
    product_close(c[torch.from_numpy(keep).cuda()], R.value8(a)[keep], R.value8(b), torch.float32, 300)


@pytest.mark.parametrize("sa,sb", [(127, 127), (1, 127), (0, 127), (254, 1), (254, 0), (64, 64), (200, 60), (255, 127)])
def test_gemm_extreme_scale_bytes(ops, sa, sb):
    """Scale bytes over their whole range, where the sum is a normal fp32 number;
    zero times any finite scale is zero, and 255 is NaN."""
    a, b = ops.empty8(128, 128), ops.empty8(64, 128)
    a.codes.fill_(0x38)
    a.codes[64:] = 0
    b.codes.fill_(0x38)
    a.scales.fill_(sa)
    b.scales.fill_(sb)
    c = ops.gemm8(a, b, dtype=torch.float32)
    if sa == 255:
        assert torch.isnan(c).all()
    else:
        assert (c[:64].double() == 128 * 2.0 ** (sa + sb - 254)).all() and (c[64:] == 0).all()
    ops.check()


def test_bad_segment_starts_stay_in_bounds(ops):
    """Starts that no routing makes are cut to block boundaries inside the
    operands: no access leaves a buffer, whatever they hold."""
    a, b = ops.quant8(rnd(1, 256, 128)), ops.quant8(rnd(2, 3, 64, 128))
    at, bt = ops.quant8_t(rnd(1, 256, 128)), ops.quant8_t(rnd(2, 256, 64))
    for o in ([0, 100, 5000, 2 ** 31 - 1], [-128, 300, 200, 100], [2 ** 31 - 1, 0, -2 ** 31, 77]):
        o = torch.tensor(o, dtype=torch.int32, device="cuda")
        ops.gemm8(a, b, offs=o)
        ops.gemm8_reduce(at, bt, o)
    ops.check()


# ---------------------------------------------------------------------------
# SwiGLU
# ---------------------------------------------------------------------------
def gu_values(rows, width, dtype):
    x = rnd(7, rows, 2 * width)
    x[0] = 0
    if rows > 4:
        x[1, :width] = 100.0
        x[2, :width] = -100.0
        x[3] *= 2.0 ** -60
        x[4, :width] = -20.0
    return x.to(dtype)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,width", [(1, 512), (2, 1), (5, 7), (130, 128), (200, 264), (19, 1040)])
def test_swiglu(ops, rows, width, dt):
    """The 8-bit results lie within half a step of the exact ones plus the
    fp32 error of silu(g) u: (|g| + 8) 2^-22 relative (the exponential's
    2 + 1.2 |g| ulp, the quotient's 2 and three roundings)."""
    for pad, shift in ((0, 0), (3, 1)):
        gu = strided(gu_values(rows, width, DT[dt]), pad, shift)
        saved = ops.empty8(rows, 2 * width, halves=True)
        act = ops.swiglu8(gu, saved=saved)
        g, u = np.split(R.as64(gu), 2, axis=1)
        codes_equal(saved, R.quant(R.as64(gu), halves=True), "saved")
        exact = g * R.sigmoid(g) * u
        err = (np.abs(g) + 8) * 2.0 ** -22 * np.abs(exact) + 1e-37 * (1 + np.abs(u))
        val = R.value8(act)
        s = 2.0 ** (np.repeat(act.scales.cpu().numpy(), 128, 1)[:, :width].astype(float) - 127)
        step = np.maximum(2.0 ** -4 * np.abs(exact), 2.0 ** -10 * s)
        close(val, exact, step * (1 + 2.0 ** -4) + err, "act")
        # scales: the least that holds the block, up to that error at a border
        for c in range(0, width, 128):
            top, slack = np.abs(exact[:, c:c + 128]).max(1), err[:, c:c + 128].max(1)
            sc = s[:, c]
            assert (top - slack <= 448 * sc).all()
            assert ((top + slack > 224 * sc) | (sc == 1) | (sc == 2.0 ** -126)).all()
        only = ops.swiglu8(gu)
        assert torch.equal(only.codes[:, :width], act.codes[:, :width]) and torch.equal(only.scales, act.scales)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,width", [(1, 512), (2, 1), (5, 7), (130, 128), (200, 264), (19, 1040)])
def test_swiglu_backward(ops, rows, width, dt):
    dtype = DT[dt]
    saved = ops.quant8(gu_values(rows, width, torch.float32), halves=True)
    g, u = np.split(R.value8(saved), 2, axis=1)
    for pad, shift in ((0, 0), (3, 1)):
        da = strided(rnd(8, rows, width, dtype=dtype), pad, shift)
        act = strided(torch.zeros(rows, width, dtype=dtype, device="cuda"), pad, shift)
        dgu = strided(torch.zeros(rows, 2 * width, dtype=dtype, device="cuda"), pad, shift)
        ops.swiglu8_bwd(da, saved, dgu=dgu, act=act)
        d, s = R.as64(da), R.sigmoid(g)
        rel = (np.abs(g) + 8) * 2.0 ** -22
        tiny = 1e-37 * (1 + np.abs(d)) * (1 + np.abs(u))
        for got, ref, mag in ((dgu[:, :width], d * u * s * (1 + g * (1 - s)), np.abs(d * u) * (s + np.abs(g) * s)),
                              (dgu[:, width:], d * g * s, np.abs(d * g * s)), (act, g * s * u, np.abs(g * s * u))):
            close(got, ref, rel * mag + tiny + HALF_STEP[dtype] * np.abs(ref) * (1 + 1e-2))


@pytest.mark.parametrize("width", [128, 264, 512])
def test_swiglu_with_infinities_and_nan(ops, width):
    """An infinity or NaN spoils its own elements alone: the rest of its block is
    as without it."""
    x = gu_values(40, width, torch.float32)
    bad = x.clone()
    bad[7, 3], bad[9, width + 5], bad[11, 0], bad[11, width] = float("nan"), float("inf"), float("-inf"), 0.0
    bad[20] = float("inf")
    saved = ops.empty8(40, 2 * width, halves=True)
    act = ops.swiglu8(bad, saved=saved)
    codes_equal(saved, R.quant(R.as64(bad), halves=True), "saved")
    v = R.value8(act)
    clean = x.clone()                              # what the others see: zeros in the spoilt places
    clean[7, 3] = clean[9, width + 5] = clean[11, 0] = clean[11, width] = 0.0
    clean[20] = 0.0
    w = R.value8(ops.swiglu8(clean))
    spoilt = np.zeros((40, width), bool)
    spoilt[7, 3] = spoilt[9, 5] = spoilt[11, 0] = True
    spoilt[20] = True
    assert np.isnan(v[spoilt]).all() and np.array_equal(v[~spoilt], w[~spoilt])


def test_swiglu_backward_by_differences(ops):
    """dgu against central differences of silu(g) u in float64 at the saved
    values: error h^2/6 of a third derivative below 1, plus the fp32 bound."""
    saved = ops.quant8(rnd(3, 40, 64), halves=True)
    g, u = np.split(R.value8(saved), 2, axis=1)
    da = rnd(4, 40, 32)
    dgu, d, h = R.as64(ops.swiglu8_bwd(da, saved)), R.as64(da), 1e-4
    f = lambda g, u: g * R.sigmoid(g) * u  # noqa: E731
    num = np.concatenate([(f(g + h, u) - f(g - h, u)) / (2 * h), (f(g, u + h) - f(g, u - h)) / (2 * h)], 1)
    dd = np.concatenate([d, d], 1)
    size = np.abs(dd) * (1 + np.abs(np.concatenate([u, g], 1))) * (1 + np.abs(np.concatenate([g, g], 1)))
    close(dgu, dd * num, size * (h * h + 1e-11 / h + 20 * 2.0 ** -22))


# ---------------------------------------------------------------------------
# streams, graphs, repetition
# ---------------------------------------------------------------------------
def chain(ops, r, idx, x, w8, wd8, w, bufs):
    """Order, gather in 8 bits, product, SwiGLU, product, combine."""
    xs8, gu, act8, saved, y, out = bufs
    r.order(idx)
    r.dispatch8(x, out=xs8)
    ops.gemm8(xs8, w8, out=gu, offs=r.offs)
    ops.swiglu8(gu, act=act8, saved=saved, n_rows=r.offs[-1:])
    ops.gemm8(act8, wd8, out=y, offs=r.offs)
    return r.combine(y, w, out=out)


def chain_inputs(ops, seed, t=300, k=2, e=6, d=256, f=136):
    r = ops.Route(t, k, e)
    idx = torch.from_numpy(choices(seed, t, k, e, "dropped")).cuda()
    x = rnd(seed, t, d, dtype=torch.bfloat16)
    w8 = ops.quant8(rnd(seed + 1, e, 2 * f, d, std=0.05), 128)
    wd8 = ops.quant8(rnd(seed + 2, e, d, f, std=0.05), 128)
    w = torch.softmax(rnd(seed + 3, t, k), 1)
    n = r.rows
    bufs = (ops.empty8(n, d), torch.zeros(n, 2 * f, dtype=torch.bfloat16, device="cuda"), ops.empty8(n, f),
            ops.empty8(n, 2 * f, halves=True), torch.zeros(n, d, dtype=torch.bfloat16, device="cuda"),
            torch.zeros(t, d, dtype=torch.bfloat16, device="cuda"))
    return r, idx, x, w8, wd8, w, bufs


def test_chain_matches_definition(ops):
    """The forward chain against float64 steps, each taking the device's own
    8-bit operands, so that every bound stays one step's."""
    r, idx, x, w8, wd8, w, bufs = chain_inputs(ops, 1)
    out = chain(ops, r, idx, x, w8, wd8, w, bufs)
    xs8, gu, act8, saved, y, _ = bufs
    offs, perm, row = R.order(idx.cpu().numpy(), 6)
    live = perm >= 0
    end = offs[-1]
    xs = np.zeros((perm.size, 256))
    xs[live] = R.as64(x)[perm[live] // 2]
    assert np.array_equal(xs8.codes.cpu().numpy()[:end], R.quant(xs[:end])[0])
    xv, av, wv, wdv = R.value8(xs8), R.value8(act8), R.value8(w8), R.value8(wd8)
    for e in range(6):
        s = slice(offs[e], offs[e + 1])
        product_close(gu[s], xv[s], wv[e], torch.bfloat16, 256)
        product_close(y[s], av[s], wdv[e], torch.bfloat16, 136)
    g, u = np.split(R.as64(gu)[:end], 2, axis=1)
    ref = g * R.sigmoid(g) * u
    sc = 2.0 ** (np.repeat(act8.scales.cpu().numpy()[:end], 128, 1)[:, :136].astype(float) - 127)
    close(av[:end], ref, np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * sc) * (1 + 2.0 ** -4) + 1e-5 * np.abs(ref))
    yy, ww = np.where(live[:, None], R.as64(y), 0.0), R.as64(w)
    term = np.where((row >= 0)[:, :, None], yy[np.maximum(row, 0)] * ww[:, :, None], 0.0)
    close(out, term.sum(1), 3 * U32 * np.abs(term).sum(1) + 2.0 ** -8 * 1.001 * np.abs(term.sum(1)))


def test_chain_captured_and_replayed(ops):
    """A captured chain gives the eager result bit for bit, also on inputs
    written after the capture, and on a stream of its own."""
    a = chain_inputs(ops, 1)
    want = chain(ops, *a).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = chain_inputs(ops, 1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        chain(ops, *b)
    for t in b[6][1:2] + b[6][4:]:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(b[6][5], want)
    c = chain_inputs(ops, 9)
    want = chain(ops, *c).clone()
    b[1].copy_(c[1])
    b[2].copy_(c[2])
    b[5].copy_(c[5])
    for dst, src in ((b[3], c[3]), (b[4], c[4])):
        dst.codes.copy_(src.codes)
        dst.scales.copy_(src.scales)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(b[6][5], want)
    ops.check()


def test_two_streams_at_once(ops):
    one, two = chain_inputs(ops, 1, t=2000), chain_inputs(ops, 2, t=1500, e=11)
    w1, w2 = chain(ops, *one).clone(), chain(ops, *two).clone()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            chain(ops, *one)
        with torch.cuda.stream(s2):
            chain(ops, *two)
    torch.cuda.synchronize()
    assert torch.equal(one[6][5], w1) and torch.equal(two[6][5], w2)
    ops.check()


def test_streams_joined_by_events(ops):
    """Each step on a stream of its own, ordered by events alone, gives the
    result of one stream."""
    r, idx, x, w8, wd8, w, bufs = chain_inputs(ops, 3, t=3000)
    want = chain(ops, r, idx, x, w8, wd8, w, bufs).clone()
    xs8, gu, act8, saved, y, out = bufs
    torch.cuda.synchronize()
    steps = (lambda: r.order(idx), lambda: r.dispatch8(x, out=xs8), lambda: ops.gemm8(xs8, w8, out=gu, offs=r.offs),
             lambda: ops.swiglu8(gu, act=act8, saved=saved, n_rows=r.offs[-1:]),
             lambda: ops.gemm8(act8, wd8, out=y, offs=r.offs), lambda: r.combine(y, w, out=out))
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(5):
        for t in (r.row, gu, y, out, xs8.codes, act8.codes):
            t.zero_()
        done = torch.cuda.current_stream().record_event()
        for s, f in zip(streams, steps):
            s.wait_event(done)
            with torch.cuda.stream(s):
                f()
                done = s.record_event()
        torch.cuda.current_stream().wait_event(done)
        assert torch.equal(out, want)
    ops.check()


def test_steps_mixed_with_other_kernels(ops):
    """Operators between plain tensor kernels that write what they read and
    read what they write, many in a row without waiting: no step starts on old
    data."""
    t, k, e, d = 4096, 2, 8, 512
    r = ops.Route(t, k, e)
    idx = torch.from_numpy(choices(1, t, k, e, "even")).cuda()
    r.order(idx)
    x, xs, back = torch.zeros(t, d, device="cuda"), torch.zeros(r.rows, d, device="cuda"), torch.zeros(t, d, device="cuda")
    for i in range(40):
        x.fill_(i + 1.0)
        r.dispatch(x, out=xs)
        xs.mul_(2.0)
        r.combine(xs, out=back)
        assert_later = back.sum() if i % 8 == 7 else None
        if assert_later is not None:
            assert float(assert_later) == float(t * d) * k * 2.0 * (i + 1.0)
    ops.check()


def test_wrapper_refusals(ops):
    x = rnd(1, 10, 64)
    r = ops.Route(10, 2, 4)
    with pytest.raises(ValueError):
        r.dispatch(x[:9])
    with pytest.raises(ValueError):
        r.dispatch(x.t().contiguous().t())
    with pytest.raises(TypeError):
        r.dispatch(x.half())
    with pytest.raises(TypeError):
        r.dispatch(x, out=torch.empty(r.rows, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        r.order(torch.zeros(10, 2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        r.combine(torch.zeros(r.rows, 64, device="cuda"), torch.zeros(10, 2, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        ops.quant8(x.expand(3, 10, 64))
    with pytest.raises(ValueError):
        ops.quant8(x, out=ops.empty8(10, 65))
    with pytest.raises(ValueError):
        ops.swiglu8(x[:, :63])
    a, b = ops.quant8(x), ops.quant8(x[:, :63].contiguous())
    from adamw_persistent_sm_gb300.trainer import StatusError
    with pytest.raises(StatusError):
        ops.gemm8(a, b)
    with pytest.raises(StatusError):
        ops.gemm8(a, ops.quant8(x), dtype=torch.bfloat16, out=torch.zeros(10, 10, dtype=torch.bfloat16, device="cuda"),
                  accumulate=True)
    with pytest.raises(StatusError):
        ops.dequant8(ops.quant8(x, block_rows=128))
    with pytest.raises(ValueError):
        ops.Tensor8(a.codes[:, :48], a.scales, 48)


def test_no_tokens(ops):
    """A routing of no tokens: every move runs and writes nothing."""
    r = ops.Route(0, 2, 4).order(torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    assert (r.offs == 0).all() and (r.perm == -1).all()
    x, w = torch.empty(0, 64, device="cuda"), torch.empty(0, 2, device="cuda")
    xs = torch.full((r.rows, 64), 7.0, device="cuda")
    assert r.dispatch(x, out=xs) is xs and (xs == 7).all()
    r.dispatch8(x)
    assert r.combine(xs, w).shape == (0, 64)
    dy, dw = r.combine_bwd(x, xs, w)
    assert dy.shape == (r.rows, 64) and dw.shape == (0, 2)
    ops.check()


def test_refusals_leave_the_device_as_it_was(ops, monkeypatch):
    """With another device current, a refused argument raises before the device
    changes, or changes it back."""
    x, r = rnd(1, 128, 64), ops.Route(128, 2, 4)
    a, saved, bad = ops.quant8(x), ops.quant8(x, halves=True), torch.zeros(2, dtype=torch.int32, device="cuda")
    xs, w, t = torch.zeros(r.rows, 64, device="cuda"), torch.zeros(128, 2, device="cuda"), ops.quant8_t(x)
    now = [7]
    monkeypatch.setattr(ops, "_current", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "set_device", lambda d: now.__setitem__(0, d))
    for call in (lambda: ops.quant8(x, n_rows=bad), lambda: ops.quant8_t(x, n_rows=bad),
                 lambda: ops.dequant8(a, n_rows=bad), lambda: ops.gemm8_reduce(t, t, bad.view(1, 2)),
                 lambda: ops.gemm8(a, a, offs=bad[:1]), lambda: ops.swiglu8(x, n_rows=bad),
                 lambda: ops.swiglu8_bwd(x[:, :32], saved, n_rows=bad), lambda: r.order(bad),
                 lambda: r.combine(xs, w.half()), lambda: r.combine_bwd(x, xs, w.half()),
                 lambda: r.combine_bwd(x, xs, w, dw=w.half())):
        with pytest.raises(ValueError):
            call()
        assert now == [7]


def with_bytes(ops, rows, cols, byte, halves=False, below=0x40):
    """Codes over the positive and negative ones below `below`, all scales one byte."""
    t = ops.empty8(rows, cols, halves=halves)
    g = torch.Generator().manual_seed(byte + 1)
    q = torch.randint(0, below, t.codes.shape, generator=g) + 128 * torch.randint(0, 2, t.codes.shape, generator=g)
    t.codes.copy_(q.to(torch.uint8).cuda())
    t.scales.fill_(byte)
    return t


@pytest.mark.parametrize("byte", [0, 1, 127, 254, 255])
def test_scale_bytes_mean_the_same_everywhere(ops, byte):
    """Bytes over their whole range stand for 2^(byte - 127), 255 for NaN, in
    every operator that reads codes as they do in products: restored values
    are exact (0 gives numbers down to 2^-136, subnormal in fp32), and so are
    the codes of their transpose."""
    rows, cols = 130, 200
    t = with_bytes(ops, rows, cols, byte)
    val = R.value8(t) if byte < 255 else np.full((rows, cols), np.nan)
    for dtype in (torch.float32, torch.bfloat16):
        assert np.array_equal(R.as64(ops.dequant8(t, dtype)), R.rounded(val, dtype), equal_nan=True)
    codes_equal(ops.quant8_t(t), R.quant(val.T), "columns")
    codes_equal(ops.quant8_t(t, block_rows=128), R.quant(val.T, 128), "blocks")
    h = with_bytes(ops, rows, cols, byte, halves=True)
    val = R.value8(h) if byte < 255 else np.full((rows, cols), np.nan)
    assert np.array_equal(R.as64(ops.dequant8(h, torch.float32)), R.rounded(val, torch.float32), equal_nan=True)
    eye = ops.quant8(torch.eye(cols, device="cuda"))
    c = R.as64(ops.gemm8(t, eye, dtype=torch.float32))
    if byte == 255:
        assert np.isnan(c).all()
    elif byte > 0:                       # a product's sums are normal numbers
        assert np.array_equal(c, R.value8(t))


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("bg,bu", [(0, 127), (127, 0), (0, 0), (1, 1), (255, 127), (127, 255)])
def test_swiglu_backward_reads_every_scale_byte(ops, bg, bu, dt):
    """g or u under the least scales, with gradients large enough that the
    results are normal numbers: the bound of test_swiglu_backward, and half a
    step of the subnormal products on the way (2^-150 each, times dact)."""
    rows, width, dtype = 20, 136, DT[dt]
    saved = with_bytes(ops, rows, 2 * width, 0, halves=True)
    saved.scales[:, :2], saved.scales[:, 2:] = bg, bu
    da = rnd(3, rows, width, std=2.0 ** 60, dtype=dtype)
    act = torch.zeros(rows, width, dtype=dtype, device="cuda")
    dgu = ops.swiglu8_bwd(da, saved, act=act)
    g, u = np.split(R.value8(saved), 2, axis=1)
    g, u = (np.full_like(v, np.nan) if b == 255 else v for v, b in ((g, bg), (u, bu)))
    d, s = R.as64(da), R.sigmoid(g)
    rel = (np.abs(g) + 8) * 2.0 ** -22
    sub = 2.0 ** -149 * (1 + np.abs(d)) * (1 + np.abs(u)) + (0 if dt == "fp32" else 2.0 ** -134)
    for got, ref, mag in ((dgu[:, :width], d * u * s * (1 + g * (1 - s)), np.abs(d * u) * (s + np.abs(g) * s)),
                          (dgu[:, width:], d * g * s, np.abs(d * g * s)), (act, g * s * u, np.abs(g * s * u))):
        close(got, ref, rel * mag + sub + HALF_STEP[dtype] * np.abs(ref) * (1 + 1e-2))


def test_check_clears_before_it_returns(ops, monkeypatch):
    """The words are zero on the device when check() raises: a failure that
    another stream reports from then on stays."""
    r = ops.Route(1, 1, 2)
    r.order(torch.full((1, 1), 5, dtype=torch.int32, device="cuda"))
    s, busy = torch.cuda.Stream(), torch.zeros(1 << 26, device="cuda")
    from adamw_persistent_sm_gb300.trainer import StatusError
    torch.cuda.synchronize()
    words = ops._status[r._dev][0]
    real = torch.Tensor.zero_

    def late(t):                             # work of another thread on the stream that clears
        if t is words:
            for _ in range(50):
                busy.add_(1.0)
        return real(t)

    monkeypatch.setattr(torch.Tensor, "zero_", late)
    with pytest.raises(StatusError):
        ops.check()
    monkeypatch.undo()
    with torch.cuda.stream(s):
        r.order(torch.full((1, 1), 7, dtype=torch.int32, device="cuda"))
    with pytest.raises(StatusError):
        ops.check()
    ops.check()


def test_chain_captured_over_several_streams(ops):
    """Each step of a chain captured on a stream of its own, joined by events,
    with a copy between two of them: replays give one stream's result."""
    r, idx, x, w8, wd8, w, bufs = chain_inputs(ops, 4, t=3000)
    want = chain(ops, r, idx, x, w8, wd8, w, bufs).clone()
    xs8, gu, act8, saved, y, out = bufs
    x2 = x.clone()
    steps = (lambda: r.order(idx), lambda: (x2.copy_(x), r.dispatch8(x2, out=xs8)),
             lambda: ops.gemm8(xs8, w8, out=gu, offs=r.offs),
             lambda: ops.swiglu8(gu, act=act8, saved=saved, n_rows=r.offs[-1:]),
             lambda: ops.gemm8(act8, wd8, out=y, offs=r.offs), lambda: r.combine(y, w, out=out))
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        done = main.record_event()
        for s, f in zip(streams, steps):
            s.wait_event(done)
            with torch.cuda.stream(s):
                f()
                done = s.record_event()
        main.wait_event(done)
    for _ in range(4):
        for t in (r.row, r.perm, x2, gu, y, out, xs8.codes, act8.codes):
            t.zero_()
        g.replay()
        assert torch.equal(out, want)
    ops.check()


def test_threads_on_streams_of_their_own(ops):
    """Host threads that launch at once, each on its own stream and buffers, get what one gets."""
    import threading
    chains = [chain_inputs(ops, 10 + i, t=500 + 700 * i) for i in range(4)]
    want = [chain(ops, *c).clone() for c in chains]
    torch.cuda.synchronize()
    failed = []

    def work(c):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    chain(ops, *c)
                torch.cuda.current_stream().synchronize()
        except Exception as e:               # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(c,)) for c in chains]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    assert all(torch.equal(c[6][5], v) for c, v in zip(chains, want))
    ops.check()


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_matrices_of_no_rows(ops, dt):
    x = torch.empty(0, 64, dtype=DT[dt], device="cuda")
    a = ops.quant8(x)
    assert a.shape == (0, 64) and ops.quant8(x, 128).shape == (0, 64) and ops.quant8(x, halves=True).shape == (0, 64)
    assert ops.dequant8(a).shape == (0, 64)
    b = ops.quant8(rnd(1, 30, 64))
    assert ops.gemm8(a, b).shape == (0, 30) and ops.gemm8(b, a).shape == (30, 0)
    saved = ops.empty8(0, 64, halves=True)
    assert ops.swiglu8(x, saved=saved).shape == (0, 32) and ops.swiglu8_bwd(x[:, :32], saved).shape == (0, 64)
    offs = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert ops.gemm8(a, ops.quant8(rnd(2, 2, 30, 64), 128), offs=offs).shape == (0, 30)
    assert ops.quant8(torch.empty(0, 30, 64, device="cuda"), 128).shape == (0, 30, 64)
    assert ops.quant8_t(torch.empty(0, 30, 64, device="cuda")).shape == (0, 64, 30)
    ops.check()


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("n,k", [(72, 130), (1024, 100), (1001, 256)])
def test_gemm_by_expert_adds_to_its_rows(ops, n, k, block_rows):
    """accumulate by expert: rows of the segments grow, all others stay."""
    offs, rows, e = [128, 128, 384, 1024], 1300, 3
    a, b = ops.quant8(rnd(1, rows, k)), ops.quant8(rnd(2, e, n, k, std=0.02), block_rows=block_rows)
    o = torch.tensor(offs, dtype=torch.int32, device="cuda")
    for pad, shift in ((0, 0), (3, 1)):
        out = strided(rnd(3, rows, n), pad, shift)
        before = R.as64(out)
        ops.gemm8(a, b, out=out, offs=o, accumulate=True)
        av, bv = R.value8(a), R.value8(b)
        for i in range(e):
            s = slice(offs[i], offs[i + 1])
            product_close(out[s], av[s], bv[i], torch.float32, k, before[s])
        after = R.as64(out)
        assert np.array_equal(after[:128], before[:128]) and np.array_equal(after[1024:], before[1024:])
    ops.check()


@pytest.mark.parametrize("t", [500, 40000, 90000])
def test_route_of_tensors_ordered_again(ops, t):
    """A Route made of a routing's tensors sorts into them, in a capture too
    (its workspace is then the graph's)."""
    k, e = 2, 6
    a = ops.Route(t, k, e)
    r = ops.Route.of(a.offs, a.perm, a.row)
    idx = torch.from_numpy(choices(1, t, k, e, "dropped")).cuda()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.order(idx)
    for seed in (2, 3):
        new = choices(seed, t, k, e, "dropped")
        idx.copy_(torch.from_numpy(new))
        g.replay()
        for got, want in zip((a.offs, a.perm, a.row), R.order(new, e)):
            assert np.array_equal(got.cpu().numpy(), want)
    ops.check()


def test_failure_found_outside_inference_mode(ops, monkeypatch):
    """Status words made in inference mode can be read and cleared outside it."""
    monkeypatch.setattr(ops, "_status", {})
    with torch.inference_mode():
        r = ops.Route(1, 1, 2)
        idx = torch.full((1, 1), 5, dtype=torch.int32, device="cuda")
    r.order(idx)
    from adamw_persistent_sm_gb300.trainer import StatusError
    with pytest.raises(StatusError, match="out of range"):
        ops.check()
    ops.check()
