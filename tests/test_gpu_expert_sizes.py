"""The expert operators at the sizes where their kernels take other forms
than for a few rows - four rows to a warp, several chunks of columns in
flight, a second tile to a CTA - against the definitions in float64, on the
device (tests/expert_ref.py)."""
import pytest
import torch

import expert_ref as R

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def ops():
    from adamw_persistent_sm_gb300 import expert_ops
    yield expert_ops
    expert_ops.check()


def values(seed, rows, cols, dtype):
    """Rows over many magnitudes; a zero row, and infinities and NaN early, late and at the edges."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, cols, device="cuda", generator=g)
    x *= torch.pow(2.0, torch.randint(-30, 30, (rows, 1), device="cuda", generator=g).float())
    x[rows // 3] = 0
    x[1, 2], x[rows - 1, cols - 1], x[rows - 2, 0] = float("inf"), float("nan"), float("-inf")
    x[rows // 2, cols // 2:] = float("nan")
    return x.to(dtype)


def strided(t, pad, shift):
    buf = torch.full((t.shape[0], t.shape[1] + pad + shift), float("nan"), dtype=t.dtype, device=t.device)
    v = buf[:, shift:shift + t.shape[1]]
    v.copy_(t)
    return v


LAYOUTS = [(0, 0), (8, 0), (3, 1)]         # rows on 16-byte boundaries, apart, off them


def stained(ops, rows, cols, **kw):
    t = ops.empty8(rows, cols, **kw)
    t.codes.fill_(0x55)
    t.scales.fill_(0x33)
    return t


def same(t, want, rows=None):
    """t's codes and scale bytes up to a row (a whole number of blocks of rows) are the definition's."""
    codes, scales = want
    n = t.rows if rows is None else rows
    nb = -(-n // t.block_rows)
    assert torch.equal(t.codes[:n, :t.cols], codes[:n]) and torch.equal(t.scales[:nb], scales[:nb])
    assert (t.codes[n:] == 0x55).all() and (t.scales[nb:] == 0x33).all()


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("pad,shift", LAYOUTS)
@pytest.mark.parametrize("rows,cols", [(2500, 1100), (2501, 768), (10001, 130)])
def test_quant_rows(ops, rows, cols, pad, shift, dt):
    x = strided(values(1, rows, cols, DT[dt]), pad, shift)
    for halves in (False, True):
        want = R.quant_t(x.double(), halves=halves)
        t = stained(ops, rows, cols, halves=halves)
        same(ops.quant8(x, out=t), want)
        for limit in (2311, 2432, rows - 1):          # inside a warp's four rows, behind them
            t = stained(ops, rows, cols, halves=halves)
            ops.quant8(x, out=t, n_rows=torch.tensor([limit], dtype=torch.int32, device="cuda"))
            same(t, want, limit)
        val = R.value_t(*want, cols, halves=halves)
        full = ops.quant8(x, halves=halves)
        assert torch.equal(ops.dequant8(full, torch.float32).double().nan_to_num(7e77), val.nan_to_num(7e77))
        assert torch.equal(ops.dequant8(full).nan_to_num(7e30), val.float().bfloat16().nan_to_num(7e30))


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("pad,shift", LAYOUTS)
@pytest.mark.parametrize("rows,cols", [(2500, 3100), (2561, 2688), (130, 64000)])
def test_quant_tiles(ops, rows, cols, pad, shift, dt):
    """Straight and transposed, 1 x 128 and 128 x 128, from values and from codes."""
    x = strided(values(2, rows, cols, DT[dt]), pad, shift)
    x64 = x.double()
    same(ops.quant8(x, 128), R.quant_t(x64, 128))
    xt = x64.T.contiguous()
    want = R.quant_t(xt)
    same(ops.quant8_t(x), want)
    same(ops.quant8_t(x, 128), R.quant_t(xt, 128))
    held = ops.quant8(x)
    vt = R.value_t(held.codes, held.scales, cols).T.contiguous()
    want8 = R.quant_t(vt)
    same(ops.quant8_t(held), want8)
    same(ops.quant8_t(held, 128), R.quant_t(vt, 128))
    limit = (rows - 1) // 256 * 128
    n = torch.tensor([limit], dtype=torch.int32, device="cuda")
    for src, (codes, scales) in ((x, want), (held, want8)):
        t = ops.quant8_t(src, out=stained(ops, cols, rows), n_rows=n)
        nb = limit // 128
        assert torch.equal(t.codes[:, :limit], codes[:, :limit]) and (t.codes[:, limit:] == 0x55).all()
        assert torch.equal(t.scales[:, :nb], scales[:, :nb]) and (t.scales[:, nb:] == 0x33).all()


@pytest.mark.parametrize("batch,rows,cols", [(3, 1500, 1400), (40, 300, 520)])
def test_quant_tile_stacks(ops, batch, rows, cols):
    """Stacks as a layer's weights are held: every matrix with tiles of its own."""
    x = torch.stack([values(3 + i, rows, cols, torch.float32) for i in range(batch)])
    for v in (x, x.bfloat16()):
        a, b, c = ops.quant8(v, 128), ops.quant8_t(v, 128), ops.quant8_t(v)
        for i in range(batch):
            x64, xt = v[i].double(), v[i].double().T.contiguous()
            same(a[i], R.quant_t(x64, 128))
            same(b[i], R.quant_t(xt, 128))
            same(c[i], R.quant_t(xt))


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("pad,shift", LAYOUTS)
@pytest.mark.parametrize("t,k,width", [(3000, 2, 768), (3001, 3, 1100), (1500, 8, 2050)])
def test_dispatch8(ops, t, k, width, pad, shift, dt):
    e = 9
    g = torch.Generator(device="cuda").manual_seed(t)
    idx = torch.rand(t, e, generator=g, device="cuda").topk(k, 1).indices.to(torch.int32).contiguous()
    idx[torch.rand(t, generator=g, device="cuda") < 0.2] = -1
    r = ops.Route(t, k, e).order(idx)
    x = strided(values(5, t, width, DT[dt]), pad, shift)
    out = r.dispatch8(x, out=stained(ops, r.rows, width))
    end = int(r.offs[-1])
    live = (r.perm >= 0)[:, None]
    xs = torch.where(live, x.double()[(r.perm.clamp(min=0) // k).long()], 0.0)
    same(out, R.quant_t(xs), end)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("pad,shift", [(0, 0), (3, 1)])
@pytest.mark.parametrize("rows,width", [(2500, 512), (2501, 1100), (9001, 264)])
def test_swiglu(ops, rows, width, pad, shift, dt):
    """Two rows to a warp.  The results lie within half a step of the exact
    ones plus (|g| + 8) 2^-22 relative for the fp32 silu(g) u, and no scale is
    larger than its block needs; the checkpoints' codes are exact."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    gu = torch.randn(rows, 2 * width, device="cuda", generator=g)
    gu *= torch.pow(2.0, torch.randint(-20, 4, (rows, 1), device="cuda", generator=g).float())
    gu = strided(gu.to(DT[dt]), pad, shift)
    for limit in (rows, 2311):
        act, saved = stained(ops, rows, width), stained(ops, rows, 2 * width, halves=True)
        ops.swiglu8(gu, act=act, saved=saved, n_rows=torch.tensor([limit], dtype=torch.int32, device="cuda"))
        same(saved, R.quant_t(gu.double(), halves=True), limit)
        assert (act.codes[limit:] == 0x55).all() and (act.scales[limit:] == 0x33).all()
        gg, u = gu[:limit].double().split(width, 1)
        exact = gg / (1 + torch.exp(-gg)) * u
        err = (gg.abs() + 8) * 2.0 ** -22 * exact.abs() + 1e-37 * (1 + u.abs())
        val = R.value_t(act.codes[:limit], act.scales[:limit], width)
        blk = torch.arange(width, device="cuda") // 128
        s = R.power_t(act.scales[:limit].long() - 127)
        step = torch.maximum(2.0 ** -4 * exact.abs(), 2.0 ** -10 * s[:, blk])
        assert ((val - exact).abs() <= step * (1 + 2.0 ** -4) + err).all()
        for c in range(0, width, 128):
            top, slack, sc = exact[:, c:c + 128].abs().amax(1), err[:, c:c + 128].amax(1), s[:, c // 128]
            assert (top - slack <= 448 * sc).all() and ((top + slack > 224 * sc) | (sc == 2.0 ** -126)).all()
        only = ops.swiglu8(gu)
        assert torch.equal(only.codes[:limit, :width], act.codes[:limit, :width])
        assert torch.equal(only.scales[:limit], act.scales[:limit])


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("m,n", [(100, 64), (700, 700), (2600, 4100)])
def test_long_products_are_their_parts_added_in_order(ops, m, n, block_rows):
    """A reduction of 32,768 and more is the fp32 sum, in order, of the products
    of its parts of 4,096 bit for bit: tensor memory, whose additions cut off,
    sums no more than a part."""
    k, part = 32768 + 500, 4096
    g = torch.Generator(device="cuda").manual_seed(m)
    a = ops.quant8(torch.rand(m, k, device="cuda", generator=g))
    b = ops.quant8(torch.rand(n, k, device="cuda", generator=g), block_rows)
    want = None
    for lo in range(0, k, part):
        hi = min(lo + part, k)
        ld = -(-(hi - lo) // 16) * 16
        cut = [ops.Tensor8(t.codes[:, lo:lo + ld].contiguous(), t.scales[:, lo // 128:-(-hi // 128)].contiguous(), hi - lo,
                           t.block_rows) for t in (a, b)]
        c = ops.gemm8(*cut, dtype=torch.float32)
        want = c if want is None else want + c
    assert torch.equal(ops.gemm8(a, b, dtype=torch.float32), want)
    # the weight gradients' form of the same sums, where b has a scale per row
    if block_rows == 1:
        offs = torch.tensor([0, -(-k // 128) * 128], dtype=torch.int32, device="cuda")
        assert torch.equal(ops.gemm8_reduce(a, b, offs)[0], want)


def test_offsets_past_32_bits(ops):
    """Matrices of more than 2^31 elements: rows behind that point are as exact as those before."""
    rows, cols = 70_001, 32_768
    dt, n = torch.bfloat16, 300
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(rows, cols, dtype=dt, device="cuda")
    x[:n], x[-n:] = (torch.randn(n, cols, device="cuda", generator=g).to(dt) for _ in range(2))
    x[n:-n] = 1.0
    t = ops.quant8(x)
    for s in (slice(0, n), slice(rows - n, rows)):
        codes, scales = R.quant_t(x[s].double())
        assert torch.equal(t.codes[s], codes) and torch.equal(t.scales[s], scales)
    back = ops.dequant8(t, dt)
    assert (back[n:-n] == 1).all()
    val = R.value_t(t.codes[-n:], t.scales[-n:], cols)
    assert torch.equal(back[-n:].double(), val.to(dt).double())
    # a product that reads the codes and writes rows behind that point
    w = ops.quant8(torch.randn(40, cols, device="cuda", generator=g), 128)
    c = ops.gemm8(t, w, dtype=torch.float32)
    ref = val @ R.value_t(w.codes, w.scales, cols, 128).T
    mag = val.abs() @ R.value_t(w.codes, w.scales, cols, 128).abs().T
    assert ((c[-n:].double() - ref).abs() <= (cols + 2) * 2 * U32 * mag).all()
    del c
    # SwiGLU and its backward on the same rows
    saved, act = ops.empty8(rows, cols, halves=True), ops.empty8(rows, cols // 2)
    ops.swiglu8(x, act=act, saved=saved)
    assert torch.equal(saved.codes[-n:], t.codes[-n:]) and torch.equal(saved.scales[-n:], t.scales[-n:])
    few = ops.swiglu8(x[-n:].contiguous())
    assert torch.equal(act.codes[-n:], few.codes) and torch.equal(act.scales[-n:], few.scales)
    ops.swiglu8_bwd(x[:, :cols // 2], saved, dgu=back)
    few = ops.swiglu8_bwd(x[-n:, :cols // 2], saved.part(rows - n, rows))
    assert torch.equal(back[-n:], few)
    del saved, act, few
    # the transpose: codes of a column lie in one row of 70,016 bytes
    tt = ops.quant8_t(x)
    end = rows // 128 * 128
    codes, scales = R.quant_t(x[end - 128:].double().T.contiguous())
    assert torch.equal(tt.codes[:, end - 128:rows], codes) and torch.equal(tt.scales[:, -2:], scales)
    del tt, t
    # rows to their experts and back
    r = ops.Route(rows - 200, 1, 1).order(torch.zeros(rows - 200, 1, dtype=torch.int32, device="cuda"))
    xs = torch.empty(r.rows, cols, dtype=dt, device="cuda")
    r.dispatch(x[200:], out=xs)
    assert torch.equal(xs[rows - 200 - n:rows - 200], x[-n:])
    out = r.combine(xs)
    assert torch.equal(out, x[200:])
    d8 = r.dispatch8(x[200:])
    codes, scales = R.quant_t(x[-n:].double())
    assert torch.equal(d8.codes[rows - 200 - n:rows - 200], codes) and torch.equal(d8.scales[rows - 200 - n:rows - 200], scales)
