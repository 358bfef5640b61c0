"""The expert layer on the 8-bit operators: every step of a forward and a
backward pass against float64 on the device's own operands (so that each
bound is one step's), the trainer's path to it, and its agreement with the
update kernel's router."""
import numpy as np
import pytest
import torch

import expert_ref as R
import moe_inputs as mi

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
STEP = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}


def rnd(seed, *shape, std=1.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def near(got, want, bound):
    got = R.as64(got)
    assert np.isfinite(got).all()
    bad = np.abs(got - want) > bound
    assert not bad.any(), (int(bad.sum()), float(np.abs(got - want).max()))


def product(got, a, b, dtype, before=0.0):
    """Half a step of the output and one step (2 U32) per addition of the sum of magnitudes."""
    ref = a @ b.T + before
    near(got, ref, (a.shape[1] + 2) * 2 * U32 * (np.abs(a) @ np.abs(b).T + np.abs(before)) + STEP[dtype] * 1.001 * np.abs(ref))


def held(x, **kw):
    """What x holds after quantisation."""
    q, s = R.quant(x, **kw)
    return R.value(q, s, x.shape[1], **{k: v for k, v in kw.items()})


def routing(t, k, e, seed):
    g = np.random.default_rng(seed)
    idx = np.stack([g.permutation(e)[:k] for _ in range(t)]).astype(np.int32)
    idx[g.random(t) < 0.2] = -1
    idx[0, :] = e - 1                       # the same expert in every slot
    return idx


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("t,k,e,d,f", [(1, 2, 4, 64, 48), (150, 2, 5, 256, 136), (700, 3, 4, 128, 64), (90, 1, 1, 100, 20)])
def test_layer_step_by_step(t, k, e, d, f, dt):
    from adamw_persistent_sm_gb300 import expert_ops as ops
    from adamw_persistent_sm_gb300 import ExpertLayer8
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    wg, wu, wd = rnd(1, e, f, d, std=0.05), rnd(2, e, f, d, std=0.05), rnd(3, e, d, f, std=0.05)
    layer = ExpertLayer8(wg, wu, wd, t, k, dtype)
    idx = routing(t, k, e, 4)
    x, dout, w = rnd(5, t, d, dtype=dtype), rnd(6, t, d, dtype=dtype), torch.softmax(rnd(7, t, k), 1)
    out = layer.forward(x, torch.from_numpy(idx).cuda(), w)
    offs, perm, row = R.order(idx, e)
    end, live = offs[-1], perm >= 0
    segs = [slice(offs[i], offs[i + 1]) for i in range(e)]
    x64, d64, w64 = R.as64(x), R.as64(dout), R.as64(w)

    # the weights' blocks, in both orientations
    wgu = np.concatenate([R.as64(wg), R.as64(wu)], 1)
    for i in range(e):
        v = held(wgu[i], block_rows=128)
        assert np.array_equal(R.value8(layer.w_gu)[i], v)
        assert np.array_equal(R.value8(layer.w_gu_t)[i], held(wgu[i].T.copy(), block_rows=128))
        assert np.array_equal(R.value8(layer.w_down_t)[i], held(R.as64(wd)[i].T.copy(), block_rows=128))

    xs = np.zeros((perm.size, d))
    xs[live] = x64[perm[live] // k]
    xv = held(xs[:end]) if end else xs[:0]
    assert np.array_equal(R.value8(layer.xs8)[:end], xv)
    gu, av, y = R.as64(layer.gu), R.value8(layer.act8), R.as64(layer.y)
    for i, s in enumerate(segs):
        product(layer.gu[s], xv[s], R.value8(layer.w_gu)[i], dtype)
        product(layer.y[s], av[s], R.value8(layer.w_down)[i], dtype)
    if end:
        assert np.array_equal(R.value8(layer.saved)[:end], held(gu[:end], halves=True))
    term = np.where((row >= 0)[:, :, None], np.where(live[:, None], y, 0.0)[np.maximum(row, 0)] * w64[:, :, None], 0.0)
    near(out, term.sum(1), (k + 1) * U32 * np.abs(term).sum(1) + STEP[dtype] * 1.001 * np.abs(term.sum(1)))

    grads = tuple(rnd(8 + i, *s, std=0.1) for i, s in enumerate(((e, f, d), (e, f, d), (e, d, f))))
    before = [R.as64(g).copy() for g in grads]
    dx, dw, got = layer.backward(dout, grads, accumulate=True)
    assert all(a is b for a, b in zip(got, grads))
    b = layer._bwd
    dy = R.as64(b["dy"])
    ref = np.zeros((perm.size, d))
    ref[live] = d64[perm[live] // k] * w64.reshape(-1)[perm[live]][:, None]
    near(b["dy"][:end], ref[:end], (U32 + STEP[dtype] * 1.001) * np.abs(ref[:end]))
    prod = np.where((row >= 0)[:, :, None], d64[:, None, :] * np.where(live[:, None], y, 0.0)[np.maximum(row, 0)], 0.0)
    near(dw, prod.sum(-1), (d + 1) * U32 * np.abs(prod).sum(-1))
    if end == 0:
        return
    dyv, dguv = held(dy[:end]), held(R.as64(b["dgu"])[:end])
    sv = R.value8(layer.saved)[:end]
    g, u = sv[:, :f], sv[:, f:]
    s_, da = R.sigmoid(g), R.as64(b["dact"])[:end]
    tiny, rel = 1e-37, (np.abs(g) + 8) * 2.0 ** -22
    half = STEP[dtype] * 1.01
    for out_, ref, mag in ((b["dgu"][:end, :f], da * u * s_ * (1 + g * (1 - s_)), np.abs(da * u) * (s_ + np.abs(g) * s_)),
                           (b["dgu"][:end, f:], da * g * s_, np.abs(da * g * s_)), (b["act"][:end], g * s_ * u, np.abs(g * s_ * u))):
        near(out_, ref, rel * mag + half * np.abs(ref) + tiny)
    dyt, actt = held(dy[:end].T.copy()), held(R.as64(b["act"])[:end].T.copy())
    dgut, xst = held(R.as64(b["dgu"])[:end].T.copy()), held(xv.T.copy())
    for i, s in enumerate(segs):
        product(b["dact"][s], dyv[s], R.value8(layer.w_down_t)[i], dtype)
        product(b["dxs"][s], dguv[s], R.value8(layer.w_gu_t)[i], dtype)
        product(grads[0][i], dgut[:f, s], xst[:, s], torch.float32, before[0][i])
        product(grads[1][i], dgut[f:, s], xst[:, s], torch.float32, before[1][i])
        product(grads[2][i], dyt[:, s], actt[:, s], torch.float32, before[2][i])
    dxs = np.where(live[:, None], R.as64(b["dxs"]), 0.0)
    term = np.where((row >= 0)[:, :, None], dxs[np.maximum(row, 0)], 0.0)
    near(dx, term.sum(1), (k + 1) * U32 * np.abs(term).sum(1) + STEP[dtype] * 1.001 * np.abs(term.sum(1)))
    ops.check()


def test_layer_gradients_point_the_right_way():
    """The whole layer's gradient against float64 autograd of the unquantised
    layer: 8-bit operands are off by up to 2^-4 each, two at a time over three
    products in a row; random errors of a third of that stay below a fifth of
    the gradient's norm (a wrong sign, factor or transposition does not)."""
    from adamw_persistent_sm_gb300 import ExpertLayer8
    t, k, e, d, f = 500, 2, 4, 256, 128
    wg, wu, wd = rnd(1, e, f, d, std=0.05), rnd(2, e, f, d, std=0.05), rnd(3, e, d, f, std=0.05)
    idx = torch.from_numpy(routing(t, k, e, 4)).cuda()
    x, dout, w = rnd(5, t, d), rnd(6, t, d), torch.softmax(rnd(7, t, k), 1)
    layer = ExpertLayer8(wg, wu, wd, t, k, torch.float32)
    out = layer.forward(x, idx, w)
    dx, dw, grads = layer.backward(dout)
    p = [v.double().requires_grad_() for v in (x, w, wg, wu, wd)]
    ref = torch.zeros(t, d, dtype=torch.float64, device="cuda")
    for i in range(k):
        for j in range(e):
            at = torch.nonzero(idx[:, i] == j)[:, 0]
            h = p[0][at]
            act = torch.nn.functional.silu(h @ p[2][j].T) * (h @ p[3][j].T)
            ref = ref.index_add(0, at, p[1][at, i:i + 1] * (act @ p[4][j].T))
    ref.backward(dout.double())
    for got, want in [(out, ref)] + list(zip((dx, dw, *grads), (v.grad for v in p))):
        rel = float((got.double() - want).norm() / want.norm())
        assert rel < 0.2, rel


def test_trainer_layer_and_router_order():
    """MoETrainer.expert_layer8 on the update's own routing: the stand-alone
    order is the update's, its rows are the update's expert inputs in 8 bits,
    and the gradient views are the trainer's."""
    from adamw_persistent_sm_gb300 import binding as B
    from adamw_persistent_sm_gb300 import expert_ops as ops
    from adamw_persistent_sm_gb300.trainer import MoETrainer
    cfg = mi.get_config("tiny")
    tr = MoETrainer(cfg, "cuda:0")
    tr.load_params(mi.make_params(cfg))
    toks = torch.as_tensor(mi.make_update_tokens(cfg)[0]).cuda()
    tr.micro_step(toks, flags=B.MT_FLAG_NO_OPTIMIZER)
    assert tr.outputs().status == B.MT_OK
    T, K, E, d = cfg.tokens_per_micro, cfg.top_k, cfg.n_experts, cfg.d_model
    idx = tr.debug_view(B.MT_VIEW_TOPK_IDX, 1, torch.int32).view(T, K).clone()
    w = tr.debug_view(B.MT_VIEW_TOPK_W, 1).view(T, K).clone()
    layer = tr.expert_layer8(1)
    x = tr.debug_view(B.MT_VIEW_R2, 1).view(T, d).clone()
    out = layer.forward(x, idx, w)
    r = layer.route
    assert torch.equal(r.offs, tr.debug_view(B.MT_VIEW_ROUTE_OFFS, 1, torch.int32))
    end = int(r.offs[-1])
    assert torch.equal(r.perm[:end], tr.debug_view(B.MT_VIEW_ROUTE_PERM, 1, torch.int32)[:end])
    xs = tr.debug_view(B.MT_VIEW_EXPERT_IN, 1).view(-1, d)[:end]
    assert np.array_equal(R.value8(layer.xs8)[:end], R.value8(ops.quant8(xs.contiguous())))
    assert out.shape == (T, d) and torch.isfinite(out).all()
    grads = tr.expert_grads(1)
    layer.backward(torch.ones(T, d, device="cuda"), grads)
    assert grads[0].data_ptr() == tr.view(tr.grads, "w_gate")[1].data_ptr() and grads[0].abs().sum() > 0
    with pytest.raises(RuntimeError):
        layer.forward(x, idx, w, save=False)
        layer.backward(torch.ones(T, d, device="cuda"), grads)
    ops.check()


def test_layer_captured_while_an_eager_result_lives():
    """Forward and backward captured into one graph and replayed give the eager
    gradients bit for bit, with the eager pass's results still held."""
    from adamw_persistent_sm_gb300 import ExpertLayer8
    t, k, e, d, f = 300, 2, 4, 128, 64
    wg, wu, wd = rnd(1, e, f, d, std=0.05), rnd(2, e, f, d, std=0.05), rnd(3, e, d, f, std=0.05)
    idx = torch.from_numpy(routing(t, k, e, 4)).cuda()
    x, dout, w = rnd(5, t, d, dtype=torch.bfloat16), rnd(6, t, d, dtype=torch.bfloat16), torch.softmax(rnd(7, t, k), 1)
    eager = ExpertLayer8(wg, wu, wd, t, k)
    out = eager.forward(x, idx, w)
    dx, dw, grads = eager.backward(dout)
    layer = ExpertLayer8(wg, wu, wd, t, k)
    layer.forward(x, idx, w)
    layer.backward(dout)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o2 = layer.forward(x, idx, w)
        dx2, dw2, gr2 = layer.backward(dout)
    for _ in range(3):
        for v in (o2, dx2, dw2, *gr2):
            v.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip((o2, dx2, dw2, *gr2), (out, dx, dw, *grads)):
            assert torch.equal(a, b)


def test_failed_forward_leaves_nothing_to_go_back_through():
    """A forward that is refused halfway has changed the buffers of the one
    before: backward asks for a new one.  (A layer of no
    tokens runs too.)"""
    from adamw_persistent_sm_gb300 import ExpertLayer8
    t, k, e, d, f = 20, 2, 4, 64, 48
    wg, wu, wd = rnd(1, e, f, d, std=0.05), rnd(2, e, f, d, std=0.05), rnd(3, e, d, f, std=0.05)
    layer = ExpertLayer8(wg, wu, wd, t, k, torch.float32)
    idx, w = torch.from_numpy(routing(t, k, e, 4)).cuda(), torch.softmax(rnd(7, t, k), 1)
    x = rnd(5, t, d)
    want = layer.forward(x, idx, w).clone()
    for bad in (lambda: layer.forward(x[:, :32], idx, w), lambda: layer.forward(x, idx, w.bfloat16())):
        layer.forward(x, idx, w)
        with pytest.raises(ValueError):
            bad()
        with pytest.raises(RuntimeError):
            layer.backward(x)
    assert torch.equal(layer.forward(x, idx, w), want)
    layer.backward(x)
    none = ExpertLayer8(wg, wu, wd, 0, k, torch.float32)
    assert none.forward(x[:0], idx[:0], w[:0]).shape == (0, d)
    dx, dw, grads = none.backward(x[:0])
    assert dx.shape == (0, d) and all((g == 0).all() for g in grads)


def small_layer(dtype=torch.float32, t=60, k=2, e=4, d=64, f=48):
    from adamw_persistent_sm_gb300 import ExpertLayer8
    weights = rnd(1, e, f, d, std=0.05), rnd(2, e, f, d, std=0.05), rnd(3, e, d, f, std=0.05)
    layer = ExpertLayer8(*weights, t, k, dtype)
    idx, w = torch.from_numpy(routing(t, k, e, 4)).cuda(), torch.softmax(rnd(7, t, k), 1)
    return layer, weights, rnd(5, t, d, dtype=dtype), idx, w, rnd(6, t, d, dtype=dtype)

@pytest.mark.parametrize("captured", [False, True])
def test_weights_rewritten_between_the_passes(captured):
    """backward goes through the routing weights that forward applied, also
    where the caller has put the next microbatch's into the same tensor."""
    layer, _, x, idx, w, dout = small_layer(torch.bfloat16)
    layer.forward(x, idx, w)
    dx, dw, grads = layer.backward(dout)
    layer.forward(x, idx, w.clone().requires_grad_())
    assert not layer.w.requires_grad and torch.equal(layer.w, w)       # and no history grows with the passes
    layer.forward(x, idx, w)
    if captured:
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            layer.forward(x, idx, w)
        g.replay()
    w.fill_(float("nan"))
    dx2, dw2, grads2 = layer.backward(dout)
    assert torch.equal(dw, dw2)
    assert torch.equal(dx, dx2) and all(torch.equal(a, b) for a, b in zip(grads, grads2))


def test_refused_refresh_leaves_the_weights_alone():
    """Weights of other shapes, types or devices are refused before any is
    quantised - also a gate and an up projection whose rows add up to the same
    number - and the layer goes on with those it has."""
    layer, (wg, wu, wd), x, idx, w, _ = small_layer()
    want = layer.forward(x, idx, w).clone()
    more, less = torch.cat([wg, wg[:, :1]], 1) * 2, wu[:, 1:] * 2
    for bad in ((more, less, wd), (wg * 2, wu * 2, wd[:, :, :-1]), (wg * 2, wu * 2, wd.double()), (wg * 2, wu.half(), wd),
                (wg * 2, wu * 2, wd.cpu()), (wg.cpu(), wu.cpu(), wd), (wg * 2, wu * 2, wd.transpose(1, 2)),
                (wg * 2, wu * 2, wd[:2]), (wg[0], wu[0], wd[0])):
        with pytest.raises((ValueError, TypeError)):
            layer.refresh(*bad)
        assert torch.equal(layer.forward(x, idx, w), want)
    both = torch.cat([wg, wu], 1)          # two views of one tensor are as good as two tensors
    layer.refresh(both[:, :48], both[:, 48:], wd)
    assert torch.equal(layer.forward(x, idx, w), want)
    layer.refresh(wg * 2, wu * 2, wd.bfloat16())
    assert not torch.equal(layer.forward(x, idx, w), want)
    layer.refresh(wg, wu, wd)
    assert torch.equal(layer.forward(x, idx, w), want)

def test_refused_backward_leaves_gradients_alone():
    """Gradient buffers are looked at before any of them grows: a refused
    backward may be called again without counting anything twice."""
    layer, _, x, idx, w, dout = small_layer()
    layer.forward(x, idx, w)
    e, f, d = layer.n_experts, layer.width, layer.d
    make = lambda: [rnd(8 + i, *s) for i, s in enumerate(((e, f, d), (e, f, d), (e, d, f)))]  # noqa: E731
    want = layer.backward(dout, tuple(make()), accumulate=True)[2]
    for i in range(3):
        for spoil in (lambda g: g[:, :-1], lambda g: g.double(), lambda g: g.cpu(), lambda g: g.transpose(1, 2),
                      lambda g: g[0], lambda g: g.bfloat16()):
            grads = make()
            before = [g.clone() for g in grads]
            grads[i] = spoil(grads[i])
            with pytest.raises((ValueError, TypeError)):
                layer.backward(dout, tuple(grads), accumulate=True)
            assert all(j == i or torch.equal(g, b) for j, (g, b) in enumerate(zip(grads, before)))
    grads = make()
    before = [g.clone() for g in grads]
    for bad in (lambda: layer.backward(dout, tuple(grads[:2]), accumulate=True),
                lambda: layer.backward(dout[:-1], tuple(grads), accumulate=True),
                lambda: layer.backward(dout.bfloat16(), tuple(grads), accumulate=True)):
        with pytest.raises((ValueError, TypeError)):
            bad()
        assert all(torch.equal(g, b) for g, b in zip(grads, before))
    got = layer.backward(dout, tuple(grads), accumulate=True)[2]
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_weights_refreshed_between_the_passes():
    """A backward would go through other weights than its forward did: it asks
    for a new forward.  A refused refresh changes nothing and asks for none."""
    layer, weights, x, idx, w, dout = small_layer()
    layer.forward(x, idx, w)
    want = layer.backward(dout)[0]
    layer.forward(x, idx, w)
    with pytest.raises(ValueError):
        layer.refresh(weights[0][:1], *weights[1:])
    assert torch.equal(layer.backward(dout)[0], want)
    layer.refresh(*(v * 2 for v in weights))
    with pytest.raises(RuntimeError):
        layer.backward(dout)
    layer.refresh(*weights)
    layer.forward(x, idx, w)
    assert torch.equal(layer.backward(dout)[0], want)


def test_layer_made_in_inference_mode_trains_outside_it():
    layer, _, x, idx, w, dout = small_layer()
    layer.forward(x, idx, w)
    want = layer.backward(dout)[0]
    with torch.inference_mode():
        other = small_layer()[0]
        assert torch.equal(other.forward(x, idx, w), layer.forward(x, idx, w))
    other.forward(x, idx, w)
    assert torch.equal(other.backward(dout)[0], want)


def test_captured_forward_replayed_after_a_refresh():
    """A replay is a new forward that the layer does not see: a refresh before
    it does not keep the backward behind it from running."""
    layer, weights, x, idx, w, dout = small_layer()
    layer.forward(x, idx, w)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = layer.forward(x, idx, w)
    other = small_layer()[0]
    for scale in (1.0, 2.0, 3.0):
        new = [v * scale for v in weights]
        layer.refresh(*new)
        g.replay()
        other.refresh(*new)
        assert torch.equal(out, other.forward(x, idx, w))
        dx, dw, grads = layer.backward(dout)
        dx2, dw2, grads2 = other.backward(dout)
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and all(torch.equal(a, b) for a, b in zip(grads, grads2))
