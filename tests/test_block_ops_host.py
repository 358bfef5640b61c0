"""The operators around the expert layer without a GPU: the definitions' gradients
against differences, and argument checks of the C ABI and the torch wrappers
(every call here is refused or has nothing to do before anything is enqueued;
the addresses are never dereferenced)."""
import ctypes as C

import numpy as np
import pytest
import torch

import block_ref as R
from adamw_persistent_sm_gb300 import binding as B
from adamw_persistent_sm_gb300 import block_ops as ops

P = 1 << 20
BAD, UNS, OK, SMALL = B.MT_ERR_ARG, B.MT_ERR_UNSUPPORTED, B.MT_OK, B.MT_ERR_ARENA_SMALL
F32, BF16 = B.MT_DT_FP32, B.MT_DT_BF16
NONE, CHANNEL, TOKEN, FULL = B.MT_GATE_NONE, B.MT_GATE_CHANNEL, B.MT_GATE_TOKEN, B.MT_GATE_FULL


@pytest.fixture(scope="module")
def lib():
    return B.load(build_if_missing=True)


# ---------------------------------------------------------------------------
# the definitions
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("gate", [None, "channel", "token", "full"])
@pytest.mark.parametrize("after,before", [(True, True), (False, True), (True, False), (False, False)])
def test_joint_gradients_by_differences(gate, after, before):
    """Central differences of a scalar of h and r in float64: off by the step's
    square (1e-10) and by rounding over the step (1e-16 / 1e-5)."""
    g = np.random.default_rng(1)
    t, d, a, b, eps = 3, 5, 0.7, 1.3, 1e-2
    shape = {None: None, "channel": (1, d), "token": (t, 1), "full": (t, d)}[gate]
    p = dict(x=g.normal(size=(t, d)), y=g.normal(size=(t, d)), after=g.normal(size=(1, d)) if after else None,
             gate=None if gate is None else g.normal(size=shape), before=g.normal(size=(1, d)) if before else None)
    ch, cr = g.normal(size=(t, d)), g.normal(size=(t, d))

    def scalar(q):
        h, r, _, _ = R.joint(q["x"], q["y"], q["after"], q["gate"], q["before"], a, b, eps)
        return (ch * h).sum() + (0.0 if r is None else (cr * r).sum())

    h = R.joint(p["x"], p["y"], p["after"], p["gate"], p["before"], a, b, eps)[0]
    got = R.joint_grad(cr if before else None, ch, h, p["y"], p["after"], p["gate"], p["before"], a, b, eps)
    for name, v in p.items():
        if v is None:
            continue
        want = np.zeros_like(v)
        for i in np.ndindex(v.shape):
            q1, q2 = ({**p, name: v.copy()} for _ in range(2))
            q1[name][i] += 1e-5
            q2[name][i] -= 1e-5
            want[i] = (scalar(q1) - scalar(q2)) / 2e-5
        grad = got["d" + name][0]
        if v.shape != grad.shape:
            grad = grad.sum(0 if v.shape[0] == 1 else 1, keepdims=True)
        assert np.abs(grad - want).max() < 1e-7, name


@pytest.mark.parametrize("renormalize", [True, False])
def test_choose_gradients_by_differences(renormalize):
    g = np.random.default_rng(2)
    t, e, k = 6, 5, 2
    z, c, dl = g.normal(size=(t, e)), g.normal(size=(t, k)), np.array([0.7, 0.3])
    z[1, 3] = -np.inf
    z[4] = -np.inf
    mask = np.array([1, 1, 0, 1, 1, 1], bool)
    idx, _, counts, *_ = R.choose(z, k, mask, renormalize)

    def scalar(v):                               # the choices are constants: no step changes them
        i, w, n, losses, *_ = R.choose(v, k, mask, renormalize)
        assert np.array_equal(i, idx) and np.array_equal(n, counts)
        return (c * w).sum() + (dl * losses).sum()

    got, _ = R.choose_grad(z, idx, counts, c, dl, mask, renormalize)
    for i in np.ndindex(t, e):
        z1, z2 = z.copy(), z.copy()
        z1[i] += 1e-6
        z2[i] -= 1e-6
        want = (scalar(z1) - scalar(z2)) / 2e-6
        assert abs(got[i] - want) < 1e-8, i


def test_choose_of_an_even_load():
    """The balance loss is 1 where every expert is chosen as often and as likely."""
    z = np.zeros((4, 4))
    z[np.arange(4), np.arange(4)] = 3.0
    idx, w, counts, losses, *_ = R.choose(z, 1, None, True)
    assert np.array_equal(idx[:, 0], np.arange(4)) and counts.tolist() == [1, 1, 1, 1, 4]
    assert abs(losses[0] - 1.0) < 1e-12 and np.allclose(w, 1.0)


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
def joint(**kw):
    v = dict(rows=4, width=16, stream_dtype=F32, dtype=F32, after=P, before=P, gate=P, ldgate=0, n_rows=None,
             gate_kind=CHANNEL, res_scale=1.0, out_scale=1.0, eps=1e-5, reserved0=0)
    v.update(kw)
    return B.mt_joint(*[v[k] for k, _ in B.mt_joint._fields_])


def test_struct_layouts_match_the_header():
    assert C.sizeof(B.mt_joint) == 88 and C.sizeof(B.mt_span) == 32


FWD = dict(x=P, ldx=16, y=P, ldy=16, h=P, ldh=16, r=P, ldr=16)
BWD = dict(h=P, ldh=16, y=P, ldy=16, dr=P, lddr=16, dh=P, lddh=16, dx=P, lddx=16, dy=P, lddy=16, dgate=P, lddgate=0,
           dafter=P, dbefore=P, accumulate=0, ws=P, ws_bytes=1 << 30)
BAD_JOINTS = [dict(rows=-1), dict(width=0), dict(stream_dtype=2), dict(dtype=-1), dict(eps=0.0), dict(eps=float("nan")),
              dict(eps=float("inf")), dict(res_scale=float("inf")), dict(out_scale=float("nan")), dict(gate_kind=4),
              dict(gate_kind=-1), dict(gate_kind=NONE), dict(gate=None), dict(after=P + 2), dict(before=P + 1),
              dict(gate=P + 2), dict(n_rows=P + 2), dict(reserved0=1), dict(gate_kind=TOKEN, ldgate=0),
              dict(gate_kind=FULL, ldgate=15)]


@pytest.mark.parametrize("kw", BAD_JOINTS)
def test_joint_refusals(lib, kw):
    assert lib.mt_block_norm(joint(**kw), *FWD.values(), 0) == BAD
    assert lib.mt_block_norm_bwd(joint(**kw), *BWD.values(), 0) == BAD


def test_joint_limits(lib):
    for kw in (dict(width=8193), dict(rows=(1 << 30) + 1), dict(stream_dtype=BF16, dtype=F32)):
        assert lib.mt_block_norm(joint(**kw), *FWD.values(), 0) == UNS
        assert lib.mt_block_norm_bwd(joint(**kw), *BWD.values(), 0) == UNS
    assert lib.mt_block_norm_ws_bytes(4, 8193) == -UNS and lib.mt_block_norm_ws_bytes(-1, 8) == -BAD
    assert lib.mt_block_norm_ws_bytes(0, 8) == 0 and lib.mt_block_norm_ws_bytes(4, 16) == 0 and lib.mt_block_norm_ws_bytes(400, 16) > 0
    assert lib.mt_block_norm(None, *FWD.values(), 0) == BAD
    assert lib.mt_block_norm(joint(rows=0), *FWD.values(), 0) == OK


def test_block_norm_refusals(lib):
    for kw in (dict(x=0), dict(x=P + 2), dict(ldx=15), dict(y=0), dict(y=P + 1), dict(ldy=15), dict(h=0), dict(ldh=15),
               dict(r=0), dict(ldr=15), dict(r=P + 2), dict(h=0, r=0)):
        assert lib.mt_block_norm(joint(), *{**FWD, **kw}.values(), 0) == BAD, kw
    alone = {**FWD, "y": 0, "h": 0}
    plain = dict(after=None, gate=None, gate_kind=NONE)
    for kw in (dict(after=None), dict(gate=None, gate_kind=NONE), {**plain, "res_scale": 0.5}, {**plain, "before": None}):
        assert lib.mt_block_norm(joint(**kw), *alone.values(), 0) == BAD, kw
    assert lib.mt_block_norm(joint(before=None), *FWD.values(), 0) == BAD          # r of nothing


def test_block_norm_bwd_refusals(lib):
    for kw in (dict(h=0), dict(ldh=15), dict(y=0), dict(ldy=15), dict(dr=0), dict(lddr=15), dict(dh=P + 2),
               dict(lddh=15), dict(dx=0), dict(lddx=15), dict(dy=0), dict(lddy=15), dict(dgate=0), dict(dgate=P + 2),
               dict(dafter=0), dict(dafter=P + 2), dict(dbefore=0), dict(accumulate=2)):
        assert lib.mt_block_norm_bwd(joint(), *{**BWD, **kw}.values(), 0) == BAD, kw
    for kw in (dict(ws=0), dict(ws=P + 8)):
        assert lib.mt_block_norm_bwd(joint(rows=400), *{**BWD, **kw}.values(), 0) == BAD, kw
    need = lib.mt_block_norm_ws_bytes(400, 16)
    assert lib.mt_block_norm_bwd(joint(rows=400), *{**BWD, "ws_bytes": need - 1}.values(), 0) == SMALL
    for kw in (dict(gate_kind=TOKEN, ldgate=1), dict(gate_kind=FULL, ldgate=16)):
        assert lib.mt_block_norm_bwd(joint(**kw), *{**BWD, "lddgate": 0}.values(), 0) == BAD
    for kw in (dict(after=None), dict(before=None), dict(gate=None, gate_kind=NONE)):
        assert lib.mt_block_norm_bwd(joint(**kw), *BWD.values(), 0) == BAD
    bare = joint(after=None, before=None, gate=None, gate_kind=NONE)
    none = {**BWD, "dgate": 0, "dafter": 0, "dbefore": 0, "dr": 0, "dh": 0}
    assert lib.mt_block_norm_bwd(bare, *none.values(), 0) == BAD                    # no gradient comes in
    assert lib.mt_block_norm_bwd(joint(rows=0, after=None, before=None, gate=None, gate_kind=NONE), *none.values(), 0) == OK


CH = dict(z=P, dtype=F32, ldz=16, t=4, e=16, k=2, mask=0, renorm=1, idx=P, w=P, counts=P, losses=P, ws=P, ws_bytes=1 << 20)
CB = dict(z=P, dtype=F32, ldz=16, t=4, e=16, k=2, mask=0, renorm=1, idx=P, counts=P, dw=P, dlosses=P, dz=P, lddz=16)


def test_choose_refusals(lib):
    for kw in (dict(z=0), dict(z=P + 2), dict(dtype=2), dict(ldz=15), dict(t=-1), dict(e=0), dict(k=0), dict(renorm=2),
               dict(idx=0), dict(idx=P + 2), dict(w=0), dict(counts=0), dict(losses=0), dict(losses=P + 2), dict(ws=0),
               dict(ws=P + 4)):
        assert lib.mt_choose(*{**CH, **kw}.values(), 0) == BAD, kw
    for kw in (dict(e=65), dict(k=9), dict(e=4, k=5), dict(t=(1 << 30) + 1)):
        assert lib.mt_choose(*{**CH, **kw}.values(), 0) == UNS, kw
        assert lib.mt_choose_bwd(*{**CB, **kw}.values(), 0) == UNS, kw
    need = lib.mt_choose_ws_bytes(4, 2, 16)
    assert lib.mt_choose(*{**CH, "ws_bytes": need - 1}.values(), 0) == SMALL
    assert lib.mt_choose_ws_bytes(-1, 2, 16) == -BAD and lib.mt_choose_ws_bytes(1, 9, 16) == -UNS
    for kw in (dict(z=0), dict(dtype=5), dict(ldz=15), dict(idx=0), dict(dw=P + 2), dict(dlosses=P + 1), dict(counts=0),
               dict(dz=0), dict(lddz=15), dict(dw=0, dlosses=0), dict(renorm=-1)):
        assert lib.mt_choose_bwd(*{**CB, **kw}.values(), 0) == BAD, kw
    assert lib.mt_choose_bwd(*{**CB, "t": 0, "z": 0, "dz": 0, "idx": 0}.values(), 0) == OK


def spans(*kw):
    rows = [dict(dict(grad=P, out=P, numel=8, dtype=F32, reserved0=0), **k) for k in kw]
    return (B.mt_span * max(1, len(rows)))(*[tuple(r[k] for k, _ in B.mt_span._fields_) for r in rows])


def test_clip_refusals(lib):
    big = 1 << 30
    for kw in (dict(grad=0), dict(grad=P + 2), dict(numel=-1), dict(dtype=3), dict(reserved0=1)):
        s = spans({}, kw)
        assert lib.mt_grad_norm(s, 2, 1.0, P, P, big, 0) == BAD, kw
        assert lib.mt_grad_clip(s, 2, 1.0, 0.0, 1.0, P, P, big, 0) == BAD, kw
    assert lib.mt_grad_clip(spans(dict(out=0)), 1, 1.0, 0.0, 1.0, P, P, big, 0) == BAD
    assert lib.mt_grad_clip(spans(dict(out=P + 1)), 1, 1.0, 0.0, 1.0, P, P, big, 0) == BAD
    s = spans({})
    for a in ((s, -1, 1.0, P, P, big), (None, 1, 1.0, P, P, big), (s, 1, float("inf"), P, P, big), (s, 1, 1.0, 0, P, big),
              (s, 1, 1.0, P + 2, P, big), (s, 1, 1.0, P, 0, big), (s, 1, 1.0, P, P + 8, big)):
        assert lib.mt_grad_norm(*a, 0) == BAD
    assert lib.mt_grad_norm(s, 1, 1.0, P, P, lib.mt_grad_ws_bytes(1) - 1, 0) == SMALL
    nan, inf = float("nan"), float("inf")
    for m, e, sc in ((0.0, 0.0, 1.0), (-1.0, 0.0, 1.0), (nan, 0.0, 1.0), (inf, 0.0, 1.0), (1.0, -1e-9, 1.0),
                     (1.0, nan, 1.0), (1.0, inf, 1.0), (1.0, 0.0, nan), (1.0, 0.0, inf)):
        assert lib.mt_grad_clip(s, 1, m, e, sc, P, P, big, 0) == BAD, (m, e, sc)
    assert lib.mt_grad_norm(spans(dict(numel=(1 << 40) + 1)), 1, 1.0, P, P, big, 0) == UNS
    assert lib.mt_grad_norm(spans(*[dict(numel=1 << 40)] * 32), 32, 1.0, P, P, big, 0) == UNS
    assert lib.mt_grad_ws_bytes(-1) == -BAD and lib.mt_grad_ws_bytes(0) > 0


def test_wrappers_refuse_host_tensors():
    x, v, i = torch.zeros(4, 16), torch.ones(16), torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        ops.block_norm(x, x, after=v, before=v)
    with pytest.raises(ValueError):
        ops.block_norm_bwd(x, x, x, x, before=v)
    with pytest.raises(ValueError):
        ops.choose(x, 2)
    with pytest.raises(ValueError):
        ops.choose_bwd(x, i, dw=torch.zeros(4, 2))
    with pytest.raises(ValueError):
        ops.GradSet([x])
    with pytest.raises(ValueError):
        ops.clip_grads([x], 1.0)


@pytest.mark.parametrize("make,dense", [
    (lambda: torch.zeros(3, 4), True), (lambda: torch.zeros(3, 4).t(), True), (lambda: torch.zeros(2, 3, 4).permute(1, 2, 0), True),
    (lambda: torch.zeros(()), True), (lambda: torch.zeros(0, 3), True), (lambda: torch.zeros(3, 4)[:, :2], False),
    (lambda: torch.zeros(1, 4).expand(3, 4), False), (lambda: torch.zeros(6)[::2], False), (lambda: torch.zeros(5, 1, 2)[:, :, :1], False)])
def test_dense(make, dense):
    assert ops._dense(make()) is dense
