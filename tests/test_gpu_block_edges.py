"""The operators around the expert layer in calls that their definitions allow and
that are easily answered wrongly: gradients that are not finite beside tokens and
experts that take no part, groups of gradients with norms of their own, numbers at
the ends of the range, and arguments of neighbouring types."""
import numpy as np
import pytest
import torch

import moe_inputs as mi

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def ops():
    from adamw_persistent_sm_gb300 import block_ops
    return block_ops


def rnd(seed, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


# ---------------------------------------------------------------------------
# the logits' gradient
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t,e,k", [(1, 4, 1), (40, 7, 3), (50, 16, 2), (64, 33, 4), (70, 64, 8), (3000, 16, 2)])
@pytest.mark.parametrize("dl", [(INF, 0.0), (0.0, NAN), (-INF, INF), (NAN, 1.0)])
def test_losses_gradients_that_are_not_finite(ops, t, e, k, dl, dtype):
    """Tokens that take no part and logits of -inf get zeros whatever reaches the
    losses; every other logit shows it."""
    z = rnd(t + e, t, e, dtype=dtype)
    z[:, 1::3] = -INF
    z[1::7] = -INF
    mask = torch.ones(t, dtype=torch.bool, device="cuda")
    mask[2::4] = False
    dlosses, dw = torch.tensor(dl, device="cuda"), rnd(1, t, k)
    for renormalize in (True, False):
        for m in (None, mask):
            c = ops.choose(z, k, m, renormalize)
            part = z > -INF if m is None else (z > -INF) & m[:, None]
            for d in (dw, None):
                got = ops.choose_bwd(z, c.idx, c.counts, d, dlosses, m, renormalize)
                assert (got[~part] == 0).all()
                assert not got[part].isfinite().any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("e", [5, 8, 12, 13, 16, 24, 30, 48, 61, 64])
def test_weights_gradients_that_belong_to_nothing(ops, e, dtype):
    """Gradients at indices that name no open expert of a token that takes part -
    none, beyond the experts (whose lanes may hold more places than there are
    experts), closed, or of a token masked out - add nothing, NaN and infinities too."""
    t, k = 9, 4
    z = rnd(e, t, e, dtype=dtype)
    z[3:6, e - 1] = -INF
    mask = torch.tensor([1, 1, 1, 1, 1, 1, 1, 0, 0], dtype=torch.bool, device="cuda")
    idx = torch.zeros(t, k, dtype=torch.int32, device="cuda")
    idx[:, 1] = torch.tensor([e, e + 1, e + 2, -1, e + 3, -7, 1 << 30, 0, e], dtype=torch.int32)
    idx[:, 2] = e - 1
    idx[:, 3] = e + 5
    dw = rnd(2, t, k)
    nothing = (idx < 0) | (idx >= e) | ~mask[:, None]
    nothing |= ~nothing & (z.float().gather(1, idx.clamp(0, e - 1).long()) == -INF)
    assert nothing[:, 1].all() and nothing[:, 3].all()
    clean, none = torch.where(nothing, 0.0, dw), torch.where(nothing, -1, idx)
    for renormalize in (True, False):
        want = ops.choose_bwd(z, none, dw=clean, mask=mask, renormalize=renormalize)
        assert want.isfinite().all()
        for v in (1.0, INF, -INF, NAN):
            got = ops.choose_bwd(z, idx, dw=torch.where(nothing, v, dw), mask=mask, renormalize=renormalize)
            assert torch.equal(got, want)


# ---------------------------------------------------------------------------
# the trainer's gradients in two groups
# ---------------------------------------------------------------------------
def test_trainer_clips_selective_updates_in_two_groups():
    """Launches with MT_FLAG_SELECTIVE_EXPERTS: the shared tensors and the mean of
    the experts' gradients have norms and coefficients of their own, those that
    the update reports (as 1e-5 holds for one group)."""
    from adamw_persistent_sm_gb300 import binding as B
    from adamw_persistent_sm_gb300.trainer import MoETrainer
    sel, stay = B.MT_FLAG_SELECTIVE_EXPERTS, B.MT_FLAG_SELECTIVE_EXPERTS | B.MT_FLAG_NO_OPTIMIZER
    experts = ("w_gate", "w_up", "w_down")
    cfg = mi.get_config("tiny", micro_count=2, clip_norm=0.01)
    params, toks = mi.make_params(cfg), [torch.as_tensor(v).cuda() for v in mi.make_update_tokens(cfg)]
    one, two = MoETrainer(cfg, "cuda:0"), MoETrainer(cfg, "cuda:0")
    for tr, last in ((one, sel), (two, stay)):
        tr.load_params(params)
        tr.micro_step(toks[0], 0, flags=stay)
        if tr is two:                        # a step of the shared tensors alone, the sum of the experts' goes on
            was = tr.grads.clone()
            stats = tr.clip_grads()
            assert stats.shape == (2,) and float(stats[1]) < 1
            for n in tr.layout:
                g, w = tr.view(tr.grads, n), tr.view(was, n)
                assert torch.equal(g, w) if n in experts else torch.allclose(g, w * float(stats[1]), rtol=1e-6, atol=0)
            total = sum(float((tr.view(was, n).double() ** 2).sum()) for n in tr.layout if n not in experts)
            assert abs(float(stats[0]) - total ** 0.5) < 1e-5 * total ** 0.5
        tr.micro_step(toks[1], 1, flags=last)
        assert tr.outputs().status == B.MT_OK
    out, was = one.outputs(), two.grads.clone()
    assert out.experts_updated == 1 and out.clip_coef < 1 and out.expert_clip_coef < 1
    stats = two.clip_grads()
    assert stats.shape == (2, 2)
    for got, want in zip(stats.reshape(-1).tolist(), (out.grad_norm, out.clip_coef, out.expert_grad_norm, out.expert_clip_coef)):
        assert abs(got - want) < 1e-5 * want
    for n in two.layout:
        by = float(stats[1, 1]) / 2 if n in experts else float(stats[0, 1])
        assert torch.allclose(two.view(two.grads, n), two.view(was, n) * by, rtol=1e-6, atol=0)


def test_trainer_takes_the_groups_of_its_flags():
    """Without a launch the trainer's own flags say which groups there are; a call may say it itself."""
    from adamw_persistent_sm_gb300 import binding as B
    from adamw_persistent_sm_gb300.trainer import MoETrainer
    cfg = mi.get_config("tiny", micro_count=4)
    tr = MoETrainer(cfg, "cuda:0", flags=B.MT_FLAG_SELECTIVE_EXPERTS)
    tr.grads.copy_(rnd(1, tr.n_params))
    was = tr.grads.clone()
    assert tr.clip_grads(max_norm=1e9).shape == (2, 2)
    for n in tr.layout:
        assert torch.equal(tr.view(tr.grads, n), tr.view(was, n) * (0.25 if n in ("w_gate", "w_up", "w_down") else 1.0))
    tr.grads.copy_(was)
    assert tr.clip_grads(max_norm=1e9, scale=2.0, micro_index=2).shape == (2,)
    for n in tr.layout:
        assert torch.equal(tr.view(tr.grads, n), tr.view(was, n) * (1.0 if n in ("w_gate", "w_up", "w_down") else 2.0))
    tr.grads.copy_(was)
    assert tr.clip_grads(max_norm=1e9, scale=2.0, flags=0).shape == (2,) and torch.equal(tr.grads, was * 2.0)
    with pytest.raises(ValueError):
        tr.clip_grads(micro_index=4)


def test_trainer_flags_set_later_and_refusals():
    """Flags that the trainer is given after it was made count as well; a refused call leaves every gradient."""
    from adamw_persistent_sm_gb300 import binding as B
    from adamw_persistent_sm_gb300.trainer import MoETrainer
    tr = MoETrainer(mi.get_config("tiny", micro_count=4), "cuda:0")
    tr.flags |= B.MT_FLAG_SELECTIVE_EXPERTS
    tr.grads.copy_(rnd(1, tr.n_params))
    was = tr.grads.clone()
    for kw in (dict(max_norm=-1.0), dict(scale=INF), dict(max_norm=NAN)):
        with pytest.raises(RuntimeError):
            tr.clip_grads(**kw)
        assert torch.equal(tr.grads, was)
    assert tr.clip_grads().shape == (2, 2)


# ---------------------------------------------------------------------------
# the clip factor
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("max_norm,eps,scale", [(1e17, 1e39, 1.0), (1e-6, 1e300, 1.0), (2.0, 1e40, 1e30), (1.0, 1e37, 1.0), (1e-40, 0.0, 1.0)])
def test_factors_beyond_32_bits(ops, max_norm, eps, scale):
    """c = max_norm / (norm + eps) where one of them is beyond fp32: off by the
    roundings of c and of the product, 3 steps of 2^-24, and by half of the least
    subnormal number of each."""
    t = rnd(1, 1000)
    norm = abs(scale) * float((t.double() ** 2).sum().sqrt())
    c = min(1.0, max_norm / (norm + eps))
    out = torch.empty_like(t)
    stats = ops.GradSet([t], [out]).clip(max_norm, eps, scale)
    assert abs(float(stats[1]) - c) <= 40 * 2.0 ** -24 * c + 1e-45
    want = t.double() * (scale * c)
    assert ((out.double() - want).abs() <= 43 * 2.0 ** -24 * want.abs() + 1e-45 * (1 + t.double().abs())).all()


# ---------------------------------------------------------------------------
# arguments
# ---------------------------------------------------------------------------
def test_numbers_of_choices(ops, monkeypatch):
    """top_k is any whole number; another is refused with the device as it was."""
    z = rnd(1, 6, 8)
    c = ops.choose(z, 2)
    assert all(torch.equal(a, b) for a, b in zip(c[:4], ops.choose(z, np.int64(2))[:4]))
    assert all(torch.equal(a, b) for a, b in zip(c[:4], ops.choose(z, np.int32(2), out=ops.choose(z + 1, 2))[:4]))
    now = [7]
    monkeypatch.setattr(ops, "_current", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "set_device", lambda d: now.__setitem__(0, d))
    for out in (None, c):
        with pytest.raises(TypeError):
            ops.choose(z, 2.0, out=out)
        assert now == [7]
