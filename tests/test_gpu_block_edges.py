"""The operators around the expert layer in calls that their definitions allow and
that are easily answered wrongly: gradients that are not finite beside tokens and
experts that take no part."""
import pytest
import torch

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
