"""The operators around the expert layer as a training step uses them: together
with the layer, captured into graphs, on streams and threads, and beside the
trainer."""
import threading

import numpy as np
import pytest
import torch

import moe_inputs as mi

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from adamw_persistent_sm_gb300 import block_ops
    return block_ops


def rnd(seed, *shape, std=1.0, mean=0.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std + mean).to(dtype).cuda()


class Step:
    """One expert block of a pre-norm network with a norm and a gate behind the
    experts, forward and backward, and the clipping of its gradients."""

    def __init__(self, ops, seed=0, t=600, d=256, e=8, k=2, f=128):
        from adamw_persistent_sm_gb300 import ExpertLayer8
        self.ops, self.k = ops, k
        self.x, self.mask = rnd(seed, t, d), torch.ones(t, dtype=torch.bool, device="cuda")
        self.mask[-t // 10:] = False
        self.first, self.after, self.before = (rnd(seed + i, d, std=0.1, mean=1.0) for i in (1, 2, 3))
        self.gate, self.router = rnd(seed + 4, d, std=0.3), rnd(seed + 5, e, d, std=0.1)
        self.experts = rnd(seed + 6, e, f, d, std=0.06), rnd(seed + 7, e, f, d, std=0.06), rnd(seed + 8, e, d, f, std=0.06)
        self.layer = ExpertLayer8(*self.experts, t, k)
        self.dh, self.dr = rnd(seed + 9, t, d), rnd(seed + 10, t, d, dtype=torch.bfloat16)
        self.dlosses = torch.tensor([50.0, 5.0], device="cuda")
        self.choice = None
        self.grads = [torch.zeros_like(v) for v in (self.first, self.after, self.before, self.gate, self.router, *self.experts)]
        self.set = ops.GradSet(self.grads)

    def __call__(self):
        ops = self.ops
        gf, ga, gb, gg, gr = self.grads[:5]
        _, r = ops.block_norm(self.x, before=self.first, dtype=torch.bfloat16)
        logits = r.float() @ self.router.T
        c = self.choice = ops.choose(logits, self.k, self.mask, out=self.choice)
        y = self.layer.forward(r, c.idx, c.w)
        h2, r2 = ops.block_norm(self.x, y, after=self.after, gate=self.gate, before=self.before, out_scale=0.5)
        b = ops.block_norm_bwd(self.dr, self.dh, h2, y, after=self.after, gate=self.gate, before=self.before, out_scale=0.5,
                               dafter=ga, dgate=gg, dbefore=gb)
        dr, dw, _ = self.layer.backward(b.dy, tuple(self.grads[5:]))
        dz = ops.choose_bwd(logits, c.idx, c.counts, dw, self.dlosses, self.mask)
        torch.matmul(dz.T, r.float(), out=gr)
        dr = (dr.float() + dz @ self.router).bfloat16()
        b1 = ops.block_norm_bwd(dr, b.dx, self.x, before=self.first, dbefore=gf, dx=b.dx)
        stats = self.set.clip(1.0)
        return dict(h=h2, r=r2, dx=b1.dx, losses=c.losses, idx=c.idx, stats=stats, logits=logits, **{f"g{i}": g for i, g in enumerate(self.grads)})


def test_step_against_autograd(ops):
    """The whole step against float64 autograd of the unquantised block: 8-bit
    operands are off by up to 2^-4 each, two at a time over three products in a
    row; random errors of a third of that stay below a fifth of each gradient's
    norm (a wrong sign, factor or missing part does not).  The choices are the
    step's own."""
    s = Step(ops)
    got = s()
    p = {n: getattr(s, n).double().requires_grad_() for n in ("x", "first", "after", "before", "gate", "router")}
    w = [v.double().requires_grad_() for v in s.experts]

    def rms(v, g):
        return v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-5) * g

    r = rms(p["x"], p["first"])
    z = r @ p["router"].T
    live, idx, n = s.mask, got["idx"].long(), int(s.mask.sum())
    weight = torch.softmax(z.gather(1, idx.clamp(min=0)), 1)
    y = torch.zeros_like(r)
    for k in range(s.k):
        for e in range(len(w[0])):
            at = torch.nonzero(idx[:, k] == e)[:, 0]
            act = torch.nn.functional.silu(r[at] @ w[0][e].T) * (r[at] @ w[1][e].T)
            y = y.index_add(0, at, weight[at, k:k + 1] * (act @ w[2][e].T))
    h = p["x"] + 0.5 * p["gate"] * rms(y, p["after"])
    out = rms(h, p["before"])
    load = torch.bincount(idx[idx >= 0], minlength=len(w[0])).double()
    prob = torch.softmax(z[live], 1)
    balance = len(w[0]) * (load / (s.k * n) * prob.mean(0)).sum()
    size = (torch.logsumexp(z[live], 1) ** 2).mean()
    ((s.dh.double() * h).sum() + (s.dr.double() * out).sum() + 50.0 * balance + 5.0 * size).backward()
    want = [p[k].grad for k in ("first", "after", "before", "gate", "router")] + [v.grad for v in w]
    norm = float(torch.stack([(v * v).sum() for v in want]).sum().sqrt())
    rel = lambda a, b: float((a.double() - b.detach()).norm() / b.detach().norm())                # noqa: E731
    assert rel(got["h"], h) < 0.05 and rel(got["r"], out) < 0.05 and rel(got["dx"], p["x"].grad) < 0.2
    assert all(abs(float(a) - float(b.detach())) < 0.05 * float(b.detach()) for a, b in zip(got["losses"], (balance, size)))
    assert abs(float(got["stats"][0]) - norm) < 0.2 * norm
    clip = min(1.0, 1.0 / (norm + 1e-6))
    for i, v in enumerate(want):
        assert rel(got[f"g{i}"], v * clip) < 0.3, i
    total = float(torch.stack([(g.double() ** 2).sum() for g in s.grads]).sum().sqrt())
    assert abs(total - 1.0) < 1e-4
    # the same logits give the same choices in float64
    zz = np.where(s.mask.cpu().numpy()[:, None], got["logits"].cpu().double().numpy(), -np.inf)
    by = np.argsort(-zz, 1, kind="stable")[:, :s.k]
    assert np.array_equal(np.where(s.mask.cpu().numpy()[:, None], by, -1), got["idx"].cpu().numpy())


def clones(d):
    return {k: v.clone() for k, v in d.items()}


def test_step_captured_and_replayed(ops):
    """A captured step gives the eager one's results bit for bit, with the eager
    results still held, also on inputs written after the capture."""
    eager = Step(ops)
    want = clones(eager())
    held = eager()
    s = Step(ops)
    s()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = s()
    for _ in range(3):
        for v in out.values():
            v.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], want[k]) for k in want)
    other = Step(ops, seed=100)
    want2 = clones(other())
    for n in ("x", "first", "after", "before", "gate", "router", "dh", "dr"):
        getattr(s, n).copy_(getattr(other, n))
    s.layer.refresh(*other.experts)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[k], want2[k]) for k in want2)
    assert all(torch.equal(held[k], want[k]) for k in want)


def test_two_graphs_at_once(ops):
    """Two captured steps with nothing in common, replayed on two streams at once."""
    steps = [Step(ops, seed=s, t=t) for s, t in ((1, 900), (2, 1300))]
    want = [clones(s()) for s in steps]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in steps:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(s())
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(5):
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(o[k], w[k]) for k in w)


def test_streams_and_threads(ops):
    """Eager steps on streams of their own, from threads of their own."""
    steps = [Step(ops, seed=s, t=700 + 100 * s) for s in range(3)]
    want = [clones(s()) for s in steps]
    torch.cuda.synchronize()
    got, errors = [None] * len(steps), []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    got[i] = steps[i]()
                torch.cuda.current_stream().synchronize()
        except Exception as ex:            # noqa: BLE001
            errors.append(ex)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(steps))]
    for th in threads:
        th.start()
    for th in threads:
        th.join(60)
    torch.cuda.synchronize()
    assert not errors
    for w, o in zip(want, got):
        assert all(torch.equal(o[k], w[k]) for k in w)


def test_one_set_and_one_input_on_two_streams(ops):
    """Calls that read the same tensors at once and write others do not meet:
    workspaces are a call's own, in graphs too."""
    x, y, w = rnd(1, 4000, 768), rnd(2, 4000, 768, dtype=torch.bfloat16), rnd(3, 768, mean=1.0)
    dr, z = rnd(4, 4000, 768, dtype=torch.bfloat16), rnd(5, 40000, 64)
    gs = ops.GradSet([x, y, w])
    calls = [lambda: ops.block_norm_bwd(dr, x, x, y, after=w, gate=w, before=w), lambda: ops.choose(z, 8), lambda: (gs.norm(),)]
    want = [[v.clone() for v in f()[:5]] for f in calls]
    torch.cuda.synchronize()
    runs = []
    for f in calls:
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                out = f()
            runs.append((g, out, torch.cuda.Stream()))
    for _ in range(4):
        for g, _, st in runs:
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for i, (_, out, _) in enumerate(runs):
        n = 4 if i // 2 == 1 else 5
        assert all(torch.equal(a, b) for a, b in zip(out[:n], want[i // 2][:n]))


def test_many_tensors_captured(ops):
    """More tensors than one launch's table holds, captured and replayed on other values."""
    ts = [rnd(i, 3 + i % 7) for i in range(1100)]
    gs = ops.GradSet(ts)
    gs.norm()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        norm, stats = gs.norm(), gs.clip(2.0)
    for v in (1.0, 3.0):
        for i, t in enumerate(ts):
            t.copy_(rnd(i, t.numel()) * v)
        want = float(torch.cat(ts).double().norm())
        g.replay()
        torch.cuda.synchronize()
        assert abs(float(norm) - want) < 1e-5 * want and abs(float(stats[0]) - want) < 1e-5 * want
        assert abs(float(torch.cat(ts).double().norm()) - 2.0) < 1e-5


FIRST = """
import sys
import torch
from adamw_persistent_sm_gb300 import block_ops as ops
torch.manual_seed(0)
x, w, z = torch.randn(500, 768, device="cuda"), torch.rand(768, device="cuda"), torch.randn(50000, 64, device="cuda")
y = x.bfloat16()
g = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
def step():
    h, r = ops.block_norm(x, y, after=w, gate=w, before=w)
    b = ops.block_norm_bwd(r, h, h, y, after=w, gate=w, before=w)
    c = ops.choose(z, 8)
    return (h, r, *b, *c[:4], ops.choose_bwd(z, c.idx, c.counts, c.w, c.losses), ops.GradSet([x]).norm(), ops.GradSet([w], [torch.empty_like(w)]).clip(1.0))
with torch.cuda.graph(g):
    out = step()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, step()))
print("same")
"""


def test_first_calls_of_a_process_captured():
    """No operator needs a call before the capture that holds its first."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and done.stdout.strip().endswith("same"), done.stderr[-2000:]


def test_between_other_kernels(ops):
    """Plain tensor kernels write what the operators read and read what they write, without waiting."""
    t, d = 3000, 512
    x, y, w = torch.zeros(t, d, device="cuda"), torch.zeros(t, d, device="cuda"), torch.ones(d, device="cuda")
    h, r = torch.empty_like(x), torch.empty_like(x)
    z, c = torch.zeros(t, 16, device="cuda"), None
    for i in range(30):
        x.fill_(i + 1.0)
        y.fill_(2.0 * i)
        ops.block_norm(x, y, before=w, h=h, r=r)
        assert_later = h.sum()
        z.zero_()
        z[:, i % 16] = 5.0
        c = ops.choose(z, 1, out=c)
        at = c.idx.sum()
        g = [h.clone(), r.clone()]
        s = ops.clip_grads(g, 1.0)
        assert float(assert_later) == (3.0 * i + 1.0) * t * d and int(at) == t * (i % 16)
        assert abs(float(torch.stack([v.double().pow(2).sum() for v in g]).sum()) - 1.0) < 1e-3 and float(s[1]) < 1.0


def test_modes_and_requires_grad(ops):
    """No history is recorded, whatever the inputs require; results made in inference mode can be used."""
    x, y, w = rnd(1, 50, 64).requires_grad_(), rnd(2, 50, 64).requires_grad_(), rnd(3, 64).requires_grad_()
    h, r = ops.block_norm(x, y, after=w, gate=w, before=w)
    g = ops.block_norm_bwd(r, h, h, y, after=w, gate=w, before=w)
    c = ops.choose(x, 2)
    z = ops.choose_bwd(x, c.idx, c.counts, c.w, c.losses)
    for v in (h, r, *g, *c, z, ops.GradSet([x]).norm(), ops.clip_grads([y], 1e9)):
        assert not v.requires_grad
    with torch.inference_mode():
        h2, r2 = ops.block_norm(x, y, after=w, gate=w, before=w)
        c2 = ops.choose(x, 2)
    assert torch.equal(h, h2) and torch.equal(r, r2) and all(torch.equal(a, b) for a, b in zip(c[:4], ops.choose(x, 2, out=c2)[:4]))


def test_refusals_leave_the_device_as_it_was(ops, monkeypatch):
    """With another device current, a refused argument raises before the device changes, or changes it back."""
    x, w, z = rnd(1, 6, 64), rnd(2, 64), rnd(3, 6, 8)
    gs, c = ops.GradSet([x]), ops.choose(z, 2)
    now = [7]
    monkeypatch.setattr(ops, "_current", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "set_device", lambda d: now.__setitem__(0, d))
    for call in (lambda: ops.block_norm(x, x, before=w[:-1]), lambda: ops.block_norm(x, x, before=w, eps=0.0),
                 lambda: ops.block_norm(x, x, before=w, eps="small"), lambda: ops.block_norm_bwd(x, x, x, x, before=w, eps=-1.0),
                 lambda: ops.block_norm_bwd(x, x, x, x, before=w, dbefore=x), lambda: ops.choose(z, 9), lambda: ops.choose(z, "2"),
                 lambda: ops.choose_bwd(z, c.idx), lambda: ops.choose_bwd(z, c.idx.long(), dw=c.w), lambda: gs.clip(-1.0),
                 lambda: gs.clip("one"), lambda: gs.norm(float("nan")), lambda: gs.norm(None)):
        with pytest.raises(Exception):
            call()
        assert now == [7]


def test_trainer_clips_as_its_update_does(ops):
    """MoETrainer.clip_grads on the gradients of a launch without its optimizer:
    the norm and the coefficient that the update's own step reports (its norm is an
    fp32 sum of a quarter of a million squares: within 1e-5)."""
    from adamw_persistent_sm_gb300 import binding as B
    from adamw_persistent_sm_gb300.trainer import MoETrainer
    cfg = mi.get_config("tiny")
    params, toks = mi.make_params(cfg), torch.as_tensor(mi.make_update_tokens(cfg)[0]).cuda()
    one, two = MoETrainer(cfg, "cuda:0"), MoETrainer(cfg, "cuda:0")
    for tr, flags in ((one, 0), (two, B.MT_FLAG_NO_OPTIMIZER)):
        tr.load_params(params)
        tr.micro_step(toks, flags=flags)
        assert tr.outputs().status == B.MT_OK
    out, grads = one.outputs(), two.grads.clone()
    stats = two.clip_grads()
    assert abs(float(stats[0]) - out.grad_norm) < 1e-5 * out.grad_norm and abs(float(stats[1]) - out.clip_coef) < 1e-5
    assert torch.allclose(two.grads, grads * float(stats[1]), rtol=1e-6, atol=0)
    before = two.grads.clone()
    stats = two.clip_grads(max_norm=1e6, scale=2.0)
    assert float(stats[1]) == 1.0 and torch.equal(two.grads, before * 2.0)
