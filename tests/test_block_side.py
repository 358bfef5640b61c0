"""The helper that says which side a wrong output comes from, with each mistake planted on the host."""
import torch

from block_side import which_side


def case(dtype=torch.float32):
    x = torch.randn(5, 7, generator=torch.Generator().manual_seed(1)).to(dtype)
    return x, x * 2, lambda: x * 2


def test_no_side():
    for dtype in (torch.float32, torch.bfloat16):
        x, out, again = case(dtype)
        assert which_side(out, out.clone(), again, {"x": (x, x.clone())})[0].startswith("none")
        out[2, 3] = float("nan")              # the same bits on both sides
        assert which_side(out, out.clone(), lambda: out.clone(), {})[0].startswith("none")


def test_each_side():
    for dtype in (torch.float32, torch.bfloat16):
        x, out, again = case(dtype)
        wrong = out.clone()
        wrong[2, 3] += 16
        found = which_side(out, wrong, again, {"x": (x, x.clone())})
        assert len(found) == 1 and found[0].startswith("copy: 1 element") and "(2, 3)" in found[0]
        found = which_side(wrong, wrong.clone(), again, {"x": (x, x.clone())})
        assert len(found) == 1 and found[0].startswith("device: 1 element") and "(2, 3)" in found[0]
        sent = x.clone()
        sent[0] = -sent[0]
        found = which_side(out, out.clone(), again, {"y": (x, x.clone()), "x": (x, sent)})
        assert len(found) == 1 and found[0].startswith("input x: 7 elements (7 of a second copy)")
