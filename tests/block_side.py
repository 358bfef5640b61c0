"""Which side a wrong output comes from: the device that made it, the copy that
brought it to the host, or the inputs that the device had."""
import torch


def _bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


def _differ(a, b):
    """Number of elements whose bits differ, and the first few with both values."""
    at = torch.nonzero(_bits(a) != _bits(b))
    return len(at), [(tuple(i), float(a[tuple(i)]), float(b[tuple(i)])) for i in at[:4].tolist()]


def which_side(out, copy, again, inputs):
    """``out``: the output where it was made, ``copy``: what the host was given of
    it, ``again``: makes it once more from the same inputs, ``inputs``: name ->
    (tensor there, what the host had sent).  A list of the findings."""
    found = []
    n, at = _differ(out.cpu(), copy)
    if n:
        found.append(f"copy: {n} elements of a second copy of the output differ from the first's, {at}")
    n, at = _differ(again(), out)
    if n:
        found.append(f"device: {n} elements of another call's output differ, {at}")
    for name, (there, sent) in inputs.items():
        n, at = _differ(there.cpu(), sent)
        if n:
            n2, _ = _differ(there.cpu(), sent)
            found.append(f"input {name}: {n} elements ({n2} of a second copy) differ from what was sent, {at}")
    return found or ["none: output, copies, another call and inputs agree"]
