"""Stand-alone operators around the expert layer, on torch tensors.

What a training step needs between, before and after the operators of
:mod:`.expert_ops`, with the same conventions (``include/moe_train.h`` has each
operator's definition): arguments are checked on the host, work is enqueued on
the tensors' device and its current stream, outputs may be given and are
allocated through torch otherwise, nothing synchronises or records autograd
history.

* :func:`block_norm`, :func:`block_norm_bwd` - the joint between two blocks: the
  norm after a block, its gate, the scaled residual sum, the norm before the next;
* :func:`choose`, :func:`choose_bwd` - the experts of each token from the router's
  logits, counts, a balance loss and a loss on the logits' size;
* :class:`GradSet`, :func:`grad_norm`, :func:`clip_grads` - the global norm of many
  gradient tensors, and their clipping.

Matrices may be views whose rows are contiguous (any row stride).
"""
from __future__ import annotations

import operator
from typing import NamedTuple, Sequence

import torch

from . import binding as B
from .expert_ops import _DTYPES, _current, _error, _limit, _mat, _raw_stream

__all__ = ["block_norm", "block_norm_bwd", "BlockGrads", "choose", "choose_bwd", "Choice", "GradSet", "grad_norm",
           "clip_grads"]


def _vec(t: torch.Tensor | None, what: str, dev: int, n: int) -> int | None:
    """Address of a contiguous fp32 vector [n], None for none."""
    if t is None:
        return None
    if t.dtype is not _F32 or t.get_device() != dev or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{what}: expected contiguous float32 [{n}] on cuda:{dev}, got {t.dtype} {tuple(t.shape)} "
                         f"on {t.device}")
    return t.data_ptr()


def _rows(t: torch.Tensor, what: str, dev: int, shape, dtype) -> int:
    """:func:`_mat` of a matrix of this shape and type, quicker where it is contiguous."""
    if t.shape == shape and t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
        return shape[1]
    return _mat(t, what, dev, shape[0], shape[1], dtype)


class _Space:
    """Memory of a call's own, on a device and for its current stream, from
    torch's allocator and back to it when the object goes (a tensor for it would
    cost a call 5 us more)."""

    __slots__ = ("ptr",)

    def __init__(self, nbytes: int, dev: int):
        self.ptr = 0
        here = _current()
        if here != dev:
            torch.cuda.set_device(dev)
        try:
            self.ptr = torch._C._cuda_cudaCachingAllocator_raw_alloc(nbytes, _raw_stream(dev))
        finally:
            if here != dev:
                torch.cuda.set_device(here)

    def __del__(self):
        if self.ptr:
            torch._C._cuda_cudaCachingAllocator_raw_delete(self.ptr)


_F32 = torch.float32
_load = B.load


# ---------------------------------------------------------------------------
# the joint between two blocks
# ---------------------------------------------------------------------------
class BlockGrads(NamedTuple):
    """Gradients of :func:`block_norm`; None where there is no such input."""
    dx: torch.Tensor
    dy: torch.Tensor | None
    dafter: torch.Tensor | None
    dgate: torch.Tensor | None
    dbefore: torch.Tensor | None


def _joint(shape, stream, dtype, after, gate, before, res_scale, out_scale, eps, n_rows, dev):
    """The C ABI's description of a joint."""
    rows, width = shape
    kind = ldgate = 0
    pg = None
    if gate is not None:
        if gate.dim() == 1:
            kind, pg = B.MT_GATE_CHANNEL, _vec(gate, "gate", dev, width)
        elif gate.dim() == 2 and gate.shape[1] == 1 and (width > 1 or gate.dtype is _F32):
            kind, ldgate = B.MT_GATE_TOKEN, _mat(gate, "gate", dev, rows, 1, _F32)
        else:
            kind, ldgate = B.MT_GATE_FULL, _rows(gate, "gate", dev, shape, dtype)
        pg = gate.data_ptr() or 16          # of no rows: present, and read by nothing
    return B.mt_joint(rows, width, _DTYPES[stream], _DTYPES[dtype], _vec(after, "after", dev, width),
                      _vec(before, "before", dev, width), pg, ldgate, None if n_rows is None else _limit(n_rows, dev),
                      kind, res_scale, out_scale, eps, 0)


def _summed(given, grad, what: str, dev: int, width: int, accumulate: bool):
    """The gradient of a vector that rows share, and its address."""
    if given is None:
        raise ValueError(f"{what} of nothing")
    if grad is None:
        if accumulate:
            raise ValueError(f"accumulate needs {what}")
        grad = torch.empty(width, dtype=_F32, device=dev)
        return grad, grad.data_ptr()
    return grad, _vec(grad, what, dev, width)


def _alone(after, gate, res_scale) -> None:
    if after is not None or gate is not None or res_scale != 1.0:
        raise ValueError("after, gate and res_scale belong to a block's output y")


def block_norm(x: torch.Tensor, y: torch.Tensor | None = None, *, after: torch.Tensor | None = None,
               gate: torch.Tensor | None = None, before: torch.Tensor | None = None, res_scale: float = 1.0,
               out_scale: float = 1.0, eps: float = 1e-5, h: torch.Tensor | None = None,
               r: torch.Tensor | None = None, n_rows: torch.Tensor | None = None,
               dtype: torch.dtype | None = None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """The joint between two blocks, in one pass: with rms(v) = sqrt(mean(v^2) +
    eps) over the columns,

        h = res_scale * x + out_scale * gate * (y / rms(y) * after)
        r = h / rms(h) * before

    x [rows, width] is the residual stream (float32 or bfloat16, as h), y the
    block's output.  ``after`` and ``before`` are float32 [width]; without
    ``after`` y is taken as it is, without ``before`` r is None.  ``gate`` is
    float32 [width], float32 [rows, 1], or [rows, width] of y's type.  Without y
    the call is the norm before the first block: h is x itself.  y and r have
    one type, the stream's or bfloat16 (``dtype`` gives r's where there is no y).
    ``h`` may be x (in place).  ``n_rows`` (device int32 [1]): rows from it on are
    left as they were.  Up to 8192 columns.  Returns (h, r)."""
    dev, shape, stream = x.get_device(), x.shape, x.dtype
    ldx = _mat(x, "x", dev)
    ldy = ldh = ldr = 0
    py = ph = pr = None
    if y is None:
        _alone(after, gate, res_scale)
        if before is None or h is not None:
            raise ValueError("without y there is no h to write, and before is needed")
        dtype = r.dtype if r is not None else dtype or stream
        if dtype not in _DTYPES:
            raise TypeError(f"r: {dtype} where float32 or bfloat16 is needed")
    else:
        if dtype is not None and dtype is not y.dtype:
            raise TypeError(f"r has y's type {y.dtype}, not {dtype}")
        dtype = y.dtype
        if dtype not in _DTYPES:
            raise TypeError(f"y: {dtype} where float32 or bfloat16 is needed")
        ldy = _rows(y, "y", dev, shape, dtype)
        if h is None:
            h = torch.empty(shape, dtype=stream, device=dev)
        ldh = _rows(h, "h", dev, shape, stream)
        py, ph = y.data_ptr(), h.data_ptr()
    if before is not None:
        if r is None:
            r = torch.empty(shape, dtype=dtype, device=dev)
        ldr = _rows(r, "r", dev, shape, dtype)
        pr = r.data_ptr()
    elif r is not None:
        raise ValueError("r needs before")
    j = _joint(shape, stream, dtype, after, gate, before, res_scale, out_scale, eps, n_rows, dev)
    lib, px, here = _load(), x.data_ptr(), _current()
    if here != dev:
        torch.cuda.set_device(dev)
    st = lib.mt_block_norm(j, px, ldx, py, ldy, ph, ldh, pr, ldr, _raw_stream(dev))
    if here != dev:
        torch.cuda.set_device(here)
    if st:
        raise _error("mt_block_norm", st)
    return (x if y is None else h), r


def block_norm_bwd(dr: torch.Tensor | None, dh: torch.Tensor | None, h: torch.Tensor, y: torch.Tensor | None = None, *,
                   after: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                   before: torch.Tensor | None = None, res_scale: float = 1.0, out_scale: float = 1.0,
                   eps: float = 1e-5, dx: torch.Tensor | None = None, dy: torch.Tensor | None = None,
                   dgate: torch.Tensor | None = None, dafter: torch.Tensor | None = None,
                   dbefore: torch.Tensor | None = None, accumulate: bool = False,
                   n_rows: torch.Tensor | None = None) -> BlockGrads:
    """Gradients of :func:`block_norm` from those of r and h, at the h and y that
    it left (nothing else is kept).  ``dh`` is what reaches h along the residual
    stream, of h's type (None: nothing); ``dr`` has y's type (None exactly where
    ``before`` is).  ``dx`` may be dh (in place).  ``dafter``, ``dbefore`` and the
    gradient of a gate [width] are sums over the rows, float32; with
    ``accumulate`` they are added to what the given tensors hold."""
    accumulate = int(bool(accumulate))
    dev, shape, stream = h.get_device(), h.shape, h.dtype
    ldh = _mat(h, "h", dev)
    rows, width = shape
    if dr is None and dh is None:
        raise ValueError("a gradient of r or of h is needed")
    if (dr is None) != (before is None):
        raise ValueError("dr and before come together")
    dtype = y.dtype if y is not None else dr.dtype if dr is not None else stream
    if dtype not in _DTYPES:
        raise TypeError(f"y or dr: {dtype} where float32 or bfloat16 is needed")
    lddr = lddh = ldy = lddy = lddgate = 0
    pdr = pdh = py = pdy = pdg = pda = pdb = None
    if dr is not None:
        lddr, pdr = _rows(dr, "dr", dev, shape, dtype), dr.data_ptr()
    if dh is not None:
        lddh, pdh = _rows(dh, "dh", dev, shape, stream), dh.data_ptr()
    if y is None:
        _alone(after, gate, res_scale)
        if dy is not None:
            raise ValueError("dy needs y")
    else:
        ldy, py = _rows(y, "y", dev, shape, dtype), y.data_ptr()
    j = _joint(shape, stream, dtype, after, gate, before, res_scale, out_scale, eps, n_rows, dev)
    if dx is None:
        dx = torch.empty(shape, dtype=stream, device=dev)
    lddx = _rows(dx, "dx", dev, shape, stream)
    if y is not None:
        if dy is None:
            dy = torch.empty(shape, dtype=dtype, device=dev)
        lddy, pdy = _rows(dy, "dy", dev, shape, dtype), dy.data_ptr()
    if after is not None or dafter is not None:
        dafter, pda = _summed(after, dafter, "dafter", dev, width, accumulate)
    if before is not None or dbefore is not None:
        dbefore, pdb = _summed(before, dbefore, "dbefore", dev, width, accumulate)
    channel = gate is not None and gate.dim() == 1
    if channel or gate is None and dgate is not None:
        dgate, pdg = _summed(gate, dgate, "dgate", dev, width, accumulate)
    elif gate is not None:
        if dgate is None:
            dgate = torch.empty(gate.shape, dtype=gate.dtype, device=dev)
        lddgate = _mat(dgate, "dgate", dev, rows, gate.shape[1], gate.dtype)
        pdg = dgate.data_ptr()
    lib, px, nbytes, pws = _load(), dx.data_ptr(), 0, None
    if after is not None or before is not None or channel:
        nbytes = lib.mt_block_norm_ws_bytes(rows, width)
        if nbytes < 0:
            raise _error("mt_block_norm_bwd", -nbytes)
        if nbytes:
            ws = _Space(nbytes, dev)        # held until the launches
            pws = ws.ptr
    ph, here = h.data_ptr(), _current()
    if here != dev:
        torch.cuda.set_device(dev)
    st = lib.mt_block_norm_bwd(j, ph, ldh, py, ldy, pdr, lddr, pdh, lddh, px, lddx, pdy, lddy, pdg, lddgate, pda, pdb,
                               accumulate, pws, nbytes, _raw_stream(dev))
    if here != dev:
        torch.cuda.set_device(here)
    if st:
        raise _error("mt_block_norm_bwd", st)
    return BlockGrads(dx, dy, dafter, dgate, dbefore)


# ---------------------------------------------------------------------------
# the router's choice
# ---------------------------------------------------------------------------
class Choice(NamedTuple):
    """The experts of a batch of tokens, as :func:`choose` leaves them."""
    idx: torch.Tensor       # int32 [tokens, top_k], best first, -1: none
    w: torch.Tensor         # float32 [tokens, top_k]
    counts: torch.Tensor    # int32 [experts + 1]: tokens that chose each, and the number that take part
    losses: torch.Tensor    # float32 [2]: balance, mean squared log of the sum of exponentials
    ws: torch.Tensor        # workspace


def _logits(z: torch.Tensor, mask) -> tuple[int, int]:
    dev = z.get_device()
    ldz = _mat(z, "logits", dev)
    if mask is not None and (mask.dtype not in (torch.bool, torch.uint8) or mask.get_device() != dev
                             or mask.shape != z.shape[:1] or not mask.is_contiguous()):
        raise ValueError(f"mask: expected contiguous bool [{z.shape[0]}] on cuda:{dev}, got {mask.dtype} "
                         f"{tuple(mask.shape)} on {mask.device}")
    return dev, ldz


def _plain(t: torch.Tensor, what: str, dev: int, shape, dtype) -> int:
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what}: expected contiguous {dtype} {tuple(shape)} on cuda:{dev}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def choose(logits: torch.Tensor, top_k: int, mask: torch.Tensor | None = None, renormalize: bool = True,
           out: Choice | None = None) -> Choice:
    """The ``top_k`` experts of each token by its logits [tokens, experts]
    (float32 or bfloat16; equal logits: the lowest expert first), their weights
    (softmax, divided by the chosen ones' sum with ``renormalize``), the tokens
    that chose each expert, and two losses: the balance loss experts * sum_e f_e
    P_e of the shares f and the mean probabilities P, and the mean squared
    logsumexp.  ``mask`` (bool [tokens]): False takes no part and goes nowhere.
    An expert whose logit is -inf is never chosen.  ``out`` is refilled; calls
    that refill or read one Choice, captured ones too, have to be ordered by the
    caller."""
    dev, ldz = _logits(logits, mask)
    t, e = logits.shape
    top_k = operator.index(top_k)
    lib, picked = _load(), (t, top_k)
    if out is None:
        nbytes = lib.mt_choose_ws_bytes(t, top_k, e)
        if nbytes < 0:
            raise _error("mt_choose", -nbytes)
        out = Choice(torch.empty(picked, dtype=torch.int32, device=dev), torch.empty(picked, dtype=_F32, device=dev),
                     torch.empty(e + 1, dtype=torch.int32, device=dev), torch.empty(2, dtype=_F32, device=dev),
                     torch.empty(nbytes, dtype=torch.uint8, device=dev))
    idx, w, counts, losses, ws = out
    nbytes = ws.numel()
    args = (_plain(idx, "idx", dev, picked, torch.int32), _plain(w, "w", dev, picked, _F32),
            _plain(counts, "counts", dev, (e + 1,), torch.int32), _plain(losses, "losses", dev, (2,), _F32),
            _plain(ws, "ws", dev, (nbytes,), torch.uint8))
    what, pm, keep = (logits.data_ptr(), _DTYPES[logits.dtype], ldz, t, e), None if mask is None else mask.data_ptr(), int(renormalize)
    here = _current()
    if here != dev:
        torch.cuda.set_device(dev)
    st = lib.mt_choose(*what, top_k, pm, keep, *args, nbytes, _raw_stream(dev))
    if here != dev:
        torch.cuda.set_device(here)
    if st:
        raise _error("mt_choose", st)
    return out


def choose_bwd(logits: torch.Tensor, idx: torch.Tensor, counts: torch.Tensor | None = None,
               dw: torch.Tensor | None = None, dlosses: torch.Tensor | None = None, mask: torch.Tensor | None = None,
               renormalize: bool = True, out: torch.Tensor | None = None) -> torch.Tensor:
    """The gradient for the logits, of their type: through the weights of the
    chosen (``dw`` float32 [tokens, top_k]) and through the two losses
    (``dlosses`` float32 [2] on the device, with the ``counts`` of the choice);
    either may be None."""
    dev, ldz = _logits(logits, mask)
    t, e = logits.shape
    if dw is None and dlosses is None:
        raise ValueError("dw or dlosses is needed")
    if idx.dim() != 2:
        raise ValueError(f"idx: expected [tokens, top_k], got {tuple(idx.shape)}")
    k = idx.shape[1]
    pi = _plain(idx, "idx", dev, (t, k), torch.int32)
    pw = None if dw is None else _plain(dw, "dw", dev, (t, k), torch.float32)
    pl = pc = None
    if dlosses is not None:
        if counts is None:
            raise ValueError("dlosses needs counts")
        pl, pc = _plain(dlosses, "dlosses", dev, (2,), torch.float32), _plain(counts, "counts", dev, (e + 1,), torch.int32)
    if out is None:
        out = torch.empty((t, e), dtype=logits.dtype, device=dev)
    ldo = _rows(out, "out", dev, logits.shape, logits.dtype)
    keep, po = int(renormalize), out.data_ptr()
    lib, here = _load(), _current()
    if here != dev:
        torch.cuda.set_device(dev)
    st = lib.mt_choose_bwd(logits.data_ptr(), _DTYPES[logits.dtype], ldz, t, e, k,
                           None if mask is None else mask.data_ptr(), keep, pi, pc, pw, pl, po, ldo, _raw_stream(dev))
    if here != dev:
        torch.cuda.set_device(here)
    if st:
        raise _error("mt_choose_bwd", st)
    return out


# ---------------------------------------------------------------------------
# the gradient norm and clipping
# ---------------------------------------------------------------------------
def _dense(t: torch.Tensor) -> bool:
    """Whether a tensor's elements fill one run of memory (in any order of dimensions)."""
    if t.is_contiguous():
        return True
    run = 1
    for step, n in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n > 1):
        if step != run:
            return False
        run *= n
    return True


class GradSet:
    """A set of gradient tensors on one device (float32 or bfloat16, mixed as
    they come) for :meth:`norm` and :meth:`clip`; ``out``: tensors that receive
    the clipped ones (default: in place).  Tensors are dense (contiguous, or a
    permutation of that) and do not overlap; an output is its gradient itself, or
    has its type, shape and strides and overlaps no tensor of the set.

    The set is of the memory that the tensors have when it is made, which it keeps
    alive: each call takes the values that are there then, and looks at no tensor
    again (500 of them would take 110 us).  Tensors that were given other memory
    since (``t.data = ...``, a new ``.grad``) need a new set; memory may not be
    taken from under it (a storage resized).  Results and workspaces are new at
    each call."""

    def __init__(self, tensors: Sequence[torch.Tensor], out: Sequence[torch.Tensor] | None = None,
                 device: str | torch.device | None = None):
        tensors = list(tensors)
        out = tensors if out is None else list(out)
        if len(out) != len(tensors):
            raise ValueError(f"{len(out)} outputs for {len(tensors)} tensors")
        if device is None:
            device = tensors[0].device if tensors else "cuda"
        self.device = torch.device(device)
        if self.device.type != "cuda":
            raise ValueError(f"expected tensors on a CUDA device, got {self.device}")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self._dev = dev = self.device.index
        spans, runs = [], []
        for i, (t, o) in enumerate(zip(tensors, out)):
            if t.dtype not in _DTYPES or t.get_device() != dev or t.layout is not torch.strided or not _dense(t):
                raise ValueError(f"tensor {i}: expected dense float32 or bfloat16 on cuda:{dev}, got {t.dtype} "
                                 f"{tuple(t.shape)} on {t.device}")
            if o is not t and (o.dtype is not t.dtype or o.get_device() != dev or o.shape != t.shape
                               or o.stride() != t.stride()):
                raise ValueError(f"output {i}: expected {t.dtype} {tuple(t.shape)} with strides {t.stride()} on "
                                 f"cuda:{dev}, got {o.dtype} {tuple(o.shape)} with strides {o.stride()} on {o.device}")
            n, a, b = t.numel(), t.data_ptr(), o.data_ptr()
            if n:
                runs.append((a, a + n * t.element_size(), i))
                if a != b:
                    runs.append((b, b + n * t.element_size(), i))
            spans.append((a, b, n, _DTYPES[t.dtype], 0))
        runs.sort()
        for (_, end, i), (start, _, k) in zip(runs, runs[1:]):
            if start < end:
                raise ValueError(f"tensors or outputs {i} and {k} overlap")
        self._n = len(spans)
        self._spans = (B.mt_span * max(1, len(spans)))(*spans)
        self._bytes = B.load().mt_grad_ws_bytes(len(spans))
        self._kept = {s.data_ptr(): s for s in (t.untyped_storage() for t in (*tensors, *out))}

    def norm(self, scale: float = 1.0) -> torch.Tensor:
        """|scale| times the square root of the sum of all squares, float32 [1]."""
        ws = _Space(self._bytes, self._dev)
        norm = torch.empty(1, dtype=_F32, device=self._dev)
        scale = float(scale)
        dev, lib, here = self._dev, B.load(), _current()
        if here != dev:
            torch.cuda.set_device(dev)
        st = lib.mt_grad_norm(self._spans, self._n, scale, norm.data_ptr(), ws.ptr, self._bytes,
                              _raw_stream(dev))
        if here != dev:
            torch.cuda.set_device(here)
        if st:
            raise _error("mt_grad_norm", st)
        return norm

    def clip(self, max_norm: float, eps: float = 1e-6, scale: float = 1.0) -> torch.Tensor:
        """The tensors times scale * c, c = min(1, max_norm / (norm + eps)) with
        the norm of the scaled tensors (NaN where that is NaN).  ``scale`` turns
        a sum over microbatches or of scaled losses into the gradient.  Returns
        (norm, c), float32 [2]."""
        ws = _Space(self._bytes, self._dev)
        stats = torch.empty(2, dtype=_F32, device=self._dev)
        max_norm, eps, scale = float(max_norm), float(eps), float(scale)
        dev, lib, here = self._dev, B.load(), _current()
        if here != dev:
            torch.cuda.set_device(dev)
        st = lib.mt_grad_clip(self._spans, self._n, max_norm, eps, scale, stats.data_ptr(), ws.ptr,
                              self._bytes, _raw_stream(dev))
        if here != dev:
            torch.cuda.set_device(here)
        if st:
            raise _error("mt_grad_clip", st)
        return stats


def grad_norm(tensors: Sequence[torch.Tensor], scale: float = 1.0) -> torch.Tensor:
    """:meth:`GradSet.norm` of tensors taken together once."""
    return GradSet(tensors).norm(scale)


def clip_grads(tensors: Sequence[torch.Tensor], max_norm: float, eps: float = 1e-6, scale: float = 1.0,
               out: Sequence[torch.Tensor] | None = None) -> torch.Tensor:
    """:meth:`GradSet.clip` of tensors taken together once."""
    return GradSet(tensors, out).clip(max_norm, eps, scale)
