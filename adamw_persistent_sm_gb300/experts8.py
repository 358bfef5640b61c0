"""One expert layer with 8-bit products, forward and backward, from the
stand-alone operators (:mod:`.expert_ops`): route order, gather, gate/up
product, SwiGLU, down product and combine, with 8-bit checkpoints instead of
saved activations.

Between forward and backward the layer keeps, per expert row, d + 2 F bytes of
codes (its input, and g and u) and the down product's rows for the routing
weights' gradient, and a copy of the routing weights.  Every product takes e4m3
operands with a scale per block of 128: along the features for outputs and input
gradients (weights in 128 x 128 blocks, quantised once per
:meth:`ExpertLayer8.refresh` in both orientations), along the tokens for weight
gradients.  Weight gradients are fp32.  Neither pass records autograd history:
backward is called by the training program.
"""
from __future__ import annotations

import torch

from . import expert_ops as ops


class ExpertLayer8:
    """w_gate, w_up [E, F, d] and w_down [E, d, F] (float32 or bfloat16), for
    ``n_tokens`` tokens that name up to ``top_k`` experts each.  Buffers are
    allocated here and reused by every call; ``dtype`` is the type of the
    activations outside the 8-bit operands."""

    def __init__(self, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor, n_tokens: int, top_k: int,
                 dtype: torch.dtype = torch.bfloat16):
        if w_gate.dim() != 3:
            raise ValueError(f"w_gate: expected [E, F, d], got {tuple(w_gate.shape)}")
        self.n_experts, self.width, self.d = w_gate.shape
        self.device, self.dtype = w_gate.device, dtype
        self._check_weights(w_gate, w_up, w_down)
        e, f, d, dev = self.n_experts, self.width, self.d, self.device
        self.route = ops.Route(n_tokens, top_k, e, dev)
        rows = self.route.rows
        self.w_gu, self.w_gu_t = ops.empty8(2 * f, d, dev, 128, e), ops.empty8(d, 2 * f, dev, 128, e)
        self.w_down, self.w_down_t = ops.empty8(d, f, dev, 128, e), ops.empty8(f, d, dev, 128, e)
        # kept from forward to backward
        self.xs8, self.saved = ops.empty8(rows, d, dev), ops.empty8(rows, 2 * f, dev, halves=True)
        self.y = torch.empty((rows, d), dtype=dtype, device=dev)
        with torch.inference_mode(False):       # torch itself copies into it, in any mode
            self._w = torch.empty((n_tokens, top_k), dtype=torch.float32, device=dev)
        # passing buffers
        self.act8 = ops.empty8(rows, f, dev)
        self.gu = torch.empty((rows, 2 * f), dtype=dtype, device=dev)
        self.w = None
        self._captured = False              # a saving forward is part of a graph
        self._bwd = None
        self.refresh(w_gate, w_up, w_down)

    def _check_weights(self, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor) -> None:
        e, f, d = self.n_experts, self.width, self.d
        for t, what, shape in ((w_gate, "w_gate", (e, f, d)), (w_up, "w_up", (e, f, d)), (w_down, "w_down", (e, d, f))):
            if tuple(t.shape) != shape or t.device != self.device or t.dtype not in (torch.float32, torch.bfloat16):
                raise ValueError(f"{what}: expected float32 or bfloat16 {shape} on {self.device}, got {t.dtype} "
                                 f"{tuple(t.shape)} on {t.device}")
        # read where it lies; gate and up are copied together first
        ops._as_matrix(w_down, "w_down", w_down.get_device())

    def refresh(self, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor) -> None:
        """Quantise the weights (again, after an optimizer step).  Weights of other
        shapes than the layer was made with, or of another device or type, are
        refused before any of them is written.  A :meth:`backward` after it needs a
        new :meth:`forward`: the old one went through other weights (replays of a
        captured forward are not seen here: their order is the caller's)."""
        self._check_weights(w_gate, w_up, w_down)
        if not self._captured:
            self.w = None
        gu = torch.cat([w_gate.detach(), w_up.detach()], 1)
        ops.quant8(gu, 128, out=self.w_gu)
        ops.quant8_t(gu, 128, out=self.w_gu_t)
        ops.quant8(w_down, 128, out=self.w_down)
        ops.quant8_t(w_down, 128, out=self.w_down_t)

    def forward(self, x: torch.Tensor, idx: torch.Tensor, w: torch.Tensor, out: torch.Tensor | None = None,
                save: bool = True) -> torch.Tensor:
        """sum_k w[t, k] expert[idx[t, k]](x[t]) for x [n_tokens, d], idx int32
        and w float32 [n_tokens, top_k] (idx -1: no expert).  ``save`` False
        keeps nothing for :meth:`backward`."""
        r, self.w = self.route, None        # a forward that fails leaves nothing to go back through
        r.order(idx)
        r.dispatch8(x, out=self.xs8)
        ops.gemm8(self.xs8, self.w_gu, out=self.gu, offs=r.offs)
        ops.swiglu8(self.gu, act=self.act8, saved=self.saved if save else None, n_rows=r.offs[-1:])
        ops.gemm8(self.act8, self.w_down, out=self.y, offs=r.offs)
        out = r.combine(self.y, w, out=out)
        if save:                            # a copy: the caller's may hold the next microbatch's by then
            self.w = self._w.copy_(w.detach())
            self._captured = self._captured or torch.cuda.is_current_stream_capturing()
        return out

    def backward(self, dout: torch.Tensor, grads: tuple[torch.Tensor, torch.Tensor, torch.Tensor] | None = None,
                 accumulate: bool = False) -> tuple[torch.Tensor, torch.Tensor, tuple]:
        """Gradients after a saving :meth:`forward`: dx [n_tokens, d], dw
        [n_tokens, top_k] and (w_gate's, w_up's, w_down's), float32 in the
        weights' shapes - written into ``grads``, or added with ``accumulate``.
        A refused call has written none of them."""
        if self.w is None:
            raise RuntimeError("backward needs a forward with save=True before it")
        r, f, d, e, dev = self.route, self.width, self.d, self.n_experts, self.device
        shapes = ((e, f, d), (e, f, d), (e, d, f))
        if grads is None:
            if accumulate:
                raise ValueError("accumulate needs grads")
            grads = tuple(torch.empty(s, dtype=torch.float32, device=dev) for s in shapes)
        if len(grads) != 3:
            raise ValueError(f"grads: expected w_gate's, w_up's and w_down's, got {len(grads)}")
        for g, what, s in zip(grads, ("w_gate's gradient", "w_up's gradient", "w_down's gradient"), shapes):
            ops._sums(g, what, r._dev, s)
        if self._bwd is None:
            rows = r.rows
            like = lambda c: torch.empty((rows, c), dtype=self.dtype, device=dev)  # noqa: E731
            self._bwd = dict(dy=like(d), dact=like(f), act=like(f), dgu=like(2 * f), dxs=like(d),
                             dy8=ops.empty8(rows, d, dev), dgu8=ops.empty8(rows, 2 * f, dev),
                             dy_t=ops.empty8(d, rows, dev), act_t=ops.empty8(f, rows, dev),
                             dgu_t=ops.empty8(2 * f, rows, dev), xs_t=ops.empty8(d, rows, dev))
        b, n = self._bwd, r.offs[-1:]
        _, dw = r.combine_bwd(dout, self.y, self.w, dy=b["dy"])
        # through the down product
        ops.quant8(b["dy"], out=b["dy8"], n_rows=n)
        ops.gemm8(b["dy8"], self.w_down_t, out=b["dact"], offs=r.offs)
        ops.swiglu8_bwd(b["dact"], self.saved, dgu=b["dgu"], act=b["act"], n_rows=n)
        ops.quant8_t(b["dy"], out=b["dy_t"], n_rows=n)
        ops.quant8_t(b["act"], out=b["act_t"], n_rows=n)
        ops.gemm8_reduce(b["dy_t"], b["act_t"], r.offs, out=grads[2], accumulate=accumulate)
        # through the gate and up products; the input's codes are the forward's
        ops.quant8(b["dgu"], out=b["dgu8"], n_rows=n)
        ops.gemm8(b["dgu8"], self.w_gu_t, out=b["dxs"], offs=r.offs)
        ops.quant8_t(b["dgu"], out=b["dgu_t"], n_rows=n)
        ops.quant8_t(self.xs8, out=b["xs_t"], n_rows=n)
        ops.gemm8_reduce(b["dgu_t"].part(0, f), b["xs_t"], r.offs, out=grads[0], accumulate=accumulate)
        ops.gemm8_reduce(b["dgu_t"].part(f, 2 * f), b["xs_t"], r.offs, out=grads[1], accumulate=accumulate)
        return r.dispatch_bwd(b["dxs"]), dw, grads
