"""The expert layer's stand-alone operators on torch tensors.

The functions check types, shapes and devices, pass pointers to the C ABI
(``include/moe_train.h`` has each operator's definition) on the tensors'
device and its current stream, and return the outputs.  Outputs may be given
(``out=`` and the like); otherwise they are allocated through torch.  Nothing
here synchronises, but for the first call on a device, which has to come before
a stream capture: a device-side failure is reported by :func:`check`.

* :class:`Route` - tokens sorted by expert and back, and the gradients;
* :class:`Tensor8`, :func:`quant8`, :func:`quant8_t`, :func:`dequant8`,
  :func:`gemm8`, :func:`gemm8_reduce` - products of e4m3 matrices with a
  power-of-two scale per block of 128;
* :func:`swiglu8`, :func:`swiglu8_bwd` - SwiGLU that saves its inputs in 8 bits.

Matrices may be views whose rows are contiguous (any row stride).  The
functions record no autograd history, whatever their arguments require: each
gradient is an operator of its own, called in the backward pass.
"""
from __future__ import annotations

import ctypes as C
import threading

import torch

from . import binding as B

_DTYPES = {torch.float32: B.MT_DT_FP32, torch.bfloat16: B.MT_DT_BF16}
_status: dict = {}          # device index -> (int32 [2] status words, their address)
_status_lock = threading.Lock()


def _error(what: str, st: int) -> Exception:
    from .trainer import StatusError
    return StatusError(f"{what}: {B.status_string(st)} ({st})")


_current = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


# Every operator makes its device current around the call of the C ABI (a
# no-op in the usual case) and passes that device's current stream.  Nothing
# between the two changes of device may raise: arguments are checked before.


def _status_word(dev: int) -> int:
    """Address of the device's status words."""
    t = _status.get(dev)
    if t is None:
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("the first operator, Route or Tensor8 on a device comes before a stream capture")
        with _status_lock:                      # one pair, however many threads come first
            t = _status.get(dev)
            if t is None:
                with torch.inference_mode(False):       # check() clears them in any mode
                    t = torch.zeros(2, dtype=torch.int32, device=f"cuda:{dev}")
                torch.cuda.synchronize(dev)     # once per device: zeroed before any other stream uses it
                t = _status[dev] = (t, t.data_ptr())
    return t[1]


def check(device: str | torch.device = "cuda") -> None:
    """Wait for the device and raise if an operator reported a failure there
    since the last call (an index out of range, a wait that ran out)."""
    dev = _device(device).index
    _status_word(dev)
    t = _status[dev][0]
    torch.cuda.synchronize(dev)
    st, site = t.tolist()
    if st != B.MT_OK:
        t.zero_()
        torch.cuda.synchronize(dev)             # cleared before another stream can report again
        raise _error(f"device-side check (site {site})", st)


def _device(device) -> torch.device:
    dev = torch.device(device)
    if dev.type != "cuda":
        raise ValueError(f"expected a CUDA device, got {dev}")
    return dev if dev.index is not None else torch.device("cuda", torch.cuda.current_device())


def _mat(t: torch.Tensor, what: str, dev: int, rows: int | None = None, cols: int | None = None,
         dtype=None) -> int:
    """Checks a [rows, cols] matrix with contiguous rows on a device; its row stride."""
    shape = t.shape
    if len(shape) != 2 or t.get_device() != dev or dev < 0:
        raise ValueError(f"{what}: expected a matrix on cuda:{dev}, got {tuple(shape)} on {t.device}")
    if dtype is not None and t.dtype is not dtype or dtype is None and t.dtype not in _DTYPES:
        raise TypeError(f"{what}: {t.dtype} where {dtype or 'float32 or bfloat16'} is needed")
    r, c = shape
    if (rows is not None and r != rows) or (cols is not None and c != cols):
        raise ValueError(f"{what}: expected [{rows}, {cols}], got [{r}, {c}]")
    if t.is_contiguous():
        return c
    s0, s1 = t.stride()
    if (s1 != 1 and c > 1) or (s0 < c and r > 1):
        raise ValueError(f"{what}: rows must be contiguous and may not overlap (strides {s0}, {s1})")
    return s0 if s0 >= c else c


def _ints(t: torch.Tensor, what: str, dev: int, shape) -> int:
    if t.dtype is not torch.int32 or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what}: expected contiguous int32 {tuple(shape)} on cuda:{dev}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _limit(n_rows, dev: int) -> int:
    if n_rows is None:
        return 0
    return _ints(n_rows, "n_rows", dev, (1,))


# ---------------------------------------------------------------------------
# matrices in 8 bits
# ---------------------------------------------------------------------------
class Tensor8:
    """A matrix, or a stack of them, held as e4m3 codes and scale bytes.

    ``codes`` uint8 [rows, ld] or [batch, rows, ld], ld a multiple of 16 and at
    least ``cols``; ``scales`` uint8 [rows, blocks] (block_rows 1) or
    [ceil(rows / 128), blocks] (block_rows 128), with the same batch dimension.
    Scale rows may lie further apart; a multiple of four bytes, as
    :func:`empty8` makes them, lets products read them by words.
    ``halves``: the columns are two parts with blocks of their own.
    """

    __slots__ = ("codes", "scales", "rows", "cols", "batch", "shape", "block_rows", "halves", "device", "_dev",
                 "_mat", "_ref")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, cols: int, block_rows: int = 1,
                 halves: bool = False):
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise TypeError("codes and scales are uint8")
        if codes.dim() not in (2, 3) or scales.dim() != codes.dim() or codes.device != scales.device \
                or codes.device.type != "cuda":
            raise ValueError("codes and scales are matrices, or stacks of them, on one CUDA device")
        if block_rows not in (1, 128) or cols < 1 or (halves and (cols % 2 or block_rows != 1)):
            raise ValueError(f"block_rows {block_rows}, cols {cols}, halves {halves}")
        batch = codes.shape[0] if codes.dim() == 3 else 1
        rows, ld = codes.shape[-2:]
        blocks = 2 * -(-(cols // 2) // 128) if halves else -(-cols // 128)
        need = (-(-rows // 128) if block_rows == 128 else rows, blocks)
        if tuple(scales.shape[-2:]) != need or (codes.dim() == 3 and scales.shape[0] != batch):
            raise ValueError(f"scales: expected {need} for each matrix, got {tuple(scales.shape)}")
        if ld < cols or ld % 16 or not codes.is_contiguous() or codes.data_ptr() % 16:
            raise ValueError(f"codes: rows of {ld} bytes hold {cols} columns, start on 16-byte boundaries "
                             "and are contiguous")
        lds = scales.stride(-2) if need[0] > 1 else max(scales.stride(-2), blocks)
        if lds < blocks or (blocks > 1 and scales.stride(-1) != 1) or \
                (batch > 1 and need[0] and scales.stride(0) != need[0] * lds):
            raise ValueError(f"scales: rows are contiguous and matrices follow one another (strides {scales.stride()})")
        self.codes, self.scales, self.cols, self.block_rows, self.halves = codes, scales, cols, block_rows, halves
        self.device, self._dev = codes.device, codes.get_device()
        _status_word(self._dev)
        self.rows, self.batch, self.shape = rows, batch, (*codes.shape[:-1], cols)
        # Matrices of no rows have no storage and nothing reads them: any address
        # stands in.  A stack of no matrices keeps its batch of 0, which every
        # entry point refuses: its rows would be read at that address.
        none = 16 if rows == 0 else 0
        self._mat = B.mt_mat8(codes.data_ptr() or none, scales.data_ptr() or none, rows, cols, ld, lds, block_rows,
                              batch, int(halves), 0)
        self._ref = C.byref(self._mat)

    def __getitem__(self, i: int) -> "Tensor8":
        """Matrix i of a stack (a view)."""
        if self.codes.dim() != 3:
            raise IndexError("not a stack of matrices")
        return Tensor8(self.codes[i], self.scales[i], self.cols, self.block_rows, self.halves)

    def part(self, lo: int, hi: int) -> "Tensor8":
        """Rows lo..hi-1 of a matrix with block_rows 1 (a view)."""
        if self.codes.dim() != 2 or self.block_rows != 1 or not 0 <= lo <= hi <= self.rows:
            raise IndexError(f"rows {lo}:{hi} of {self.shape}, block_rows {self.block_rows}")
        return Tensor8(self.codes[lo:hi], self.scales[lo:hi], self.cols, 1, self.halves)


def empty8(rows: int, cols: int, device="cuda", block_rows: int = 1, batch: int | None = None,
           halves: bool = False) -> Tensor8:
    """Buffers for an 8-bit matrix, or a stack of ``batch``."""
    dev = _device(device)
    lead = () if batch is None else (batch,)
    blocks = 2 * -(-(cols // 2) // 128) if halves else -(-cols // 128)
    codes = torch.empty((*lead, rows, -(-cols // 16) * 16), dtype=torch.uint8, device=dev)
    scales = torch.empty((*lead, -(-rows // 128) if block_rows == 128 else rows, -(-blocks // 4) * 4),
                         dtype=torch.uint8, device=dev)
    return Tensor8(codes, scales[..., :blocks], cols, block_rows, halves)


def _as_matrix(x: torch.Tensor, what: str, dev) -> tuple[int, int]:
    """A matrix or a stack whose matrices follow one another: (batch, row stride)."""
    if x.dim() == 2:
        return 1, _mat(x, what, dev)
    if x.dim() != 3:
        raise ValueError(f"{what}: expected a matrix or a stack of matrices, got {tuple(x.shape)}")
    if x.shape[0] > 1 and x.shape[1] > 0 and x.stride(0) != x.shape[1] * x.stride(1):
        raise ValueError(f"{what}: the matrices of a stack must follow one another")
    if x.shape[1] == 1:
        return x.shape[0], _mat(x[:, 0], what, dev)
    return x.shape[0], _mat(x[0], what, dev) if x.shape[0] else x.shape[2]


def quant8(x: torch.Tensor, block_rows: int = 1, out: Tensor8 | None = None, n_rows: torch.Tensor | None = None,
           halves: bool = False) -> Tensor8:
    """x [rows, cols] or [batch, rows, cols] in 8 bits.  ``n_rows`` (device
    int32 [1]): only rows below it are written.  ``out`` brings its own
    block_rows and halves."""
    dev = x.get_device()
    batch, ldx = _as_matrix(x, "x", dev)
    if out is None:
        out = empty8(x.shape[-2], x.shape[-1], dev, block_rows, batch if x.dim() == 3 else None, halves)
    if out.shape != tuple(x.shape) or out._dev != dev:
        raise ValueError(f"out: expected {tuple(x.shape)} on cuda:{dev}, got {out.shape} on {out.device}")
    if batch == 0:
        return out
    lim = _limit(n_rows, dev)
    here = _current()
    if here != dev:
        torch.cuda.set_device(dev)
    st = B.load().mt_quant8(x.data_ptr(), _DTYPES[x.dtype], ldx, lim, out._ref, _raw_stream(dev))
    if here != dev:
        torch.cuda.set_device(here)
    if st:
        raise _error("mt_quant8", st)
    return out


def quant8_t(x, block_rows: int = 1, out: Tensor8 | None = None, n_rows: torch.Tensor | None = None) -> Tensor8:
    """The transpose of x [rows, cols] in 8 bits, [cols, rows]: with block_rows
    1 each scale covers 128 rows of a column of x.  x is a matrix, a stack, or
    a :class:`Tensor8` saved earlier (block_rows 1)."""
    dev = x._dev if isinstance(x, Tensor8) else x.get_device()
    rows, cols = x.shape[-2:]
    lead = tuple(x.shape[:-2])
    src, ptr, dt, ldx = None, 0, 0, 0
    if isinstance(x, Tensor8):
        src = x._ref
    else:
        _, ldx = _as_matrix(x, "x", dev)
        ptr, dt = x.data_ptr(), _DTYPES[x.dtype]
    if out is None:
        out = empty8(cols, rows, dev, block_rows, lead[0] if lead else None)
    if out.shape != (*lead, cols, rows) or out._dev != dev:
        raise ValueError(f"out: expected {(*lead, cols, rows)} on cuda:{dev}, got {out.shape} on {out.device}")
    if lead and lead[0] == 0:
        return out
    lim = _limit(n_rows, dev)
    here = _current()
    if here != dev:
        torch.cuda.set_device(dev)
    st = B.load().mt_quant8_t(ptr, dt, ldx, src, lim, out._ref, _raw_stream(dev))
    if here != dev:
        torch.cuda.set_device(here)
    if st:
        raise _error("mt_quant8_t", st)
    return out


def dequant8(a: Tensor8, dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
             n_rows: torch.Tensor | None = None) -> torch.Tensor:
    """The values of an 8-bit matrix (block_rows 1)."""
    dev = a._dev
    if out is None:
        out = torch.empty(a.shape, dtype=dtype, device=dev)
    ldo, lim = _mat(out, "out", dev, a.rows, a.cols), _limit(n_rows, dev)
    here = _current()
    if here != dev:
        torch.cuda.set_device(dev)
    st = B.load().mt_dequant8(a._ref, lim, out.data_ptr(), _DTYPES[out.dtype], ldo, _raw_stream(dev))
    if here != dev:
        torch.cuda.set_device(here)
    if st:
        raise _error("mt_dequant8", st)
    return out


def gemm8(a: Tensor8, b: Tensor8, out: torch.Tensor | None = None, offs: torch.Tensor | None = None,
          dtype: torch.dtype = torch.bfloat16, accumulate: bool = False) -> torch.Tensor:
    """a b^T: a [M, K]; b [N, K], or with ``offs`` (int32 [E+1] row starts, also a
    run of consecutive experts of a routing) [E, N, K]; rows outside the segments
    are left as they were."""
    dev = a._dev
    if b._dev != dev:
        raise ValueError(f"b is on {b.device}, a on cuda:{dev}")
    seg = b.batch if offs is not None else 0
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = torch.empty((a.rows, b.rows), dtype=dtype, device=dev)
    ldc = _mat(out, "out", dev, a.rows, b.rows)
    po = 0 if offs is None else _ints(offs, "offs", dev, (seg + 1,))
    here = _current()
    if here != dev:
        torch.cuda.set_device(dev)
    st = B.load().mt_gemm8(a._ref, b._ref, po, seg, out.data_ptr(), _DTYPES[out.dtype], ldc, int(accumulate),
                           _status_word(dev), _raw_stream(dev))
    if here != dev:
        torch.cuda.set_device(here)
    if st:
        raise _error("mt_gemm8", st)
    return out


def _sums(out: torch.Tensor, what: str, dev: int, shape: tuple) -> int:
    """Checks an output of :func:`gemm8_reduce`; its row stride."""
    if out.dim() != 3 or out.dtype != torch.float32 or tuple(out.shape) != shape:
        raise ValueError(f"{what}: expected float32 {shape}, got {out.dtype} {tuple(out.shape)}")
    return _as_matrix(out, what, dev)[1]


def gemm8_reduce(a: Tensor8, b: Tensor8, offs: torch.Tensor, out: torch.Tensor | None = None,
                 accumulate: bool = False) -> torch.Tensor:
    """out[e] = a[:, offs[e]:offs[e+1]] b[:, same]^T in fp32: a [M, P], b [N, P]."""
    dev = a._dev
    seg = offs.numel() - 1
    if b._dev != dev:
        raise ValueError(f"b is on {b.device}, a on cuda:{dev}")
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = torch.empty((max(seg, 0), a.rows, b.rows), dtype=torch.float32, device=dev)
    ldc = _sums(out, "out", dev, (seg, a.rows, b.rows))
    po = _ints(offs, "offs", dev, (seg + 1,))
    here = _current()
    if here != dev:
        torch.cuda.set_device(dev)
    st = B.load().mt_gemm8_reduce(a._ref, b._ref, po, seg, out.data_ptr(), ldc,
                                  int(accumulate), _status_word(dev), _raw_stream(dev))
    if here != dev:
        torch.cuda.set_device(here)
    if st:
        raise _error("mt_gemm8_reduce", st)
    return out


def swiglu8(gu: torch.Tensor, act: Tensor8 | None = None, saved: Tensor8 | None = None,
            n_rows: torch.Tensor | None = None) -> Tensor8:
    """silu(g) * u of gu = [g | u], in 8 bits; ``saved`` (empty8 with halves)
    receives g and u for :func:`swiglu8_bwd`."""
    dev = gu.get_device()
    ld = _mat(gu, "gu", dev)
    rows, cols = gu.shape
    if cols % 2 or cols < 2:
        raise ValueError(f"gu: an even number of columns, got {cols}")
    if act is None:
        act = empty8(rows, cols // 2, dev)
    if act.shape != (rows, cols // 2) or act._dev != dev or (saved is not None and saved._dev != dev):
        raise ValueError(f"act: expected {(rows, cols // 2)} on cuda:{dev}, got {act.shape} on {act.device}")
    lim = _limit(n_rows, dev)
    here = _current()
    if here != dev:
        torch.cuda.set_device(dev)
    st = B.load().mt_swiglu8(gu.data_ptr(), _DTYPES[gu.dtype], ld, lim, act._ref,
                             saved._ref if saved is not None else None, _raw_stream(dev))
    if here != dev:
        torch.cuda.set_device(here)
    if st:
        raise _error("mt_swiglu8", st)
    return act


def swiglu8_bwd(dact: torch.Tensor, saved: Tensor8, dgu: torch.Tensor | None = None,
                act: torch.Tensor | None = None, n_rows: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of :func:`swiglu8` at the saved g and u; ``act``, where given,
    receives silu(g) * u of the saved values."""
    dev = dact.get_device()
    ldd = _mat(dact, "dact", dev, saved.rows, saved.cols // 2)
    if saved._dev != dev:
        raise ValueError(f"saved is on {saved.device}, dact on cuda:{dev}")
    if dgu is None:
        dgu = torch.empty(saved.shape, dtype=dact.dtype, device=dev)
    ldg = _mat(dgu, "dgu", dev, saved.rows, saved.cols, dact.dtype)
    lda = 0 if act is None else _mat(act, "act", dev, *dact.shape, dact.dtype)
    lim = _limit(n_rows, dev)
    here = _current()
    if here != dev:
        torch.cuda.set_device(dev)
    st = B.load().mt_swiglu8_bwd(dact.data_ptr(), _DTYPES[dact.dtype], ldd, saved._ref, lim,
                                 dgu.data_ptr(), ldg, 0 if act is None else act.data_ptr(), lda, _raw_stream(dev))
    if here != dev:
        torch.cuda.set_device(here)
    if st:
        raise _error("mt_swiglu8_bwd", st)
    return dgu


# ---------------------------------------------------------------------------
# tokens sorted by expert and back
# ---------------------------------------------------------------------------
class Route:
    """Buffers of a routing of ``n_tokens`` x ``top_k`` assignments over
    ``n_experts``, refilled by :meth:`order`: ``offs`` [E+1] segment starts,
    ``perm`` [rows] the assignment at each row, ``row`` [n_tokens, top_k] the
    row of each assignment (all int32, -1 for none).  Calls that refill or read
    one Route, captured ones too, have to be ordered by the caller."""

    def __init__(self, n_tokens: int, top_k: int, n_experts: int, device="cuda"):
        dev = _device(device)
        rows = B.load().mt_route_rows(n_tokens, top_k, n_experts)
        if rows < 0:
            raise _error("mt_route_rows", -rows)
        self._set(torch.empty(n_experts + 1, dtype=torch.int32, device=dev),
                  torch.empty(rows, dtype=torch.int32, device=dev),
                  torch.empty((n_tokens, top_k), dtype=torch.int32, device=dev))
        self._workspace()

    def _workspace(self) -> None:
        self.ws = torch.empty(B.load().mt_route_ws_bytes(self.n_tokens, self.top_k, self.n_experts),
                              dtype=torch.uint8, device=self.device)
        self._ws = (self.ws.data_ptr(), self.ws.numel())

    @classmethod
    def of(cls, offs: torch.Tensor, perm: torch.Tensor, row: torch.Tensor) -> "Route":
        """A routing ordered before, from its three tensors."""
        r = cls.__new__(cls)
        r._set(offs, perm, row)
        r.ws = None
        return r

    def _set(self, offs, perm, row):
        self.device, self._dev = offs.device, offs.get_device()
        if self._dev >= 0:
            _status_word(self._dev)
        if row.dim() != 2 or offs.dim() != 1 or perm.dim() != 1 or self.device.type != "cuda":
            raise ValueError("offs [E+1], perm [rows] and row [tokens, top_k] on a CUDA device")
        self.n_tokens, self.top_k = row.shape
        self.n_experts, self.rows = offs.numel() - 1, perm.numel()
        rows = B.load().mt_route_rows(self.n_tokens, self.top_k, self.n_experts)
        if rows < 0:
            raise _error("mt_route_rows", -rows)
        if rows != self.rows:
            raise ValueError(f"perm: expected {rows} rows, got {self.rows}")
        self.offs, self.perm, self.row = offs, perm, row
        dev = self._dev
        self._ptrs = (_ints(offs, "offs", dev, offs.shape), _ints(perm, "perm", dev, perm.shape),
                      _ints(row, "row", dev, row.shape))

    def order(self, idx: torch.Tensor) -> "Route":
        """Sort idx int32 [n_tokens, top_k] (-1: no expert)."""
        dev = self._dev
        if self.ws is None:
            self._workspace()
        p = _ints(idx, "idx", dev, self.row.shape)
        here = _current()
        if here != dev:
            torch.cuda.set_device(dev)
        st = B.load().mt_route_order(p, self.n_tokens, self.top_k, self.n_experts, *self._ptrs, *self._ws,
                                     _status_word(dev), _raw_stream(dev))
        if here != dev:
            torch.cuda.set_device(here)
        if st:
            raise _error("mt_route_order", st)
        return self

    def dispatch(self, x: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
        """x [n_tokens, width] to the rows of its experts, [rows, width]; zeros
        in padding rows; rows behind the last segment are left as they were."""
        dev = self._dev
        ldx = _mat(x, "x", dev, self.n_tokens)
        if out is None:
            out = torch.empty((self.rows, x.shape[1]), dtype=x.dtype, device=dev)
        ldo = _mat(out, "out", dev, self.rows, x.shape[1], x.dtype)
        here = _current()
        if here != dev:
            torch.cuda.set_device(dev)
        st = B.load().mt_dispatch(x.data_ptr(), _DTYPES[x.dtype], ldx, self.n_tokens, x.shape[1], self.top_k,
                                  self.n_experts, *self._ptrs, self.rows, out.data_ptr(), ldo, _raw_stream(dev))
        if here != dev:
            torch.cuda.set_device(here)
        if st:
            raise _error("mt_dispatch", st)
        return out

    def dispatch8(self, x: torch.Tensor, out: Tensor8 | None = None) -> Tensor8:
        """:meth:`dispatch` with the rows quantised on their way."""
        dev = self._dev
        ldx = _mat(x, "x", dev, self.n_tokens)
        if out is None:
            out = empty8(self.rows, x.shape[1], dev)
        if out.shape != (self.rows, x.shape[1]) or out._dev != dev:
            raise ValueError(f"out: expected {(self.rows, x.shape[1])} on cuda:{dev}, got {out.shape} on {out.device}")
        here = _current()
        if here != dev:
            torch.cuda.set_device(dev)
        st = B.load().mt_dispatch8(x.data_ptr(), _DTYPES[x.dtype], ldx, self.n_tokens, self.top_k, self.n_experts,
                                   *self._ptrs, out._ref, _raw_stream(dev))
        if here != dev:
            torch.cuda.set_device(here)
        if st:
            raise _error("mt_dispatch8", st)
        return out

    def _weights(self, w: torch.Tensor, what: str) -> int:
        if w.dtype is not torch.float32 or w.get_device() != self._dev or w.shape != self.row.shape \
                or not w.is_contiguous():
            raise ValueError(f"{what}: expected contiguous float32 {tuple(self.row.shape)} on {self.device}")
        return w.data_ptr()

    def combine(self, y: torch.Tensor, w: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
        """Rows y [rows, width] back to tokens, weighted by w float32
        [n_tokens, top_k] (None: plain sums)."""
        dev = self._dev
        ldy = _mat(y, "y", dev, self.rows)
        if out is None:
            out = torch.empty((self.n_tokens, y.shape[1]), dtype=y.dtype, device=dev)
        ldo = _mat(out, "out", dev, self.n_tokens, y.shape[1], y.dtype)
        pw = 0 if w is None else self._weights(w, "w")
        here = _current()
        if here != dev:
            torch.cuda.set_device(dev)
        st = B.load().mt_combine(y.data_ptr(), _DTYPES[y.dtype], ldy, self.rows, self._ptrs[2], pw, self.n_tokens,
                                 self.top_k, y.shape[1], out.data_ptr(), ldo, _raw_stream(dev))
        if here != dev:
            torch.cuda.set_device(here)
        if st:
            raise _error("mt_combine", st)
        return out

    def dispatch_bwd(self, dxs: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
        """Gradient of :meth:`dispatch`: the sum of each token's rows."""
        return self.combine(dxs, None, out)

    def combine_bwd(self, dout: torch.Tensor, y: torch.Tensor, w: torch.Tensor, dy: torch.Tensor | None = None,
                    dw: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
        """Gradients of :meth:`combine` for y (zeros in padding rows, rows
        behind the last segment left as they were) and for w."""
        dev = self._dev
        width = dout.shape[-1]
        ldd = _mat(dout, "dout", dev, self.n_tokens)
        ldy = _mat(y, "y", dev, self.rows, width, dout.dtype)
        if dy is None:
            dy = torch.empty((self.rows, width), dtype=dout.dtype, device=dev)
        if dw is None:
            dw = torch.empty(self.row.shape, dtype=torch.float32, device=dev)
        ldg = _mat(dy, "dy", dev, self.rows, width, dout.dtype)
        pw, pdw = self._weights(w, "w"), self._weights(dw, "dw")
        here = _current()
        if here != dev:
            torch.cuda.set_device(dev)
        st = B.load().mt_combine_bwd(dout.data_ptr(), _DTYPES[dout.dtype], ldd, y.data_ptr(), ldy, *self._ptrs,
                                     self.rows, pw, self.n_tokens, self.top_k, self.n_experts,
                                     width, dy.data_ptr(), ldg, pdw, _raw_stream(dev))
        if here != dev:
            torch.cuda.set_device(here)
        if st:
            raise _error("mt_combine_bwd", st)
        return dy, dw
