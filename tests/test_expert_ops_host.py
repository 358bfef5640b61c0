"""Argument checks of the stand-alone expert operators (C ABI and torch
wrappers).  Every call here is refused or has nothing to do before anything
is enqueued: the addresses are never dereferenced."""
import ctypes as C

import numpy as np
import pytest
import torch

import expert_ref as R
from adamw_persistent_sm_gb300 import binding as B
from adamw_persistent_sm_gb300 import expert_ops as ops

P = 1 << 20                     # an aligned address
BAD, UNS = B.MT_ERR_ARG, B.MT_ERR_UNSUPPORTED
F32, BF16 = B.MT_DT_FP32, B.MT_DT_BF16


@pytest.fixture(scope="module")
def lib():
    return B.load(build_if_missing=True)


def mat(rows=64, cols=256, **kw):
    m = dict(codes=P, scales=P, rows=rows, cols=cols, ld=-(-cols // 16) * 16, lds=-(-cols // 128), block_rows=1,
             batch=1, halves=0, reserved0=0)
    m.update(kw)
    return C.byref(B.mt_mat8(*[m[k] for k, _ in B.mt_mat8._fields_]))


def test_mat8_layout_matches_header():
    assert C.sizeof(B.mt_mat8) == 64


@pytest.mark.parametrize("t,k,e,want", [(0, 1, 1, 128), (1, 2, 16, 2048), (32768, 2, 16, 67584), (10, 8, 64, 8320)])
def test_route_rows(lib, t, k, e, want):
    assert lib.mt_route_rows(t, k, e) == want == R.rows_max(t, k, e)
    assert lib.mt_route_ws_bytes(t, k, e) > 0


@pytest.mark.parametrize("t,k,e,code", [(-1, 1, 1, BAD), (1, 0, 4, BAD), (1, 1, 0, BAD), (1, 9, 16, UNS), (1, 3, 2, UNS),
                                        (1, 1, 65, UNS), (1 << 30, 2, 4, UNS), (1 << 40, 1, 1, UNS)])
def test_route_limits(lib, t, k, e, code):
    assert lib.mt_route_rows(t, k, e) == -code
    assert lib.mt_route_ws_bytes(t, k, e) == -code
    assert lib.mt_route_order(P, t, k, e, P, P, P, P, 1 << 30, P, 0) == code
    rows = 128
    assert lib.mt_dispatch(P, F32, 8, t, 8, k, e, P, P, P, rows, P, 8, 0) == code


def test_route_order_refusals(lib):
    ok = [P, 4, 2, 4, P, P, P, P, 1 << 20, P, 0]
    for i in (0, 4, 5, 6, 9):
        a = list(ok)
        a[i] = 0
        assert lib.mt_route_order(*a) == BAD, i
        a[i] = P + 2
        assert lib.mt_route_order(*a) == BAD, i
    big = [P, 100000, 2, 4, P, P, P, P, lib.mt_route_ws_bytes(100000, 2, 4) - 1, P, 0]
    assert lib.mt_route_order(*big) == B.MT_ERR_ARENA_SMALL
    big[7] = 0
    assert lib.mt_route_order(*big) == BAD


def test_move_refusals(lib):
    rows = lib.mt_route_rows(4, 2, 4)
    d = [P, F32, 8, 4, 8, 2, 4, P, P, P, rows, P, 8, 0]
    for i, v in ((0, 0), (0, P + 1), (1, 2), (1, -1), (2, 7), (4, 0), (7, 0), (8, 0), (9, P + 2), (10, rows - 128),
                 (10, -1), (11, 0), (12, 7)):
        a = list(d)
        a[i] = v
        assert lib.mt_dispatch(*a) == BAD, (i, v)
    d8 = [P, F32, 8, 4, 2, 4, P, P, P]
    for m in (mat(rows, 8, block_rows=128), mat(rows, 8, batch=2), mat(rows, 8, halves=1), mat(rows + 128, 8),
              mat(rows, 8, codes=P + 8), mat(rows, 8, ld=24), mat(rows, 8, lds=0), mat(rows, 8, reserved0=1), None):
        assert lib.mt_dispatch8(*d8, m, 0) == BAD
    c = [P, BF16, 8, rows, P, P, 4, 2, 8, P, 8, 0]
    for i, v in ((0, 0), (1, 7), (2, 7), (3, -1), (4, 0), (5, P + 2), (8, 0), (9, P + 1), (10, 4)):
        a = list(c)
        a[i] = v
        assert lib.mt_combine(*a) == BAD, (i, v)
    b = [P, BF16, 8, P, 8, P, P, P, rows, P, 4, 2, 4, 8, P, 8, P, 0]
    for i, v in ((0, 0), (1, 3), (2, 7), (3, 0), (4, 7), (5, 0), (6, 0), (7, 0), (8, 128), (9, 0), (14, 0), (15, 7),
                 (16, 0), (16, P + 2)):
        a = list(b)
        a[i] = v
        assert lib.mt_combine_bwd(*a) == BAD, (i, v)
    # nothing to move: no buffer is needed
    r0 = lib.mt_route_rows(0, 2, 4)
    assert lib.mt_dispatch(0, F32, 8, 0, 8, 2, 4, P, P, P, r0, P, 8, 0) == B.MT_OK
    assert lib.mt_combine(P, F32, 8, r0, 0, 0, 0, 2, 8, 0, 8, 0) == B.MT_OK


def test_quant_refusals(lib):
    assert lib.mt_quant8(P, F32, 256, 0, mat(rows=0), 0) == B.MT_OK
    for a in ((0, F32, 256, 0, mat()), (P + 2, F32, 256, 0, mat()), (P, 2, 256, 0, mat()), (P, F32, 255, 0, mat()),
              (P, F32, 256, P + 1, mat()), (P, F32, 256, P, mat(block_rows=128)), (P, F32, 256, P, mat(batch=2)),
              (P, F32, 256, 0, mat(block_rows=64)), (P, F32, 256, 0, mat(cols=0)), (P, F32, 256, 0, mat(rows=-1)),
              (P, F32, 256, 0, mat(batch=0)), (P, F32, 256, 0, mat(halves=1, cols=255)),
              (P, F32, 256, 0, mat(halves=1, block_rows=128)), (P, F32, 256, 0, mat(halves=2)),
              (P, F32, 256, 0, mat(scales=0)), (P, F32, 256, 0, mat(ld=250)), (P, F32, 256, 0, mat(rows=1 << 31)),
              (P, F32, 256, 0, mat(cols=260, halves=1, lds=3)), (P, F32, 256, 0, None)):
        assert lib.mt_quant8(*a, 0) == BAD
    for a in ((P, F32, 64, mat(), 0, mat()), (0, F32, 64, None, 0, mat()), (P, F32, 63, None, 0, mat()),
              (P, F32, 64, None, 0, mat(halves=1)), (P, F32, 64, None, P, mat(batch=2)),
              (0, 0, 0, mat(rows=256, cols=64, halves=1), 0, mat()), (0, 0, 0, mat(rows=255, cols=64), 0, mat()),
              (0, 0, 0, mat(rows=256, cols=64, block_rows=128), 0, mat())):
        assert lib.mt_quant8_t(*a, 0) == BAD
    for a in ((mat(block_rows=128), 0, P, F32, 256), (mat(batch=2), 0, P, F32, 256), (mat(), 0, 0, F32, 256),
              (mat(), 0, P, F32, 255), (mat(), 0, P, 9, 256), (mat(), P + 2, P, F32, 256)):
        assert lib.mt_dequant8(*a, 0) == BAD
    assert lib.mt_quant8(P, F32, 256, 0, mat(block_rows=128, batch=65536), 0) == UNS


def test_gemm_refusals(lib):
    a, b = mat(100, 256), mat(300, 256)
    st = P
    for x in ((a, mat(300, 255), 0, 0, P, F32, 300, 0, st), (a, b, 0, 1, P, F32, 300, 0, st),
              (a, b, P, 0, P, F32, 300, 0, st), (a, b, P, 2, P, F32, 300, 0, st),
              (a, mat(300, 256, batch=2), 0, 0, P, F32, 300, 0, st), (mat(100, 256, block_rows=128), b, 0, 0, P, F32, 300, 0, st),
              (mat(100, 256, batch=2), b, 0, 0, P, F32, 300, 0, st), (a, b, 0, 0, P, BF16, 300, 1, st),
              (a, b, 0, 0, P, F32, 300, 2, st), (a, b, 0, 0, P, F32, 299, 0, st), (a, b, 0, 0, 0, F32, 300, 0, st),
              (a, b, 0, 0, P, F32, 300, 0, 0), (a, b, 0, 0, P, 5, 300, 0, st), (mat(100, 256, halves=1), b, 0, 0, P, F32, 300, 0, st),
              (a, b, P + 2, 1, P, F32, 300, 0, st)):
        assert lib.mt_gemm8(*x, 0) == BAD
    assert lib.mt_gemm8(a, mat(300, 256, batch=65), P, 65, P, F32, 300, 0, st, 0) == UNS
    assert lib.mt_gemm8(mat(0, 256), b, 0, 0, 0, F32, 300, 0, st, 0) == B.MT_OK
    for x in ((a, b, 0, 1, P, 300, 0, st), (a, b, P, 0, P, 300, 0, st), (a, mat(300, 256, block_rows=128, lds=2), P, 1, P, 300, 0, st),
              (a, mat(300, 128), P, 1, P, 300, 0, st), (a, b, P, 1, P, 299, 0, st), (a, b, P, 1, 0, 300, 0, st),
              (a, b, P, 1, P, 300, 0, 0)):
        assert lib.mt_gemm8_reduce(*x, 0) == BAD
    assert lib.mt_gemm8_reduce(a, b, P, 65, P, 300, 0, st, 0) == UNS


def test_swiglu_refusals(lib):
    act, sv = mat(10, 200), mat(10, 400, halves=1, lds=4)
    for x in ((0, F32, 400, 0, act, sv), (P, 4, 400, 0, act, sv), (P, F32, 399, 0, act, sv),
              (P, F32, 400, P + 2, act, sv), (P, F32, 400, 0, mat(10, 200, halves=1), sv),
              (P, F32, 400, 0, act, mat(10, 400)), (P, F32, 400, 0, act, mat(9, 400, halves=1)),
              (P, F32, 400, 0, act, mat(10, 200, halves=1)), (P, F32, 400, 0, None, sv)):
        assert lib.mt_swiglu8(*x, 0) == BAD
    assert lib.mt_swiglu8(0, F32, 400, 0, mat(0, 200), None, 0) == B.MT_OK
    for x in ((0, F32, 200, sv, 0, P, 400, 0, 0), (P, F32, 199, sv, 0, P, 400, 0, 0), (P, F32, 200, act, 0, P, 400, 0, 0),
              (P, F32, 200, sv, 0, 0, 400, 0, 0), (P, F32, 200, sv, 0, P, 399, 0, 0), (P, F32, 200, sv, 0, P, 400, P, 199),
              (P, F32, 200, sv, 0, P, 400, P + 1, 200), (P, 3, 200, sv, 0, P, 400, 0, 0)):
        assert lib.mt_swiglu8_bwd(*x, 0) == BAD


def test_wrappers_refuse_host_tensors():
    q, s = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.uint8)
    with pytest.raises(ValueError):
        ops.Tensor8(q, s, 128)
    with pytest.raises(TypeError):
        ops.Tensor8(q.float(), s, 128)
    with pytest.raises(ValueError):
        ops.empty8(4, 128, device="cpu")
    with pytest.raises(ValueError):
        ops.Route.of(torch.zeros(5, dtype=torch.int32), torch.zeros(512, dtype=torch.int32),
                     torch.zeros(4, 2, dtype=torch.int32))


def test_reference_quantiser_pins():
    """The tests' own e4m3: known codes, ties to even, torch's conversion."""
    assert R.TABLE[0x7E] == 448 and R.TABLE[0x08] == 2.0 ** -6 and R.TABLE[1] == 2.0 ** -9
    x = np.concatenate([np.random.default_rng(0).normal(size=4000) * 2.0 ** np.random.default_rng(1).integers(-12, 8, 4000),
                        [0.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, 448.0, -448.0]])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.e4m3_code(x.astype(np.float64)), want)
    assert [R.scale_exponent(a) for a in (0.0, 448.0, 448.0001, 1.75, 1.7500001, 1e-300)] == [0, 0, 1, -8, -7, -126]


def test_moves_of_no_tokens_need_no_rows(lib):
    """The row numbers of no assignments have no storage; the other two do."""
    r0 = lib.mt_route_rows(0, 2, 4)
    assert lib.mt_dispatch(0, F32, 8, 0, 8, 2, 4, P, P, 0, r0, P, 8, 0) == B.MT_OK
    assert lib.mt_dispatch8(0, F32, 8, 0, 2, 4, P, P, 0, mat(r0, 8), 0) == B.MT_OK
    assert lib.mt_combine_bwd(0, F32, 8, P, 8, P, P, 0, r0, 0, 0, 2, 4, 8, P, 8, 0, 0) == B.MT_OK
    assert lib.mt_dispatch(0, F32, 8, 0, 8, 2, 4, P, 0, 0, r0, P, 8, 0) == BAD
    assert lib.mt_dispatch(0, F32, 8, 0, 8, 2, 4, 0, P, 0, r0, P, 8, 0) == BAD


class OnDevice:
    """A host tensor that says it lies on cuda:0, for the arguments a wrapper passes on."""

    def __init__(self, t):
        self._t, self.device = t, torch.device("cuda", 0)

    def __getattr__(self, name):
        return getattr(self._t, name)

    def get_device(self):
        return 0


def described(monkeypatch, codes, scales, cols, **kw):
    """Tensor8's description of host buffers of these shapes."""
    monkeypatch.setattr(ops, "_status_word", lambda dev: P)
    return ops.Tensor8(OnDevice(torch.zeros(codes, dtype=torch.uint8)), OnDevice(torch.zeros(scales, dtype=torch.uint8)),
                       cols, **kw)


def test_empty_stacks_have_no_address(lib, monkeypatch):
    """A stack of no matrices has no storage: whatever takes or fills one is
    refused on the host, and no address stands in for it.  (A matrix of no rows
    is valid and nothing reads it.)"""
    rows = lib.mt_route_rows(4, 2, 4)
    a = described(monkeypatch, (0, 64, 256), (0, 64, 2), 256)
    b = described(monkeypatch, (0, 64, 256), (0, 1, 2), 256, block_rows=128)
    s = described(monkeypatch, (0, 64, 512), (0, 64, 4), 512, halves=True)
    x = described(monkeypatch, (0, rows, 16), (0, rows, 1), 8)
    for t in (a, b, s, x):
        assert t._mat.batch == 0 and not t._mat.codes and not t._mat.scales
    full, held = mat(), mat(64, 512, halves=1)
    for st in (lib.mt_gemm8(a._ref, full, 0, 0, P, F32, 64, 0, P, 0), lib.mt_gemm8(full, a._ref, 0, 0, P, F32, 64, 0, P, 0),
               lib.mt_gemm8(full, b._ref, 0, 0, P, F32, 64, 0, P, 0), lib.mt_gemm8(full, b._ref, P, 1, P, F32, 64, 0, P, 0),
               lib.mt_gemm8(full, b._ref, P, 0, P, F32, 64, 0, P, 0),
               lib.mt_gemm8_reduce(a._ref, full, P, 1, P, 64, 0, P, 0), lib.mt_gemm8_reduce(full, a._ref, P, 1, P, 64, 0, P, 0),
               lib.mt_quant8(P, F32, 256, 0, a._ref, 0), lib.mt_quant8(P, F32, 256, 0, b._ref, 0),
               lib.mt_quant8_t(0, 0, 0, a._ref, 0, mat(256, 64), 0), lib.mt_quant8_t(P, F32, 64, None, 0, a._ref, 0),
               lib.mt_dequant8(a._ref, 0, P, F32, 256, 0), lib.mt_swiglu8(P, F32, 512, 0, full, s._ref, 0),
               lib.mt_swiglu8(P, F32, 512, 0, a._ref, held, 0), lib.mt_swiglu8_bwd(P, F32, 256, s._ref, 0, P, 512, 0, 0, 0),
               lib.mt_dispatch8(P, F32, 8, 4, 2, 4, P, P, P, x._ref, 0)):
        assert st == BAD
    none = described(monkeypatch, (0, 256), (0, 2), 256)
    assert none._mat.batch == 1 and none._mat.codes and none._mat.scales
    assert lib.mt_gemm8(none._ref, full, 0, 0, 0, F32, 64, 0, P, 0) == B.MT_OK
    assert lib.mt_quant8(0, F32, 256, 0, none._ref, 0) == B.MT_OK


def test_status_words_are_made_once_by_any_number_of_threads(monkeypatch):
    """Threads that use a device for the first time together get the same
    status words: a second pair would leave the first address, which a launch
    may already have, to the allocator."""
    import threading
    made, inside = [], threading.Event()

    def zeros(*args, **kw):
        made.append(torch.empty(2, dtype=torch.int32))
        return made[-1]

    def synchronize(dev):                  # lets the other threads run, as the real one does
        inside.set()
        threading.Event().wait(0.2)

    monkeypatch.setattr(ops, "_status", {})
    monkeypatch.setattr(ops.torch, "zeros", zeros)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "synchronize", synchronize)
    got = []
    threads = [threading.Thread(target=lambda: got.append(ops._status_word(0))) for _ in range(4)]
    threads[0].start()
    assert inside.wait(10)
    for t in threads[1:]:
        t.start()
    for t in threads:
        t.join(10)
    assert len(made) == 1 and got == [made[0].data_ptr()] * 4


@pytest.mark.parametrize("rows,cols", [(1, 2), (7, 100), (130, 264), (257, 300)])
def test_reference_quantiser_on_tensors(rows, cols):
    """The vectorised definition gives the block by block one's codes, scales and values."""
    g = np.random.default_rng(rows)
    x = g.normal(size=(rows, cols)) * 2.0 ** g.integers(-140, 120, (rows, 1))
    x[0] = 0
    if rows > 5:
        x[1], x[2, ::2], x[3, 5], x[4, 7], x[5] = 448.0, 448.0 * (1 + 2.0 ** -40), np.nan, -np.inf, np.inf
    for kw in ({}, dict(block_rows=128), dict(halves=True)):
        want = R.quant(x, **kw)
        got = R.quant_t(torch.from_numpy(x), **kw)
        assert all(np.array_equal(a.numpy(), b) for a, b in zip(got, want))
        val = R.value_t(*got, cols, **kw)
        assert np.array_equal(val.numpy(), R.value(*want, cols, **kw), equal_nan=True)
