"""The expert operators' definitions in float64 NumPy / torch on the host, for
the tests: written from the formulas, sharing nothing with the package."""
import numpy as np
import torch

BLOCK = 128


def as64(t):
    return t.detach().cpu().double().numpy()


def rows_max(n_tokens, top_k, n_experts):
    return -(-(n_tokens * top_k + n_experts * 127) // 128) * 128


def order(idx, n_experts):
    """(offs, perm, row) of a stable sort by expert with segments padded to 128 rows."""
    idx = np.asarray(idx)
    flat = idx.reshape(-1)
    rows = rows_max(idx.shape[0], idx.shape[1], n_experts)
    offs = np.zeros(n_experts + 1, np.int64)
    perm = np.full(rows, -1, np.int64)
    row = np.full(flat.size, -1, np.int64)
    for e in range(n_experts):
        at = np.nonzero(flat == e)[0]
        perm[offs[e]:offs[e] + at.size] = at
        row[at] = offs[e] + np.arange(at.size)
        offs[e + 1] = offs[e] + -(-at.size // 128) * 128
    return offs, perm, row.reshape(idx.shape)


def scale_exponent(amax):
    """Least e >= -126 with amax <= 448 * 2^e, 0 for amax = 0 (one number)."""
    if amax == 0:
        return 0
    e = -126
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def e4m3_table():
    v = np.empty(256)
    for b in range(256):
        ex, m = (b >> 3) & 15, b & 7
        x = (8 + m) * 2.0 ** (ex - 10) if ex else m * 2.0 ** -9
        v[b] = np.nan if (b & 127) == 127 else -x if b & 128 else x
    return v


TABLE = e4m3_table()
_POS = TABLE[:127]                       # ascending codes 0..126


def e4m3_code(x):
    """Nearest e4m3 code of each element (ties to even, |x| <= 448; NaN -> 127)."""
    a = np.abs(x)
    hi = np.clip(np.searchsorted(_POS, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    c = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    c = np.where(a == _POS[hi], hi, c)
    return np.where(np.isnan(x), 127, c | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def _quant_block(b):
    fin = np.isfinite(b)
    e = scale_exponent(np.max(np.abs(b[fin]), initial=0.0))
    return e4m3_code(np.where(fin, b, np.nan) * 2.0 ** -e), e + 127


def quant(x, block_rows=1, halves=False):
    """(codes [R, C], scale bytes) of float64 x [R, C]."""
    rows, cols = x.shape
    codes = np.empty((rows, cols), np.uint8)
    parts = [(0, cols // 2), (cols // 2, cols)] if halves else [(0, cols)]
    spans = [(c, min(c + BLOCK, hi)) for lo, hi in parts for c in range(lo, hi, BLOCK)]
    scales = np.empty((-(-rows // block_rows), len(spans)), np.uint8)
    for i in range(scales.shape[0]):
        for j, (lo, hi) in enumerate(spans):
            s = np.s_[i * block_rows:(i + 1) * block_rows, lo:hi]
            codes[s], scales[i, j] = _quant_block(x[s])
    return codes, scales


def value(codes, scales, cols, block_rows=1, halves=False):
    """float64 values of codes [R, >= cols] with scale bytes."""
    v = TABLE[codes[:, :cols]]
    r = np.arange(codes.shape[0]) // block_rows
    c = np.arange(cols)
    blk = np.where(c < cols // 2, c // BLOCK, -(-(cols // 2) // BLOCK) + (c - cols // 2) // BLOCK) if halves else c // BLOCK
    return v * 2.0 ** (scales[r][:, blk].astype(np.float64) - 127)


def value8(t):
    """float64 values of a Tensor8 matrix or stack."""
    q, s = t.codes.cpu().numpy(), t.scales.cpu().numpy()
    if q.ndim == 3:
        return np.stack([value(a, b, t.cols, t.block_rows, t.halves) for a, b in zip(q, s)])
    return value(q, s, t.cols, t.block_rows, t.halves)


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def rounded(x, dtype):
    """float64 -> dtype -> float64 through torch (one rounding)."""
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).double().numpy()


def power_t(e):
    """2^e as float64, exactly, for whole e (a device's pow is not exact)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def quant_t(x, block_rows=1, halves=False):
    """:func:`quant` on a float64 tensor where it lies, for sizes that take the loop above too long."""
    rows, cols = x.shape
    if halves:
        parts = [quant_t(p) for p in x.split(cols // 2, 1)]
        return tuple(torch.cat(p, 1) for p in zip(*parts))
    b = torch.nn.functional.pad(x, (0, -cols % BLOCK, 0, -rows % block_rows))
    b = b.unflatten(1, (-1, BLOCK)).unflatten(0, (-1, block_rows))
    top = torch.where(torch.isfinite(b), b.abs(), 0.0).amax((1, 3))
    m, ex = torch.frexp(top)                     # 448 = 0.875 * 2^9
    e = torch.where(top > 0, (ex - 9 + (m > 0.875).int()).clamp(min=-126), 0)
    v = b * power_t(-e)[:, None, :, None]
    v = v.flatten(2).flatten(0, 1)[:rows, :cols]
    pos = torch.from_numpy(_POS).to(x.device)
    a = v.abs().nan_to_num(0.0, 0.0).contiguous()
    hi = torch.searchsorted(pos, a).clamp(0, 126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - pos[lo], pos[hi] - a
    c = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    c = torch.where(a == pos[hi], hi, c) + 128 * torch.signbit(v).int()
    return torch.where(torch.isfinite(v), c, 127).to(torch.uint8), (e + 127).to(torch.uint8)


def value_t(codes, scales, cols, block_rows=1, halves=False):
    """:func:`value` on tensors where they lie."""
    v = torch.from_numpy(TABLE).to(codes.device)[codes[:, :cols].long()]
    r = torch.arange(codes.shape[0], device=codes.device) // block_rows
    c = torch.arange(cols, device=codes.device)
    nb = -(-(cols // 2) // BLOCK)
    blk = torch.where(c < cols // 2, c // BLOCK, nb + (c - cols // 2) // BLOCK) if halves else c // BLOCK
    return v * power_t(scales[r][:, blk].long() - 127)
