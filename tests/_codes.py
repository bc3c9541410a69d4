"""The 8-bit code formats in plain NumPy: the reference of the blockwise quantizer's tests.

`quantize` repeats the definition's fp32 operations (a / Q, Q / a and the product, each rounded to
nearest, which float32 arrays do), so its codes and scales are the kernels' bit for bit.
`e4m3` values are built from the format: 1 sign, 4 exponent bits (bias 7), 3 fraction bits, no
infinities, 0x7f the NaN, largest finite value 448."""
import numpy as np

TOP = {"int8": 127.0, "e4m3": 448.0}
ZERO_BLOCK = np.float32(2.0 ** -100)


def _e4m3_table():
    t = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        if c & 127 == 127:
            v = np.nan
        t[c] = -v if c & 128 else v
    return t


E4M3 = _e4m3_table()
_POS = E4M3[:127]                                   # the non-negative codes, ascending


def round_e4m3(t):
    """Codes (uint8) of the nearest e4m3 value, ties to the even code, saturating; NaN keeps 0x7f."""
    t = np.asarray(t, dtype=np.float64)
    m = np.minimum(np.abs(np.where(np.isnan(t), 0.0, t)), 448.0)
    hi = np.clip(np.searchsorted(_POS, m), 0, 126)  # first code with value >= m
    lo = np.maximum(hi - 1, 0)
    dh, dl = _POS[hi] - m, m - _POS[lo]
    code = np.where(dh < dl, hi, np.where(dl < dh, lo, np.where(hi % 2 == 0, hi, lo)))
    code = np.where(m == _POS[hi], hi, code).astype(np.uint8)
    code = np.where(np.signbit(t), code | 128, code).astype(np.uint8)
    return np.where(np.isnan(t), np.uint8(0x7F), code)


def _spread(s, brows, bcols, shape):
    return np.repeat(np.repeat(s, brows, 0), bcols, 1)[: shape[0], : shape[1]]


def quantize(v, brows, bcols, code):
    """(codes, scales) of the float32 matrix v: int8 values, or the e4m3 codes as uint8."""
    v = np.asarray(v, dtype=np.float32)
    r, c = v.shape
    pr, pc = -(-r // brows) * brows, -(-c // bcols) * bcols
    pad = np.zeros((pr, pc), np.float32)
    pad[:r, :c] = v
    a = np.abs(pad).reshape(pr // brows, brows, pc // bcols, bcols).max(axis=(1, 3))   # NaN stays
    top = np.float32(TOP[code])
    with np.errstate(all="ignore"):
        live = a >= ZERO_BLOCK
        scale = np.where(a < ZERO_BLOCK, np.float32(0), a / top).astype(np.float32)
        factor = np.where(live, top / np.where(live, a, np.float32(1)), np.float32(0)).astype(np.float32)
        t = (v * _spread(factor, brows, bcols, v.shape)).astype(np.float32)
    if code == "int8":
        return np.clip(np.rint(np.where(np.isnan(t), 0, t)), -127, 127).astype(np.int8), scale
    return round_e4m3(t), scale


def decode(q, scale, brows, bcols, code):
    """The values in 64 bits, code * scale."""
    v = q.astype(np.float64) if code == "int8" else E4M3[q.view(np.uint8)]
    with np.errstate(all="ignore"):
        return v * _spread(scale.astype(np.float64), brows, bcols, q.shape)


def to_numpy(q):
    """A tensor of codes as int8 values or e4m3 codes (uint8)."""
    import torch
    return q.cpu().numpy() if q.dtype == torch.int8 else q.view(torch.uint8).cpu().numpy()


def check_error(v64, q, scale, brows, bcols, code, what=""):
    """The decoded values against what was quantized: off by at most half a step (int8: s / 2;
    e4m3: 2^-4 of the value, or 2^-10 steps of s below the normal range), with three fp32
    roundings (a / Q, Q / a, the product: 4 x 2^-24 of the value, rounded up) on top."""
    got = decode(q, scale, brows, bcols, code)
    s = _spread(scale.astype(np.float64), brows, bcols, v64.shape)
    half = s / 2 if code == "int8" else np.maximum(np.abs(v64) * 2.0 ** -4, s * 2.0 ** -10)
    bad = np.abs(got - v64) > half * (1 + 2.0 ** -20) + 4 * 2.0 ** -24 * np.abs(v64) + 2.0 ** -100
    assert not bad.any(), f"{what}: {int(bad.sum())} values off by more than half a step"
