"""The 8-bit dense operators in 64 bits, from their definitions (numpy): e4m3 codes, power-of-two
scales per block, the residual norm, the block-scaled product and the gated product."""
from __future__ import annotations

import numpy as np


def e4m3_table() -> np.ndarray:
    """Value of each of the 256 codes (NaN for 0x7f and 0xff)."""
    t = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        a = np.nan if (e, m) == (15, 7) else (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
        t[c] = -a if c & 128 else a
    return t


TABLE = e4m3_table()
POSITIVE = TABLE[:127]  # codes 0 .. 126, increasing


def round_e4m3(v: np.ndarray) -> np.ndarray:
    """Nearest code of |v| <= 448, ties to the even code (the codes of one sign are consecutive, so a
    code's parity is its last mantissa bit); NaN -> 0x7f."""
    a = np.abs(v)
    hi = np.clip(np.searchsorted(POSITIVE, np.nan_to_num(a), side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = np.nan_to_num(a) - POSITIVE[lo], POSITIVE[hi] - np.nan_to_num(a)
    c = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    c = c | np.where(np.signbit(v), 128, 0)
    return np.where(np.isnan(v), 0x7F, c).astype(np.uint8)


def spread(s: np.ndarray, shape, block_rows: int) -> np.ndarray:
    """A block's value at each of its elements."""
    return s[np.arange(shape[0]) // block_rows][:, np.arange(shape[1]) // 128]


def block_max(v: np.ndarray, block_rows: int) -> np.ndarray:
    R, C = v.shape
    full = np.zeros((-(-R // block_rows) * block_rows, -(-C // 128) * 128))
    full[:R, :C] = np.abs(v)
    return full.reshape(full.shape[0] // block_rows, block_rows, -1, 128).max(axis=(1, 3))


def scale_bytes(amax: np.ndarray) -> np.ndarray:
    """127 + the smallest e with amax / 2^e <= 448 (clamped to >= 0); 127 for a block of zeros, 255
    where amax is not finite."""
    out = np.empty(amax.shape, np.int64)
    for i, a in np.ndenumerate(amax):
        if not np.isfinite(a):
            out[i] = 255
        elif a == 0:
            out[i] = 127
        else:
            m, x = np.frexp(a)  # a = m 2^x, m in [1/2, 1);  448 = 7/8 2^9
            out[i] = max(0, 127 + (x - 9 if m <= 0.875 else x - 8))
    return out.astype(np.uint8)


def scale_values(b: np.ndarray) -> np.ndarray:
    return np.where(b == 255, np.nan, np.exp2(b.astype(np.float64) - 127))


def quantize(v: np.ndarray, block_rows: int):
    """-> (codes uint8, scale bytes uint8)."""
    v = np.asarray(v, np.float64)
    b = scale_bytes(block_max(v, block_rows))
    with np.errstate(invalid="ignore"):
        return round_e4m3(v / spread(scale_values(b), v.shape, block_rows)), b


def values(codes: np.ndarray, b: np.ndarray, block_rows: int) -> np.ndarray:
    return TABLE[codes] * spread(scale_values(b), codes.shape, block_rows)


def rmsnorm(x, resid, w, eps):
    """-> (r, y)"""
    r = np.asarray(x, np.float64) + (0 if resid is None else np.asarray(resid, np.float64))
    with np.errstate(invalid="ignore"):
        return r, r / np.sqrt((r * r).mean(axis=1, keepdims=True) + eps) * np.asarray(w, np.float64)


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g))


def check_codes(codes, b, ref, err):
    """Codes and scale bytes of `ref` [T, n] known up to the absolute error `err` [T, n]: each scale is
    the reference's unless the block's maximum may lie on the other side of a border (448 2^e), and each
    value is within half a step of its code (2^-4 of the value, 2^-10 scales below the smallest normal)."""
    amax, slack = block_max(ref, 1), block_max(err, 1)
    lo, hi = scale_bytes(np.maximum(amax - slack, 0)), scale_bytes(amax + slack)
    lo = np.where(amax - slack <= 0, 0, lo)
    assert ((b >= np.minimum(lo, hi)) & (b <= np.maximum(lo, hi))).all()
    assert (b == scale_bytes(amax))[slack < 1e-6 * amax].mean() > 0.99 if (slack < 1e-6 * amax).any() else True
    s = spread(scale_values(b), ref.shape, 1)
    got = TABLE[codes] * s
    assert np.isfinite(got).all()
    tol = (np.abs(ref) + err) * 2.0 ** -4
    tol = np.maximum(tol, s * 2.0 ** -10) + err
    worst = np.abs(got - ref) - tol
    assert worst.max() <= 0, "off by %.3e more than half a step" % worst.max()
