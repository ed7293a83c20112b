"""fp64 oracle of the microscaled formats (numpy): blocks of 32 channels with one
power-of-two scale, elements in int8 (m / 64), e4m3 or e2m1.

TEST INFRASTRUCTURE ONLY, as the rest of this directory.  Elements are found in
a table of the format's values, nearest first, a tie going to the even code;
the scale by trying exponents from the bottom.  Neither shares a formula with
the CUDA library.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32


def _minifloat(exp_bits: int, man_bits: int, bias: int, count: int) -> np.ndarray:
    """Values of codes 0 .. count - 1 (sign bit clear) of a small float type."""
    out = []
    for c in range(count):
        e, m = c >> man_bits, c & ((1 << man_bits) - 1)
        out.append(m * 2.0 ** (1 - bias - man_bits) if e == 0 else (1 + m / (1 << man_bits)) * 2.0 ** (e - bias))
    return np.array(out)


# magnitudes by code: 127 / 64 is the largest int8 element, 448 e4m3's, 6 e2m1's
TABLE = {
    "int8": np.arange(128) / 64.0,
    "e4m3": _minifloat(4, 3, 7, 127),  # code 127 is NaN
    "e2m1": _minifloat(2, 1, 1, 8),
}


def pitch(C: int) -> int:
    return -(-(-(-C // BLOCK)) // 4) * 4


def _blocks(x):
    C = x.shape[-1]
    pad = -C % BLOCK
    x = np.concatenate([x, np.zeros(x.shape[:-1] + (pad,))], -1)
    return x.reshape(x.shape[:-1] + (-1, BLOCK))


def scale_bytes(x, fmt: str) -> np.ndarray:
    """Scale byte of every block of [..., C] float64 values."""
    amax = np.abs(_blocks(np.asarray(x, np.float64))).max(-1)
    top = TABLE[fmt][-1]
    with np.errstate(invalid="ignore"):
        S = np.full(amax.shape, 254)
        for s in range(253, -1, -1):
            S = np.where(amax <= top * 2.0 ** (s - 127), s, S)
    return np.where(np.isfinite(amax), S, 255)


def elements(q, fmt: str):
    """(magnitude code, sign) of the element nearest to each q, ties to even."""
    tab = TABLE[fmt]
    a = np.abs(q)
    hi = np.clip(np.searchsorted(tab, a), 1, len(tab) - 1)
    lo = hi - 1
    dl, dh = a - tab[lo], tab[hi] - a
    return np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi))), np.signbit(q)


def pack(x, fmt: str):
    """(codes, scales) uint8 in the library's layout, of [..., C] float64 values."""
    x = np.asarray(x, np.float64)
    C = x.shape[-1]
    S = scale_bytes(x, fmt)
    bad = S == 255
    with np.errstate(invalid="ignore"):
        q = np.where(bad[..., None], 0.0, _blocks(x)) * 2.0 ** (127.0 - S)[..., None]
    code, neg = elements(q, fmt)
    code, neg = (v.reshape(x.shape[:-1] + (-1,))[..., :C] for v in (code, neg & ~bad[..., None]))
    if fmt == "int8":
        codes = np.where(neg, -code, code).astype(np.int8).view(np.uint8)
    elif fmt == "e4m3":
        codes = (code + 128 * neg).astype(np.uint8)
    else:
        c = (code + 8 * neg).astype(np.uint8)
        codes = c[..., 0::2] | (c[..., 1::2] << 4)
    scales = np.zeros(x.shape[:-1] + (pitch(C),), np.uint8)
    scales[..., :S.shape[-1]] = S
    return codes, scales


def unpack(codes, scales, fmt: str) -> np.ndarray:
    """float64 values of codes and scales."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    if fmt == "int8":
        v = codes.view(np.int8) / 64.0
    else:
        if fmt == "e2m1":
            codes = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (-1,))
        half = 8 if fmt == "e2m1" else 128
        tab = np.concatenate([TABLE[fmt], [np.nan]])[:half] if fmt == "e4m3" else TABLE[fmt]
        v = np.where(codes >= half, -1.0, 1.0) * tab[codes % half]
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return v * np.repeat(s, BLOCK, -1)[..., :v.shape[-1]]
