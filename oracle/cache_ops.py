"""Float64 oracle of what surrounds the attention's cache: rotary positions, caches written
as rows are produced, and attention over 8-bit rows with a scale per block of 64.

Written from the definitions, one row or pair at a time where that is clearest; shares no
code with the CUDA library.
"""
from __future__ import annotations

import math
from typing import Optional

import numpy as np

SCALE_BLOCK = 64
E4M3_MAX = 448.0
SCALE_EXP_MAX = 40


# ------------------------------------------------------------------ rotary positions

def rope_frequencies(dims: int, base: float = 10000.0, scaling: int = 0, factor: float = 1.0,
                     orig_len: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(radians per position of each pair, magnitude of the rotation)."""
    f, m = [], 1.0
    for i in range(dims // 2):
        w = base ** (-2.0 * i / dims)
        if scaling == 1:
            w = w / factor
        elif scaling == 2:
            w = (base * factor ** (dims / (dims - 2.0))) ** (-2.0 * i / dims)
        elif scaling == 3:
            def pair(turns):
                return dims * math.log(orig_len / (2 * math.pi * turns)) / (2 * math.log(base))
            low = min(max(math.floor(pair(beta_fast)), 0), dims - 1)
            high = min(max(math.ceil(pair(beta_slow)), 0), dims - 1)
            r = min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
            w = w / factor * r + w * (1 - r)
        f.append(w)
    if scaling == 3 and factor > 1:
        m = 0.1 * math.log(factor) + 1
    return np.array(f), m


def rope(x: np.ndarray, positions: np.ndarray, dims: int, offset: int = 0, layout: int = 0,
         transpose: bool = False, mscale: float = 0.0, **freq) -> np.ndarray:
    """x [n, heads, head_dim] with dims [offset, offset + dims) of each head turned."""
    f, m = rope_frequencies(dims, **freq)
    if mscale > 0:
        m = mscale
    y = np.array(x, dtype=np.float64)
    for i in range(dims // 2):
        a, b = (offset + 2 * i, offset + 2 * i + 1) if layout == 0 else (offset + i, offset + i + dims // 2)
        t = np.asarray(positions, dtype=np.float64) * f[i]
        c, s = np.cos(t)[:, None], np.sin(t)[:, None] * (-1 if transpose else 1)
        u, v = np.asarray(x[..., a], np.float64), np.asarray(x[..., b], np.float64)
        y[..., a], y[..., b] = m * (u * c - v * s), m * (u * s + v * c)
    return y


# ------------------------------------------------------------------ e4m3 with a scale per block

def e4m3_table() -> np.ndarray:
    """The value of every e4m3 code (sign, four exponent bits, three mantissa bits)."""
    v = np.empty(256)
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        mag = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if code & 127 == 127:
            mag = np.nan
        v[code] = -mag if code & 128 else mag
    return v


def e4m3_round(x: np.ndarray) -> np.ndarray:
    """x to the nearest e4m3 value, ties to the even mantissa, saturating at 448."""
    x = np.asarray(x, dtype=np.float64)
    mag = np.minimum(np.abs(x), E4M3_MAX)
    _, e = np.frexp(np.where(np.isnan(mag), 0.0, mag))
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.copysign(np.rint(mag / step) * step, x)


def scale_exponent(x: np.ndarray) -> int:
    """The smallest e in [-40, 40] with max|x| <= 448 * 2^e over the finite values."""
    x = np.asarray(x, dtype=np.float64)
    top = np.abs(x[np.isfinite(x)]).max(initial=0.0)
    for e in range(-SCALE_EXP_MAX, SCALE_EXP_MAX):
        if top <= E4M3_MAX * 2.0 ** e:
            return e
    return SCALE_EXP_MAX


class BlockCache:
    """A kv_format 5 cache: stored values and the blocks' exponents, by row."""

    def __init__(self, rows: int, dims: int):
        blocks = (rows + SCALE_BLOCK - 1) // SCALE_BLOCK
        self.codes = np.zeros((blocks * SCALE_BLOCK, dims))      # as the values of their codes
        self.exp = np.zeros(blocks, dtype=np.int64)

    def write(self, row0: int, x: np.ndarray) -> None:
        x = np.asarray(x, dtype=np.float64)
        at = row0
        while at < row0 + len(x):
            b = at // SCALE_BLOCK
            first, end = b * SCALE_BLOCK, min((b + 1) * SCALE_BLOCK, row0 + len(x))
            new = x[at - row0:end - row0]
            e = scale_exponent(new)
            if at > first:                                       # rows from before
                if self.exp[b] >= e:
                    e = int(self.exp[b])
                else:
                    self.codes[first:at] = e4m3_round(self.codes[first:at] * 2.0 ** (int(self.exp[b]) - e))
            self.exp[b] = e
            self.codes[at:end] = e4m3_round(new / 2.0 ** e)
            at = end

    def read(self, rows) -> np.ndarray:
        rows = np.asarray(rows)
        return self.codes[rows] * (2.0 ** self.exp[rows // SCALE_BLOCK].astype(np.float64))[:, None]


def stored_bytes(codes: np.ndarray, exp: np.ndarray) -> np.ndarray:
    """The library's bytes of a BlockCache whose rows were all written (no NaN): 64 rows of
    codes, then the record of the block (its scale as fp32, zeros)."""
    table = e4m3_table()
    mags = table[:127]
    code = np.searchsorted(mags, np.abs(codes)).astype(np.uint8) | (np.signbit(codes).astype(np.uint8) << 7)
    blocks, dims = len(exp), codes.shape[1]
    out = np.zeros((blocks, SCALE_BLOCK + 1, dims), np.uint8)
    out[:, :SCALE_BLOCK] = code.reshape(blocks, SCALE_BLOCK, dims)
    out[:, SCALE_BLOCK, :4] = (2.0 ** exp.astype(np.float64)).astype(np.float32).view(np.uint8).reshape(blocks, 4)
    return out.reshape(-1)


# ------------------------------------------------------------------ attention

def attention_rows(q_t: np.ndarray, rows: np.ndarray, scale: Optional[float] = None, d_v: int = 512,
                   absolute: bool = False) -> np.ndarray:
    """One token's heads q_t [16, 576] over rows [n, 576]: softmax(scale q . row) @ row[:512]
    (absolute: @ |row[:512]|, the size that rounding errors are measured against)."""
    rows = np.asarray(rows, dtype=np.float64)
    z = np.asarray(q_t, dtype=np.float64) @ rows.T * (1 / 24.0 if scale is None else scale)
    p = np.exp(z - z.max(1, keepdims=True))
    v = np.abs(rows[:, :d_v]) if absolute else rows[:, :d_v]
    return (p / p.sum(1, keepdims=True)) @ v


def attended(raw: np.ndarray, cmp: np.ndarray, topk: Optional[np.ndarray], t0: int, i: int, n_swa: int) -> np.ndarray:
    """What token t0 + i attends of per-row arrays: its selected compressed rows (topk[i], -1
    dropped), then its window of raw rows."""
    t = t0 + i
    parts = [raw[max(0, t - n_swa + 1):t + 1]]
    if topk is not None and topk.shape[1]:
        parts.insert(0, cmp[topk[i][topk[i] >= 0]])
    return np.concatenate(parts)
