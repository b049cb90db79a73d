"""fp64 statement of the paged key/value cache and of attention over it.

Plain NumPy, from the format and the formulas alone.  BF16 values are given
as bit patterns (uint16), E4M3 codes as bytes.
"""

from __future__ import annotations

import math

import numpy as np

from .oracle import decode_bf16

HEAD_DIM = 128


def e4m3_values() -> np.ndarray:
    """The 256 values of the format: sign, 4 exponent bits (bias 7), 3 bits of
    fraction; exponent 0 is subnormal, code 127 (and 255) NaN, no infinity."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m / 512.0 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        if c & 127 == 127:
            v = math.nan
        out[c] = -v if c & 128 else v
    return out


def quantise_row(bits: np.ndarray):
    """(codes uint8 [128], exponent byte) of one BF16 row, by definition."""
    x = decode_bf16(bits)
    if not np.all(np.isfinite(x)):  # the whole row is not a number
        return np.full(x.shape, 127, dtype=np.uint8), 255
    amax = float(np.abs(x).max())
    e = -126
    while amax > 448.0 * 2.0 ** e:
        e += 1
    vals = e4m3_values()[:127]  # the magnitudes, ascending with the code
    vals = vals[vals * 2.0 ** e <= 255 * 2.0 ** 120]  # that stand for a finite BF16 value
    codes = np.empty(x.shape, dtype=np.uint8)
    for i, v in enumerate(x):
        a = abs(v) * 2.0 ** -e
        hi = int(np.searchsorted(vals, a))  # vals[hi - 1] < a <= vals[hi]
        lo = max(hi - 1, 0)
        hi = min(hi, len(vals) - 1)
        dl, dh = a - vals[lo], vals[hi] - a
        c = lo if dl < dh or (dl == dh and lo % 2 == 0) else hi
        codes[i] = c | (128 if np.signbit(v) else 0)
    return codes, e + 127


def dequantise(codes: np.ndarray, exps: np.ndarray) -> np.ndarray:
    """Values of rows [..., 128] with exponent bytes [...]."""
    return e4m3_values()[codes] * 2.0 ** (exps.astype(np.float64) - 127)[..., None]


def positions(row_start, kv_len, s):
    """[(row, position)] of sequence s."""
    r0, r1 = int(row_start[s]), int(row_start[s + 1])
    return [(r, int(kv_len[s]) - (r1 - r0) + (r - r0)) for r in range(r0, r1)]


def visible(pos, length, causal, window):
    """[lo, hi) of the keys that the row at `pos` sees."""
    hi = min(length, pos + 1) if causal else length
    lo = max(0, pos + 1 - window) if window else 0
    return lo, max(lo, hi)


def gather(pages, table, s, n):
    """[n, H, 128] rows of sequence s's first n tokens (any array of pages)."""
    ps = pages.shape[2]
    j = np.arange(n)
    return pages[np.asarray(table)[s, j // ps], :, j % ps]


def paged_attention(q, k, v, pos, length, causal=True, window=0, scale=None):
    """One sequence, fp64: q [n, Hq, 128], k and v [>= visible, H, 128], pos [n].

    Returns o, lse, mass, reach: mass = sum p |v| / sum p and reach = the
    largest scale * sum |q_d k_d| of a visible key, for error bounds."""
    scale = 1 / math.sqrt(HEAD_DIM) if scale is None else scale
    n, hq, d = q.shape
    g = hq // k.shape[1]
    o, mass = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    lse, reach = np.full((n, hq), -np.inf), np.zeros((n, hq))
    for i in range(n):
        lo, hi = visible(int(pos[i]), length, causal, window)
        if hi <= lo:
            continue
        for h in range(hq):
            kk, vv = k[lo:hi, h // g], v[lo:hi, h // g]
            x = scale * (kk @ q[i, h])
            m = x.max()
            p = np.exp(x - m)
            o[i, h] = p @ vv / p.sum()
            mass[i, h] = p @ np.abs(vv) / p.sum()
            lse[i, h] = m + math.log(p.sum())
            reach[i, h] = abs(scale) * (np.abs(kk) @ np.abs(q[i, h])).max()
    return o, lse, mass, reach
