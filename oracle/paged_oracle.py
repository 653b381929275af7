"""Float64 restatement of the paged K+V cache operators (test infrastructure only).

Plain loops over sequences, pages and heads: rotation, the e4m3 grid with one
power-of-two scale per page and head, and softmax attention. Nothing here is
shared with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

EXP_MIN, EXP_MAX = -100, 120


def e4m3_table() -> np.ndarray:
    """Value of each code: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f and 0xff are NaN."""
    out = np.empty(256)
    for i in range(256):
        e, m = (i >> 3) & 15, i & 7
        v = math.nan if (e, m) == (15, 7) else m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[i] = -v if i & 128 else v
    return out


def round_e4m3(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value, ties to even, for |x| <= 448."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(np.abs(x)))
    step = np.exp2(np.maximum(e, -6.0) - 3.0)
    return np.round(x / step) * step  # np.round: ties to even


def needed_scale(amax: float) -> float:
    """Least 2^e, EXP_MIN <= e <= EXP_MAX, with amax <= 448·2^e."""
    e = EXP_MIN
    while e < EXP_MAX and amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def rotate(x: np.ndarray, cos: np.ndarray, sin: np.ndarray, interleaved: bool) -> np.ndarray:
    """x [..., dh] at one position; cos, sin [rot/2]."""
    y = np.array(x, dtype=np.float64)
    half = len(cos)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        y[..., a] = x[..., a] * cos[i] - x[..., b] * sin[i]
        y[..., b] = x[..., b] * cos[i] + x[..., a] * sin[i]
    return y


class Pages:
    """One pool: values [num_pages][Hkv][page][dh]; for e4m3 the values they stand for, and scale [num_pages][Hkv]."""

    def __init__(self, values, scale=None):
        self.values = np.array(values, dtype=np.float64)
        self.scale = None if scale is None else np.array(scale, dtype=np.float64)

    def write(self, rows, table, len0):
        """rows [n][Hkv][dh] to positions len0.. of the sequence whose pages are table."""
        page = self.values.shape[2]
        n = len(rows)
        for slot in range(len0 // page, (len0 + n - 1) // page + 1) if n else ():
            lo, hi = max(0, len0 - slot * page), min(page, len0 + n - slot * page)
            new = np.asarray(rows[slot * page + lo - len0: slot * page + hi - len0], dtype=np.float64)
            pid = table[slot]
            for h in range(self.values.shape[1]):
                x = new[:, h]
                if self.scale is None:
                    self.values[pid, h, lo:hi] = x
                    continue
                s = needed_scale(np.abs(x).max())
                if lo > 0:
                    s = max(s, self.scale[pid, h])
                    self.values[pid, h, :lo] = round_e4m3(self.values[pid, h, :lo] / s) * s
                top = 240.0 if s == 2.0 ** EXP_MAX else 448.0  # 256·2^120 is past fp32 and bf16
                self.values[pid, h, lo:hi] = round_e4m3(np.clip(x / s, -top, top)) * s
                self.scale[pid, h] = s

    def read(self, table, n):
        """Rows 0..n-1 of a sequence, [n][Hkv][dh]."""
        page = self.values.shape[2]
        if n == 0:
            return np.zeros((0,) + self.values.shape[1:2] + self.values.shape[3:])
        x = np.concatenate([self.values[table[i]].transpose(1, 0, 2) for i in range((n + page - 1) // page)])
        return x[:n]


def attend(q, K, V, last):
    """q [n][Hq][dh], K, V [T][Hkv][dh]; row j attends keys 0..last[j]. Returns (out, A, spread): the
    output, the same sum over |V|, and the largest Σ_c |q_c K_tc| / sqrt(dh) of each row and head, which
    error bounds are built from."""
    n, Hq, dh = q.shape
    G = Hq // K.shape[1]
    out, A, spread = np.zeros((n, Hq, dh)), np.zeros((n, Hq, dh)), np.zeros((n, Hq, 1))
    for j in range(n):
        T = last[j] + 1
        if T <= 0:
            continue
        for i in range(Hq):
            k, v = K[:T, i // G], V[:T, i // G]
            z = k @ q[j, i] / math.sqrt(dh)
            p = np.exp(z - z.max())
            p /= p.sum()
            out[j, i] = p @ v
            A[j, i] = p @ np.abs(v)
            spread[j, i] = (np.abs(k) @ np.abs(q[j, i])).max() / math.sqrt(dh)
    return out, A, spread
