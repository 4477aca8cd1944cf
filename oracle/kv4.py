"""The operators around the decode step, restated plainly: per-head norms
with position rotation, the 4-bit K/V cache, and attention over it.

The pages hold keys in 4-bit codes per block and channel (picx.dev summary,
"Algorithm Components" 4: the KIVI scheme); the scheme codes values per
token.  Codes are IEEE float32 step by step (every rounding written out), so
they can be compared bit for bit; norms, angles and attention are float64.
Test infrastructure only.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

F = np.float32
T_BLOCK = 64
# pi to 60 decimal places
PI = Fraction(3141592653589793238462643383279502884197169399375105820974944,
              10 ** 60)


def quantize_values(V: np.ndarray):
    """Codes uint8 [n, d], m and Delta float32 [n] of value rows [n, d]: per
    token, m = min, Delta = fl((max - min) / 15), code = clamp(rint(fl(fl(v -
    m) / Delta)), 0, 15), 0 where Delta = 0."""
    V = np.asarray(V, np.float32)
    m = V.min(axis=1)
    dl = ((V.max(axis=1) - m).astype(F) / F(15)).astype(F)
    x = (V - m[:, None]).astype(F)
    with np.errstate(invalid="ignore", divide="ignore"):
        c = np.where(dl[:, None] == 0, F(0), np.rint((x / dl[:, None]).astype(F)))
    return np.clip(c, 0, 15).astype(np.uint8), m, dl


def v4_place(t: int) -> int:
    """Nibble of token t = 32 i + 16 u + 8 v + 2 w + e in a V4 row."""
    i, u, v, w, e = t >> 5, (t >> 4) & 1, (t >> 3) & 1, (t >> 1) & 3, t & 1
    return 16 * w + 8 * i + 4 * e + 2 * u + v


def pack_values(codes: np.ndarray) -> np.ndarray:
    """V4 rows [d, 32] of one block's codes [64, d]."""
    out = np.zeros((codes.shape[1], T_BLOCK // 2), np.uint8)
    for t in range(T_BLOCK):
        p = v4_place(t)
        out[:, p // 2] |= codes[t] << (4 * (p & 1))
    return out


def stands_for(codes, m, dl):
    """fl(fl(code Delta) + m), float32."""
    return ((codes.astype(F) * dl).astype(F) + m).astype(F)


def rotation(pos: int, inv_freq) -> tuple:
    """cos and sin (float64) of pos * inv_freq, reduced exactly."""
    cs, sn = [], []
    for f in inv_freq:
        a = Fraction(float(f)) * pos
        a -= 2 * PI * round(a / (2 * PI))
        cs.append(np.cos(float(a)))
        sn.append(np.sin(float(a)))
    return np.array(cs), np.array(sn)


def norm_rope(x, w, eps, pos, inv_freq, interleaved):
    """One row x [d] (float64): norm with weights w (None: no norm), then
    the rotation of the first 2 len(inv_freq) channels at position pos."""
    x = np.asarray(x, np.float64)
    if w is not None:
        x = x / np.sqrt(np.mean(x * x) + eps) * np.asarray(w, np.float64)
    x = x.copy()
    n = len(inv_freq)
    if n:
        cs, sn = rotation(pos, inv_freq)
        ia = np.arange(n) * 2 if interleaved else np.arange(n)
        ib = ia + 1 if interleaved else ia + n
        a, b = x[ia].copy(), x[ib].copy()
        x[ia], x[ib] = a * cs - b * sn, a * sn + b * cs
    return x


def attention(q, K, V, seen):
    """softmax(q K^T / sqrt d) V of one row over the first `seen` rows
    (float64), and ln sum exp of its scores; 0 and -inf over none."""
    d = K.shape[1]
    if seen <= 0:
        return np.zeros(d), -np.inf
    s = K[:seen].astype(np.float64) @ np.asarray(q, np.float64) / np.sqrt(d)
    c = s.max()
    p = np.exp(s - c)
    return p @ V[:seen].astype(np.float64) / p.sum(), c + np.log(p.sum())
