"""The 8-bit K/V cache and the choice of its blocks, restated plainly: codes,
steps and spans in IEEE float32 step by step (every rounding written out), so
that they can be compared bit for bit; attention is float64 (``kv4.attention``).
Test infrastructure only.
"""
from __future__ import annotations

import numpy as np

F = np.float32
T_BLOCK = 64


def steps(x: np.ndarray):
    """Step float32 of a block's rows [64, d]: fl(max |x| / 127), 1 where that
    is 0."""
    s = F(np.max(np.abs(x.astype(F)))) / F(127)
    return F(1) if s == 0 else F(s)


def codes(x: np.ndarray, step):
    """clamp(rint(fl(x / step)), -127, 127), 0 for a NaN; int array."""
    with np.errstate(invalid="ignore", over="ignore"):
        c = np.rint((x.astype(F) / F(step)).astype(F))
    return np.clip(np.nan_to_num(c, nan=0.0), -127, 127).astype(np.int64)


def stands_for(c, step):
    """fl(code step), float32."""
    with np.errstate(invalid="ignore"):
        return (c.astype(F) * F(step)).astype(F)


def key_place(t: int, c: int, d: int) -> int:
    """Where a block of K8 holds token t, channel c."""
    j, g, h = t % 16 // 2, t // 16 * 2 + t % 2, c // 64
    return ((j * (d // 64) + h) * 8 + g) * 64 + c % 64


def key_places(d: int) -> np.ndarray:
    return np.array([[key_place(t, c, d) for c in range(d)] for t in range(T_BLOCK)])


def block(K: np.ndarray, V: np.ndarray):
    """K8 [64 d], V8 [d, 64], scale [2], span [2, d] of rows [64, d]."""
    d = K.shape[1]
    sk, sv = steps(K), steps(V)
    ck, cv = codes(K, sk), codes(V, sv)
    k8 = np.zeros(T_BLOCK * d, np.uint8)
    k8[key_places(d)] = ck + 128
    span = np.stack([ck.max(0), ck.min(0)]) + 128
    return k8, (cv.T + 128).astype(np.uint8), np.array([sk, sv], F), span.astype(np.uint8)


def scores(q: np.ndarray, span: np.ndarray, step: np.ndarray) -> np.ndarray:
    """Scores float32 [blocks] of a token's query heads q [G, d] against spans
    [blocks, 2, d] (uint8) and the keys' steps [blocks]; a NaN is +infinity."""
    out = np.full(span.shape[0], -np.inf, F)
    ends = span.astype(np.int64) - 128
    nan = np.zeros(span.shape[0], bool)
    for x in q.astype(F):
        sh = steps(x[None])
        c = codes(x, sh)
        dots = np.where(c >= 0, c * ends[:, 0], c * ends[:, 1]).sum(1)
        with np.errstate(over="ignore", invalid="ignore"):
            s = ((dots.astype(F) * step.astype(F)).astype(F) * sh).astype(F)
        nan |= np.isnan(s)
        out = np.maximum(out, s)
    out[nan] = np.inf
    return out


def choose(score: np.ndarray, own: int, n_sel: int, n_first: int, n_last: int):
    """The blocks chosen of 0 .. own, ascending; score [own + 1]."""
    if own + 1 <= n_sel:
        return list(range(own + 1))
    kept = set(range(n_first)) | set(range(own + 1 - n_last, own + 1))
    for j in sorted(range(own + 1), key=lambda j: (-float(score[j]), j)):
        if len(kept) == n_sel:
            break
        kept.add(j)
    return sorted(kept)
