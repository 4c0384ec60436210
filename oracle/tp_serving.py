"""fp64 CPU oracle of the attention path around an 8-bit cache and drafted
trees: norms and rotation of queries and keys (with gradients), quantised cache
rows, and attention under a mask among the new tokens.

TEST INFRASTRUCTURE ONLY, under the same rules as ``tp_oracle``: only the tests
and the package's ``smoke()`` entry may import it; no CUDA code imports or links
it.

Readings.  The pages name neither norms of queries and keys nor a rotation nor
an 8-bit cache; the definitions are the plainest standard ones, written out at
each function.  Heads shard as in ``tp_attention`` (whole heads and their cache
rows per shard), so nothing here depends on the degree.

Pinned by tests/test_oracle_serving.py against pure-Python brute force, central
differences, and ``tp_attention`` where the two overlap.
"""
from __future__ import annotations

import math
from typing import Dict, Optional, Sequence, Tuple

import numpy as np

from .tp_oracle import E4M3_TABLE, ArrayLike, to_f64


def _pairs(rot: int, layout: str) -> Tuple[np.ndarray, np.ndarray]:
    """Positions in a head of the first and second member of every rotated pair."""
    i = np.arange(rot // 2)
    return (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)


def _turn(y: np.ndarray, angle: Optional[np.ndarray], layout: str) -> np.ndarray:
    """Pairs of y [T, heads, d] turned by angle [T, rot / 2]."""
    if angle is None:
        return y
    a, b = _pairs(2 * angle.shape[1], layout)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    out = y.copy()
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., a] * s + y[..., b] * c
    return out


def _angles(positions: Sequence[int], inv_freq) -> Optional[np.ndarray]:
    if inv_freq is None or len(inv_freq) == 0:
        return None
    f = np.asarray(inv_freq, dtype=np.float32).astype(np.float64)
    return np.asarray(positions, dtype=np.float64)[:, None] * f


def qk_norm_rope(qkv: ArrayLike, nq: int, nkv: int, d: int, gamma_q, gamma_k, inv_freq,
                 positions: Sequence[int], layout: str = "half", eps: float = 1e-5) -> np.ndarray:
    """Every query and key head x of a token: z = gamma x / sqrt(mean x^2 + eps)
    (z = x without gains), then pair p of z turned by position * inv_freq[p]."""
    x = to_f64(qkv).reshape(-1, nq + 2 * nkv, d)
    out = x.copy()
    qk = x[:, :nq + nkv]
    if gamma_q is not None:
        gain = np.concatenate([np.tile(to_f64(gamma_q), (nq, 1)), np.tile(to_f64(gamma_k), (nkv, 1))])
        qk = qk / np.sqrt((qk * qk).mean(-1, keepdims=True) + eps) * gain
    out[:, :nq + nkv] = _turn(qk, _angles(positions, inv_freq), layout)
    return out.reshape(x.shape[0], -1)


def qk_norm_rope_backward(qkv: ArrayLike, dout: ArrayLike, nq: int, nkv: int, d: int, gamma_q,
                          gamma_k, inv_freq, positions: Sequence[int], layout: str = "half",
                          eps: float = 1e-5) -> Dict[str, Optional[np.ndarray]]:
    """Gradients of qk_norm_rope: dz = dout turned back, dgamma = sum dz x r,
    dx = r gamma dz - x r^3 / d sum(gamma dz x), r = 1 / sqrt(mean x^2 + eps).
    Also the sums of magnitudes of what is added (for error bounds)."""
    x = to_f64(qkv).reshape(-1, nq + 2 * nkv, d)
    dy = to_f64(dout).reshape(x.shape)
    angle = _angles(positions, inv_freq)
    dx = dy.copy()
    dz = _turn(dy[:, :nq + nkv], None if angle is None else -angle, layout)
    if gamma_q is None:
        dx[:, :nq + nkv] = dz
        return {"dqkv": dx.reshape(x.shape[0], -1), "dgamma_q": None, "dgamma_k": None,
                "mag": np.abs(dx).reshape(x.shape[0], -1)}
    gain = np.concatenate([np.tile(to_f64(gamma_q), (nq, 1)), np.tile(to_f64(gamma_k), (nkv, 1))])
    qk = x[:, :nq + nkv]
    r = 1.0 / np.sqrt((qk * qk).mean(-1, keepdims=True) + eps)
    g = gain * dz
    dx[:, :nq + nkv] = r * g - qk * r ** 3 / d * (g * qk).sum(-1, keepdims=True)
    mag = np.abs(dy)
    mag[:, :nq + nkv] = np.abs(r * g) + np.abs(qk) * r ** 3 / d * np.abs(g * qk).sum(-1, keepdims=True)
    n = dz * qk * r
    return {"dqkv": dx.reshape(x.shape[0], -1), "dgamma_q": n[:, :nq].sum((0, 1)),
            "dgamma_k": n[:, nq:].sum((0, 1)), "mag": mag.reshape(x.shape[0], -1),
            "mag_q": np.abs(n[:, :nq]).sum((0, 1)), "mag_k": np.abs(n[:, nq:]).sum((0, 1))}


# E4M3 codes of non-negative values in ascending order (0x7f is NaN)
_E4M3_POS = E4M3_TABLE[:0x7f]


def e4m3_codes(y: np.ndarray) -> np.ndarray:
    """Nearest E4M3 code of float32 values, ties to the even code, magnitudes
    over 448 to 448, NaN to the NaN code."""
    y = np.asarray(y, dtype=np.float32)
    mag = np.minimum(np.abs(y).astype(np.float64), 448.0)
    hi = np.clip(np.searchsorted(_E4M3_POS, mag), 1, 0x7e)
    lo = hi - 1
    up = mag - _E4M3_POS[lo] > _E4M3_POS[hi] - mag
    tie = mag - _E4M3_POS[lo] == _E4M3_POS[hi] - mag
    code = np.where(up | (tie & (hi % 2 == 0)), hi, lo)
    code = np.where(np.isnan(y), 0x7f, code)
    return (code | np.where(np.signbit(y), 0x80, 0)).astype(np.uint8)


def kv8_quantize(x: ArrayLike) -> Tuple[np.ndarray, np.ndarray]:
    """(codes uint8, scale float32) of rows x [..., d]: scale = max|x| / 448 (NaN
    not counted), code = E4M3(x / scale), in float32; a row of zeros has scale 0
    and codes 0."""
    xf = to_f64(x).astype(np.float32)
    amax = np.fmax.reduce(np.abs(xf), axis=-1, initial=np.float32(0))
    scale = (amax / np.float32(448)).astype(np.float32)
    with np.errstate(invalid="ignore"):
        return e4m3_codes(xf / np.where(amax > 0, scale, np.float32(1))[..., None]), scale


def kv8_values(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """scale * e4m3(code) in float64."""
    return E4M3_TABLE[np.asarray(codes)] * np.asarray(scale, dtype=np.float64)[..., None]


def tree_visible(T: int, words: Optional[np.ndarray]) -> np.ndarray:
    """[T, T] truth values: new token i sees new token j (words None: j <= i)."""
    if words is None:
        return np.tril(np.ones((T, T), dtype=bool))
    w = np.asarray(words).astype(np.int64)
    return np.array([[(int(w[i, j // 64]) >> (j % 64)) & 1 for j in range(T)] for i in range(T)],
                    dtype=bool)


def attn_masked(q: ArrayLike, k: np.ndarray, v: np.ndarray, visible: np.ndarray, nq: int, nkv: int,
                d: int) -> Tuple[np.ndarray, np.ndarray]:
    """ctx [T, nq d] of q [T, nq d] over k, v [nkv, past + T, d]: every cached key
    and the new keys that `visible` [T, T] names.  Also sum_j p_j |v_j| (for
    error bounds).  A row that sees nothing is zero."""
    qf = to_f64(q).reshape(-1, nq, d)
    T, past = qf.shape[0], k.shape[1] - visible.shape[1]
    ctx, mag = np.zeros((T, nq, d)), np.zeros((T, nq, d))
    for i in range(T):
        seen = np.concatenate([np.arange(past), past + np.flatnonzero(visible[i])])
        if seen.size == 0:
            continue
        for h in range(nq):
            kg, vg = k[h // (nq // nkv)][seen], v[h // (nq // nkv)][seen]
            s = kg @ qf[i, h] / math.sqrt(d)
            p = np.exp(s - s.max())
            p /= p.sum()
            ctx[i, h] = p @ vg
            mag[i, h] = p @ np.abs(vg)
    return ctx.reshape(T, -1), mag.reshape(T, -1)
