"""Plain float64 / IEEE float32 forms of the serving operators (test infrastructure only).

* ``norm_rope``       RMS norm and position rotation of head rows, float64;
* ``k_codes``, ``v_codes``  the cache's codes and scales, in IEEE float32 as the write defines them;
* ``read``            codes back to values, float32 as the read defines it;
* ``decode``          attention of one query token over float64 keys and values, with the terms that
                      bound an fp32 evaluation of it.

Written from the formulas in include/sage.h; shares no code with the CUDA library.
"""
from __future__ import annotations

import numpy as np

from . import fp8

TINY = np.float32(2.0 ** -100)


def norm_rope(x, norm, eps, w, cos_sin, pos, interleaved):
    """x (tokens, heads, d); cos_sin (n_pos, rot) or None; pos (tokens,).  Returns (y, magnitude): the
    result in float64, and sum |terms| of every element, which scales its rounding errors."""
    x = np.asarray(x, np.float64)
    d = x.shape[-1]
    n = x
    if norm:
        n = x / np.sqrt((x * x).sum(-1, keepdims=True) / d + eps)
        if w is not None:
            n = n * np.asarray(w, np.float64)
    y, mag = n.copy(), np.abs(n)
    if cos_sin is not None:
        h = cos_sin.shape[1] // 2
        row = np.asarray(cos_sin, np.float64)[pos][:, None]
        c, s = row[..., :h], row[..., h:]
        i = np.arange(h)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        y[..., a] = n[..., a] * c - n[..., b] * s
        y[..., b] = n[..., b] * c + n[..., a] * s
        mag[..., a] = np.abs(n[..., a] * c) + np.abs(n[..., b] * s)
        mag[..., b] = np.abs(n[..., b] * c) + np.abs(n[..., a] * s)
    return y, mag


def _scales(x, top):
    top = np.float32(top)
    bad = ~np.isfinite(x).all(-1)
    a = np.where(bad, np.float32(1), np.abs(np.where(np.isfinite(x), x, 0)).max(-1)).astype(np.float32)
    keep = (a >= TINY) & ~bad
    safe = np.where(keep, a, np.float32(1)).astype(np.float32)
    scale = np.where(keep, (safe / top).astype(np.float32), np.float32(0))
    scale = np.where(bad, np.float32(np.nan), scale).astype(np.float32)
    inv = np.where(keep, (top / safe).astype(np.float32), np.float32(0)).astype(np.float32)
    return scale, inv, keep


def k_codes(k, k_mean=None):
    """k (..., Hkv, d) float32 values (exactly representable): int8 codes and float32 scales."""
    y = np.asarray(k, np.float32)
    if k_mean is not None:
        y = y - np.asarray(k_mean, np.float32)
    scale, inv, keep = _scales(y, 127)
    with np.errstate(invalid="ignore"):
        c = np.clip(np.rint((y * inv[..., None]).astype(np.float32)), -127, 127)
    return np.where(keep[..., None], c, 0).astype(np.int8), scale


def v_codes(v):
    y = np.asarray(v, np.float32)
    scale, inv, keep = _scales(y, 448)
    with np.errstate(invalid="ignore"):
        c = fp8.encode(np.where(keep[..., None], (y * inv[..., None]).astype(np.float32), 0))
    return np.where(keep[..., None], c, 0).astype(np.uint8), scale


def read(k8, ks, v8, vs, k_mean=None):
    """float32 values before the rounding to 16 bits."""
    with np.errstate(invalid="ignore"):
        k = (k8.astype(np.float32) * ks[..., None]).astype(np.float32)
        if k_mean is not None:
            k = (k + np.asarray(k_mean, np.float32)).astype(np.float32)
        v = (fp8.decode(v8).astype(np.float32) * vs[..., None]).astype(np.float32)
    return k, v


def decode(q, k, v, scale):
    """q (Hq, d), k and v (n, Hkv, d) float64.  Returns (out, spread, delta), each (Hq, d) or (Hq, 1):
    out the attention, spread = sum_j p_j |v_j|, delta = max_j scale sum_c |q_c k_jc| (the score's
    magnitude before cancellation)."""
    Hq, d = q.shape
    n, Hkv = k.shape[:2]
    if n == 0:
        z = np.zeros((Hq, d))
        return z, z, np.zeros((Hq, 1))
    G = Hq // Hkv
    kk, vv = np.repeat(k, G, 1), np.repeat(v, G, 1)
    s = np.einsum("hd,nhd->hn", q, kk) * scale
    delta = np.einsum("hd,nhd->hn", np.abs(q), np.abs(kk)).max(1, keepdims=True) * scale
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    return np.einsum("hn,nhd->hd", p, vv), np.einsum("hn,nhd->hd", p, np.abs(vv)), delta
