"""Plain float64 forms of the paged K/V cache's calls and of draft verification.

Rows are quantised with the f32 arithmetic that defines the formats (so codes and scales
are exact), everything else is computed in float64, one sequence and one head at a time.
"""
from __future__ import annotations

import numpy as np

from . import qsa_oracle as O

GROUP = 32


def quantise(rows, fmt: str):
    """Stored form of rows [..., D] f16: (codes, scales); scales None for f16."""
    rows = np.asarray(rows, np.float16)
    if fmt == "f16":
        return rows.copy(), None
    one = np.float32(1.0)
    if fmt == "fp8":
        x = rows.astype(np.float32)
        amax = np.abs(x).max(-1)
        safe = np.where(amax == 0, one, amax)
        scale = np.where(amax == 0, one, safe * (one / np.float32(448.0))).astype(np.float32)
        factor = np.where(amax == 0, np.float32(0.0), np.float32(448.0) * (one / safe)).astype(np.float32)
        return O.e4m3_encode(x * factor[..., None]), scale
    g = rows.reshape(*rows.shape[:-1], rows.shape[-1] // GROUP, GROUP).astype(np.float32)
    with np.errstate(all="ignore"):
        amax = np.abs(g).max(-1)
        scale = np.where(np.isfinite(amax), amax * (one / np.float32(7.0)), np.float32(np.nan)).astype(np.float16)
        scale = np.minimum(scale, np.float16(9352))     # the largest f16 that 7 times is one (a NaN stays)
        s = scale.astype(np.float32)[..., None]
        inv = one / s
        codes = np.where(np.isfinite(inv), np.clip(np.rint(g * inv), -7, 7), 0).astype(np.int32) + 8
    byte = codes[..., :GROUP // 2] | (codes[..., GROUP // 2:] << 4)
    return byte.astype(np.uint8).reshape(*rows.shape[:-1], rows.shape[-1] // 2), scale


def values(codes, scales, fmt: str) -> np.ndarray:
    """The float64 values that stored rows stand for."""
    if fmt == "f16":
        return np.asarray(codes, np.float16).astype(np.float64)
    if fmt == "fp8":
        return O.dequantize_kv_rows(codes, scales)
    c = np.asarray(codes, np.uint8).reshape(*codes.shape[:-1], codes.shape[-1] // (GROUP // 2), GROUP // 2).astype(np.int32)
    c = np.concatenate([c & 15, c >> 4], -1) - 8
    v = c * np.asarray(scales, np.float16).astype(np.float64)[..., None]   # exact: 4 x 11 bits
    return v.astype(np.float16).astype(np.float64).reshape(*codes.shape[:-1], codes.shape[-1] * 2)


def attention(q, k, v, sm_scale=None):
    """The T newest tokens' queries q [T, Hq, D] over k, v [n, Hkv, D] float64: (out, lse,
    bound, depth) with bound = sum_c p_c |V_c| per output and depth = the largest
    sum_d |q_d K_cd| * scale per head, which rounding errors are proportional to."""
    q = np.asarray(q, np.float64)
    T, Hq, D = q.shape
    n, Hkv = k.shape[0], k.shape[1]
    sm_scale = 1.0 / np.sqrt(D) if not sm_scale else float(sm_scale)
    out, bound = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, depth = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for u in range(T):
        cells = n - T + u + 1
        if cells <= 0:
            continue
        for h in range(Hq):
            g = h // (Hq // Hkv)
            z = k[:cells, g] @ q[u, h] * sm_scale
            m = z.max()
            e = np.exp(z - m)
            p = e / e.sum()
            out[u, h] = p @ v[:cells, g]
            bound[u, h] = p @ np.abs(v[:cells, g])
            lse[u, h] = m + np.log(e.sum())
            depth[u, h] = (np.abs(k[:cells, g]) @ np.abs(q[u, h])).max() * sm_scale
    return out, lse, bound, depth


def verify(target, draft, tokens, uniforms):
    """One sequence: target [n + 1, V], draft [n, V] or None, tokens [n], uniforms [n + 1] (the
    last draws the next token): (accepted, next token)."""
    target = np.asarray(target, np.float64)
    n, vocab = len(tokens), target.shape[1]
    m = 0
    while m < n:
        d = int(tokens[m])
        if not 0 <= d < vocab:
            break
        q = 1.0 if draft is None else float(draft[m][d])
        u = 0.0 if uniforms[m] < 0 else float(uniforms[m])   # a NaN keeps nothing
        if not u * q < target[m, d]:
            break
        m += 1
    w = target[m].copy()
    if m < n and draft is not None:
        w = np.maximum(w - np.asarray(draft[m], np.float64), 0.0)
    elif m < n and 0 <= int(tokens[m]) < vocab:
        w[int(tokens[m])] = 0.0
    total, upto = w.sum(), 0.0
    if not total > 0:
        return m, int(np.argmax(target[m]))
    t = float(np.fmax(uniforms[-1], 0.0)) * np.cumsum(w)[-1]   # a NaN counts as 0
    for j in np.flatnonzero(w):
        upto += w[j]
        if upto > t:
            return m, int(j)
    return m, int(np.flatnonzero(w)[-1])
