"""Attention with modified scores and masks, and the int8 cache, in fp64 -- TEST INFRASTRUCTURE ONLY.

The definitions, row by row, with nothing blocked or fused. A query row at
position pos sees the keys lo <= t < hi,
    lo = max(0, pos - window + 1 (window > 0), key_start), hi = max(pos + 1, min(prefix, len)),
and only those enter its scores, softmax and sum: whatever other positions hold
has no effect.
"""
from __future__ import annotations

import numpy as np


def visible(pos, length, window=0, key_start=None, prefix=None):
    lo = max(0, pos - window + 1) if window > 0 else 0
    if key_start is not None:
        lo = max(lo, int(key_start))
    hi = pos + 1
    if prefix is not None:
        hi = max(hi, min(int(prefix), length))
    return lo, hi


def attend_row(q, k, v, pos, length, scale, softcap=0.0, slopes=None, window=0, key_start=None, prefix=None):
    """q [H_q, Dh]; k, v [length, H_kv, Dh] (fp64) -> [H_q, Dh]."""
    H_q, Dh = q.shape
    g = H_q // k.shape[1]
    out = np.zeros((H_q, Dh))
    lo, hi = visible(pos, length, window, key_start, prefix)
    if lo >= hi:
        return out
    t = np.arange(lo, hi)
    with np.errstate(all="ignore"):
        for h in range(H_q):
            s = scale * (k[lo:hi, h // g] @ q[h])
            if softcap > 0:
                s = softcap * np.tanh(s / softcap)
            if slopes is not None:
                s = s - float(slopes[h]) * np.abs(pos - t)
            w = np.exp(s - np.max(s))
            out[h] = (w[:, None] * v[lo:hi, h // g]).sum(0) / w.sum()
    return out


def gather(pages, table_row, length, page_size):
    """Logical rows [length, H_kv, ...] of one sequence from pools [num_pages, H_kv, P, ...]."""
    t = np.arange(length)
    return pages[np.asarray(table_row)[t // page_size], :, t % page_size]


def quantise_int8(x):
    """(codes int8, scales fp32) of rows x [..., Dh] (fp32 values): scale = a / 127, code = rint(x * (127 / a)), the
    divisions and the product rounded to fp32 on their own."""
    x = np.asarray(x, np.float32)
    a = np.abs(x).max(-1)
    finite = np.isfinite(x).all(-1)
    live = finite & (a >= np.float32(2.0) ** -100)
    one = np.where(live, a, np.float32(1))
    inv = (np.float32(127) / one).astype(np.float32)
    safe = np.where(live[..., None], x, np.float32(0))
    codes = np.rint((safe * inv[..., None]).astype(np.float32)).astype(np.int8)
    scales = np.where(live, (one / np.float32(127)).astype(np.float32), np.float32(0))
    return codes, np.where(finite, scales, np.float32(np.nan)).astype(np.float32)


def norm_rope(x, weight, eps, positions, cos_sin, style):
    """RMS norm of rows x [B, H, Dh], then the rotation by the fp32 table's entries, in fp64."""
    x = np.asarray(x, np.float64)
    Dh = x.shape[-1]
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    c = np.asarray(cos_sin, np.float64)[positions][:, None, :]
    cos, sin = c[..., :Dh // 2], c[..., Dh // 2:]
    i, j = (np.arange(Dh // 2), np.arange(Dh // 2, Dh)) if style == "half" else (np.arange(0, Dh, 2), np.arange(1, Dh, 2))
    out = np.empty_like(y)
    out[..., i] = y[..., i] * cos - y[..., j] * sin
    out[..., j] = y[..., j] * cos + y[..., i] * sin
    return out
