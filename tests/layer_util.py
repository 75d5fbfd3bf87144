"""Plain 64-bit forms of the norm, the router and the q4_0 cache, and the
tolerances their kernels are held to."""
from __future__ import annotations

import numpy as np

from tests import kv_util as U

F = {"f32": np.float32, "f16": np.float16}


def norm(x, residual, weight, offset, eps):
    """float64 rows: (y, h)."""
    h = np.asarray(x, np.float64) + (0.0 if residual is None else np.asarray(residual, np.float64))
    w = 1.0 if weight is None else np.asarray(weight, np.float64) + offset
    return h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * w, h


def norm_tol(y, out):
    """|error| of a row in fp32: h is rounded once; a sum of squares has up to 32 terms
    a thread (D / 1024 in rows read twice) and ten steps between threads, each
    2^-24 of it, and its root halves that; the mean, eps, the root (2 ulp), weight +
    offset and two products: 8 more. Then the output's own rounding."""
    d = y.shape[-1]
    return np.abs(y) * ((1 + (32 + d / 1024 + 10) / 2 + 8) * 2.0 ** -24 + U.UNIT[out]) + U.TINY[out]


def blocks_q8(y):
    """Bytes of fp32 rows (n, D) as Q8_0 blocks, by definition: (n, D / 32 * 34)."""
    q, d = U.quantise(y)
    out = np.empty((*y.shape[:-1], y.shape[-1] // 32, 34), np.uint8)
    out[..., :2] = d[..., None].view(np.uint8).reshape(*d.shape, 2)
    out[..., 2:] = q.reshape(*d.shape, 32).view(np.uint8)
    return out.reshape(*y.shape[:-1], -1)


def route(logits, top_k, score, bias, groups, top_groups, group_top, renorm, scale):
    """(ids, weights, c) of float64 logits (T, E), ties to the lower index."""
    x = np.asarray(logits, np.float64)
    T, E = x.shape
    with np.errstate(all="ignore"):
        if score == "softmax":
            top = x.max(-1, keepdims=True)
            e = np.where(np.isneginf(top), 0.0, np.exp(x - top))
            s = e / np.where(e.sum(-1, keepdims=True) == 0, 1.0, e.sum(-1, keepdims=True))
        else:
            s = 1.0 / (1.0 + np.exp(-x))
    c = s if bias is None else s + np.asarray(bias, np.float64)
    # without a bias the logits have the scores' order (and more of it)
    order_by = x if bias is None else c
    keep = np.ones((T, E), bool)
    if groups > 1:
        by = (c if bias is not None or group_top == 2 else x).reshape(T, groups, -1)
        value = np.sort(by, -1)[..., ::-1][..., :group_top].sum(-1)
        best = np.argsort(-value, axis=-1, kind="stable")[:, :top_groups]
        kept = np.zeros((T, groups), bool)
        np.put_along_axis(kept, best, True, -1)
        keep = np.repeat(kept, E // groups, -1)
    # those that do not stay behind all others, infinite values included
    key = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -order_by, ~keep), axis=-1)[:, :top_k]
    w = np.take_along_axis(s, key, -1)
    if renorm:
        total = w.sum(-1, keepdims=True)
        w = np.where(total == 0, 0.0, w / np.where(total == 0, 1.0, total))
    return key.astype(np.int32), w * scale, c


def quantise4(x):
    """float32 rows -> (codes int8 in [-8, 7], scales float16) of Q4_0, by definition."""
    x = np.asarray(x, np.float32)
    b = x.reshape(*x.shape[:-1], -1, 32)
    with np.errstate(all="ignore"):
        m = np.take_along_axis(b, np.abs(b).argmax(-1)[..., None], -1)[..., 0]   # the first of the largest
        d = (m / np.float32(-8)).astype(np.float16)
        bad = ~np.isfinite(b).all(-1) | ~np.isfinite(d.astype(np.float32))
        d[bad] = np.nan
        df = d.astype(np.float32)
        q = np.rint(b / df[..., None])
        q = np.where(np.isfinite(df) & (df != 0), 1, 0)[..., None] * np.nan_to_num(q, nan=0, posinf=0, neginf=0)
    return np.clip(q, -8, 7).astype(np.int8).reshape(x.shape), d


def nibbles(codes):
    """Bytes of codes (..., D): elements 2 j in the low half of byte j, plus 8."""
    u = (codes.astype(np.int16) + 8).astype(np.uint8)
    return u[..., 0::2] | (u[..., 1::2] << 4)


def q4_values(cache, page, heads, dim):
    """(pages, heads, page, dim) float64 values of a (pages, bytes) uint8 tensor."""
    import torch
    u = cache.contiguous().view(cache.shape[0], heads, -1)
    by = u[:, :, :page * dim // 2].contiguous().view(-1, heads, page, dim // 2)
    codes = torch.stack([by & 15, by >> 4], -1).flatten(-2).double() - 8
    scales = u[:, :, page * dim // 2:].contiguous().view(torch.float16).view(-1, heads, page, dim // 32, 1).double()
    return (codes.unflatten(-1, (-1, 32)) * scales).flatten(-2)
