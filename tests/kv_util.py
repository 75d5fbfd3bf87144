"""Plain 64-bit forms of the rotary, cache and attention operators, and the
tolerances their fp32 kernels are held to."""
from __future__ import annotations

import math

import numpy as np

UNIT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}    # unit roundoff
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}  # half the smallest subnormal


def dtype(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def rotate(x, pos, freq, mscale, layout):
    """float64 (T, H, D) rotated at pos by radians-per-position freq."""
    x = np.asarray(x, np.float64)
    n = len(freq)
    a = np.asarray(pos, np.float64)[:, None, None] * np.asarray(freq, np.float64)
    c, s = mscale * np.cos(a), mscale * np.sin(a)
    y = x.copy()
    i = np.arange(n)
    first, second = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., second] * c + x[..., first] * s
    return y


def rotate_tol(x, freq, mscale, layout, out):
    """|error| of the fp32 rotation: the angle is off by pi 2^-25 (the half-turn
    count's rounding) and 2 pi 2^-32 (the phase's lowest bits), sin and cos by 2
    ulp, products and their sum by 3 roundings: below 6 * 2^-24 of |x1| + |x2|;
    then the output's own rounding."""
    x = np.abs(np.asarray(x, np.float64))
    n = len(freq)
    i = np.arange(n)
    first, second = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
    t = UNIT[out] * x
    both = abs(mscale) * (x[..., first] + x[..., second])
    t[..., first] = t[..., second] = both * (7 * 2.0 ** -24 + UNIT[out])
    return t + TINY[out]


def cache_values(fmt, cache, page, heads, dim):
    """(pages, heads, page, dim) float64 values of a (pages, bytes) uint8 tensor."""
    import torch
    c = cache.contiguous()
    n = c.shape[0]
    if fmt != "q8_0":
        return c.view(dtype(fmt)).view(n, heads, page, dim).double()
    u = c.view(n, heads, -1)
    codes = u[:, :, :page * dim].contiguous().view(torch.int8).view(n, heads, page, dim // 32, 32).double()
    scales = u[:, :, page * dim:].contiguous().view(torch.float16).view(n, heads, page, dim // 32, 1).double()
    return (codes * scales).view(n, heads, page, dim)


def quantise(x):
    """float32 rows -> (codes int8, scales float16) of Q8_0, by definition."""
    x = np.asarray(x, np.float32)
    b = x.reshape(*x.shape[:-1], -1, 32)
    with np.errstate(all="ignore"):
        d = (np.abs(b).max(-1) / np.float32(127)).astype(np.float16)
        bad = ~np.isfinite(b).all(-1) | ~np.isfinite(d.astype(np.float32))
        d[bad] = np.nan
        q = np.rint(b / d.astype(np.float32)[..., None])
        q = np.where(np.isfinite(d.astype(np.float32)) & (d > 0), 1, 0)[..., None] * np.nan_to_num(q, nan=0, posinf=0, neginf=0)
    return np.clip(q, -127, 127).astype(np.int8).reshape(x.shape), d


def attend(q, K, V, scale, softcap=0.0, acc="f32", n_terms=3):
    """One sequence in 64 bits: q (Hq, D), K and V (n, Hkv, D) of the positions in
    range. Returns out, lse and tolerances for both.

    Score error: products are exact and summed in fp32 in D / 16 MMA steps of up
    to 3 terms, q is off by 2^-22: delta = S (3 D / 16 + 8) 2^-23 with S = scale
    sum |q k|, its largest; the exponent adds 2 ulp of S log2 e. A relative
    weight error is then below 2.5 delta (a weight and the sum). Weights enter
    the second product to 2^-22 (fp32) or 2^-16 (16-bit outputs) and are summed
    in n / 16 steps per term."""
    import torch
    n, hkv, d = K.shape
    group = q.shape[0] // hkv
    if n == 0:
        return torch.zeros_like(q), torch.full((q.shape[0],), -math.inf, dtype=q.dtype, device=q.device), \
            torch.zeros_like(q), torch.zeros(q.shape[0], dtype=q.dtype, device=q.device)
    qg = q.view(hkv, group, d)
    s = torch.einsum("hgd,nhd->hgn", qg, K) * scale
    S = (torch.einsum("hgd,nhd->hgn", qg.abs(), K.abs()) * abs(scale)).amax(-1)
    if softcap:
        s = softcap * torch.tanh(s / softcap)
    lse = torch.logsumexp(s, -1)
    w = torch.exp(s - lse[..., None])
    out = torch.einsum("hgn,nhd->hgd", w, V)
    wv = torch.einsum("hgn,nhd->hgd", w, V.abs())
    delta = S * (3 * d / 16 + 12) * 2.0 ** -23 + 2.0 ** -20
    rel = 2.5 * delta + (n_terms * n / 16 + 16) * 2.0 ** -23 + (2.0 ** -20 if acc == "f32" else 2.0 ** -16)
    tol = wv * rel[..., None] + UNIT[acc] * out.abs() + TINY[acc]
    ltol = delta + (n / 16 + 16) * 2.0 ** -23 + 2.0 ** -22 * lse.abs()
    return out.reshape(-1, d), lse.reshape(-1), tol.reshape(-1, d), ltol.reshape(-1)
