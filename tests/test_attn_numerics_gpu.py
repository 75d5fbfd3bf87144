"""qattn_decode where fp32 arithmetic itself gets coarse: scores past 2^24, over
every cache format and activation type, capped or not, and near the lowest
float; query rows of any
magnitude, cache scales of either sign, key channels far above the others."""
import math

import numpy as np
import pytest

from tests import kv_util as U
from tests.test_attn_decode_gpu import Q, call, check, problem  # noqa: F401

pytestmark = pytest.mark.gpu


def rows(Q, fmt, p, K, V):
    """Writes K and V (n, heads, dim) to the first sequence's positions."""
    import torch
    j = np.arange(K.shape[0])
    slots = torch.from_numpy(p["host"][0][0, j // p["page"]].astype(np.int64) * p["page"] + j % p["page"]).cuda()
    Q.qkv_store(fmt, K, V, slots, p["kc"], p["vc"], p["page"])
    pg, row = slots // p["page"], slots % p["page"]
    return tuple(U.cache_values(fmt, c, p["page"], p["Hkv"], p["D"])[pg, :, row] for c in (p["kc"], p["vc"]))


def equal_keys(Q, fmt, dt, n=70, D=128, k=1.5, q=1.0):
    """One sequence whose keys are all the same, so that every score is and the
    weights are 1 / n whatever the scores."""
    import torch
    p = problem(Q, fmt, dt, D, 1, 2, 16, [n], 3)
    p["q"].fill_(q)
    V = torch.randn((n, 1, D), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    return (p, *rows(Q, fmt, p, torch.full((n, 1, D), k, device="cuda"), V))


def check_equal(Q, p, K, V, score, **kw):
    """The mean of V, and the lse. Equal weights: what is left of the tolerance of
    kv_util.attend is the weights' terms and the sums; the lse follows the
    score's own error, its sum's D / 16 steps of up to 3 terms and three roundings."""
    import torch
    out, lse = call(Q, p, return_lse=True, **kw)
    n, acc = V.shape[0], p["dt"]
    want, mag = V[:, 0].mean(0), V[:, 0].abs().mean(0)
    rel = (3 * n / 16 + 16) * 2.0 ** -23 + (2.0 ** -20 if acc == "f32" else 2.0 ** -16)
    tol = mag * rel + U.UNIT[acc] * want.abs() + U.TINY[acc]
    assert bool(torch.isfinite(out).all()), f"score {score:.3e}: not finite"
    assert bool(((out[0].double() - want).abs() <= tol).all()), f"score {score:.3e}"
    ltol = abs(score) * (3 * p["D"] / 16 + 12) * 2.0 ** -23 + 2.0 ** -20
    assert bool(((lse.double() - (score + math.log(n))).abs() <= ltol).all()), f"score {score:.3e}"


@pytest.mark.parametrize("fmt", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_scores_past_the_integers_of_fp32(Q, fmt, dt):
    """From 2^24 (in log2 units) on, a score less 14 is not a float any more: the
    reference that weights are taken from must not round below it."""
    p, K, V = equal_keys(Q, fmt, dt)
    dot = float((p["q"][0, 0].double() * K[0, 0]).sum())
    for e in range(22, 31):
        for f in (1.0, 1.21, 1.5, 1.87):
            for sign in (1, -1):
                score = sign * 2.0 ** e * f * math.log(2)
                scale = float(np.float32(score / dot))
                check_equal(Q, p, K, V, scale * dot, scale=scale)


@pytest.mark.parametrize("fmt,dt", [("f16", "f16"), ("q8_0", "f16"), ("q8_0", "f32"), ("f16", "f32")])
def test_large_activations_at_the_usual_scale(Q, fmt, dt):
    p, K, V = equal_keys(Q, fmt, dt, k=4000.0, q=4000.0)
    check_equal(Q, p, K, V, float((p["q"][0, 0].double() * K[0, 0]).sum()) * 128 ** -0.5)


@pytest.mark.parametrize("fmt,dt", [("f16", "f16"), ("q8_0", "f32"), ("f16", "f32"), ("bf16", "bf16")])
def test_large_softcaps(Q, fmt, dt):
    p, K, V = equal_keys(Q, fmt, dt)
    dot = float((p["q"][0, 0].double() * K[0, 0]).sum())
    for cap in (3e7, 1.4e8, 2.0 ** 28 * 1.3, 7e8, 3e9):
        for sign in (1, -1):
            scale = float(np.float32(sign * 4 * cap / dot))
            cap32 = float(np.float32(cap))
            check_equal(Q, p, K, V, cap32 * math.tanh(scale * dot / cap32), scale=scale, softcap=cap32)


def negate_blocks(cache, page, heads, dim, seed, share):
    """A share of a q8_0 cache's blocks as (-scale) * (-code): the same values."""
    import torch
    u = cache.view(cache.shape[0], heads, -1)
    codes = u[:, :, :page * dim].view(torch.int8).view(-1, heads, page, dim // 32, 32)
    scales = u[:, :, page * dim:].view(torch.float16).view(-1, heads, page, dim // 32)
    g = torch.Generator(device="cuda").manual_seed(seed)
    flip = torch.rand(scales.shape, generator=g, device="cuda") < share
    codes.copy_(torch.where(flip[..., None], -codes, codes))
    scales.copy_(torch.where(flip, -scales, scales))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,group", [(64, 4), (96, 12), (128, 3), (192, 2), (256, 8)])
@pytest.mark.parametrize("size,share", [(1.0, 0.5), (3000.0, 0.5), (3000.0, 1.0), (1e-3, 1.0)])
def test_negative_scales(Q, dt, D, group, size, share):
    """A block's value is scale * code whatever the scale's sign (a cache may
    come from elsewhere: qkv_store writes none below zero)."""
    import torch
    p = problem(Q, "q8_0", dt, D, 2, group, 16, [333, 40, 0, 1, 3000], D, garbage=False)
    v = p["vc"].view(p["vc"].shape[0], 2, -1)[:, :, 16 * D:].view(torch.float16)
    v.copy_((v.float() * size).half())
    for c, s in ((p["kc"], 1), (p["vc"], 2)):
        negate_blocks(c, 16, 2, D, s, share)
    check(Q, p)


@pytest.mark.parametrize("fmt", ["f16", "q8_0"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_enormous_queries(Q, fmt, dt):
    """Query rows near the end of fp32's range over small keys: finite scores,
    1e29 apart, so that one key takes all."""
    import torch
    p = problem(Q, fmt, dt, 64, 1, 2, 16, [100], 3)
    g = torch.Generator(device="cuda").manual_seed(2)
    K, V = rows(Q, fmt, p, 1e-4 * torch.randn((100, 1, 64), generator=g, device="cuda"), torch.randn((100, 1, 64), generator=g, device="cuda"))
    for size in (2.0 ** 100, 2.0 ** 112, 2.0 ** 118, 2.0 ** 122):
        r = dict(p, q=(p["q"].double() * size).to(p["q"].dtype))
        out, lse = call(Q, r, return_lse=True)
        s = torch.einsum("hd,nd->hn", r["q"][0].double(), K[:, 0]) * 0.125
        best = V[s.argmax(-1), 0]
        tol = 2.0 ** -22 + U.UNIT[dt]
        assert bool(((out[0].double() - best).abs() <= tol * best.abs() + 1e-30).all()), f"q of {size:.1e}"
        assert bool(((lse[0].double() / s.amax(-1) - 1).abs() < 1e-5).all()), f"q of {size:.1e}"


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("outlier", [1.0, 50.0, 500.0])
def test_key_channels_above_the_others(Q, dt, D, outlier):
    """A channel of K far above the others, where q is small, leaves small codes
    elsewhere in its block. The score is the fp32 sum of its terms all the same.
    One key a sequence: its lse is the score. Summed one after another in fp32, the terms
    give an error of a quarter of 2^-23 of S = sum |q k| (rms over many scores);
    1 is allowed."""
    import torch
    n = 96
    p = problem(Q, "q8_0", dt, D, 1, 8, 16, [1] * n, 5)
    g = torch.Generator(device="cuda").manual_seed(4)
    K = torch.randn((n, 1, D), generator=g, device="cuda")
    K[..., 7] *= outlier
    slots = torch.from_numpy(p["host"][0][:, 0].astype(np.int64) * 16).cuda()
    Q.qkv_store("q8_0", K, K, slots, p["kc"], p["vc"], 16)
    K = U.cache_values("q8_0", p["kc"], 16, 1, D)[slots // 16, 0, 0]
    q = 300.0 * torch.randn(p["q"].shape, generator=g, device="cuda")
    q[..., 7] *= 1e-3 if outlier > 1 else 1.0
    p["q"] = q.to(p["q"].dtype)
    _, lse = call(Q, p, return_lse=True)
    terms = p["q"].double() * K[:, None] * D ** -0.5
    err = (lse.double() - terms.sum(-1)) / terms.abs().sum(-1)
    assert float(err.square().mean().sqrt()) <= 2.0 ** -23


@pytest.mark.parametrize("fmt,dt", [("f16", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32"), ("q8_0", "f32")])
def test_scores_near_the_lowest_float(Q, fmt, dt):
    """Finite scores are real ones down to the lowest float (in log2 units)."""
    p, K, V = equal_keys(Q, fmt, dt, D=64, k=1.0)
    dot = float((p["q"][0, 0].double() * K[0, 0]).sum())
    for log2_score in (-1e38, -2.9e38, -3.1e38, -3.39e38):
        scale = float(np.float32(log2_score * math.log(2) / dot))
        check_equal(Q, p, K, V, scale * dot, scale=scale)
