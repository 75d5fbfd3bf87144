"""qrope, qkv_store and qkv_load at prompt sizes, where a thread takes several
items or heads: every group size, last groups cut short, strided views, part of
a head; against plain forms on the GPU."""
import math

import numpy as np
import pytest

from tests import kv_util as U
from tests.test_rope_kv_gpu import Q, freqs, place, randn, turns_of  # noqa: F401

pytestmark = pytest.mark.gpu


def sms():
    import torch
    return torch.cuda.get_device_properties(0).multi_processor_count


def rotated(x, pos, f, mscale, layout):
    """kv_util.rotate and kv_util.rotate_tol (of an fp32 result) in torch."""
    import torch
    a = pos.double()[:, None, None] * torch.from_numpy(np.asarray(f)).cuda()
    c, s = mscale * a.cos(), mscale * a.sin()
    y, tol = x.double().clone(), x.double().abs() * U.UNIT["f32"]
    n = len(f)
    first, second = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    x1, x2 = x.double()[..., first], x.double()[..., second]
    y[..., first], y[..., second] = x1 * c - x2 * s, x2 * c + x1 * s
    tol[..., first] = tol[..., second] = mscale * (x1.abs() + x2.abs()) * 8 * 2.0 ** -24
    return y, tol


@pytest.mark.parametrize("dt,T,H,D,rot,pad,items", [
    ("f16", 3001, 13, 128, 128, 0, 2), ("bf16", 8192, 33, 128, 128, 8, 4), ("f32", 3001, 13, 128, 64, 4, 2),
    ("f32", 9001, 14, 128, 128, 0, 4), ("f16", 5003, 21, 96, 48, 0, 2), ("bf16", 5003, 7, 80, 80, 2, 2), ("f16", 4999, 9, 64, 20, 1, 2),
    ("f32", 8191, 11, 96, 64, 0, 2), ("f32", 15013, 11, 96, 64, 0, 4), ("f16", 8009, 5, 112, 112, 1, 4), ("f32", 2999, 3, 2048, 2048, 0, 4)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope(Q, dt, T, H, D, rot, pad, items, layout):
    import torch
    buf = randn((T, H + 1, D + pad), dt, T)
    x = buf[:, 1:, pad // 2: pad // 2 + D]
    size = 4 if dt == "f32" else 2
    vec = next(n for n in (16 // size, 2, 1) if rot % (2 * n) == 0 and (D - rot) % n == 0 and ((D + pad) * size) % min(16, n * size) == 0
               and x.data_ptr() % min(16, n * size) == 0)
    units = rot // (2 * vec) + (D - rot + 2 * vec - 1) // (2 * vec)
    per_sm = T * H * units // (sms() * 256)
    assert (4 if per_sm >= 48 else 2 if per_sm >= 4 else 1) == items        # what the kernel's choice goes by
    pos = torch.arange(7, 7 + T, dtype=torch.int32, device="cuda")
    f = freqs(rot)
    y = Q.qrope(x, pos, turns_of(f), layout=layout, mscale=1.25)
    want, tol = rotated(x, pos, f, 1.25, layout)
    assert bool(((y.double() - want).abs() <= tol + U.UNIT[dt] * want.abs() + U.TINY[dt]).all())
    before = buf.clone()
    Q.qrope(x, pos, turns_of(f), layout=layout, mscale=1.25, out=x)
    assert torch.equal(x, y)
    x.copy_(before[:, 1:, pad // 2: pad // 2 + D])
    assert torch.equal(buf, before)


def stored(fmt, x):
    """What a cache of `fmt` holds of x, as doubles: kv_util.quantise in torch."""
    import torch
    if fmt != "q8_0":
        return x.to(U.dtype(fmt)).double()
    b = x.float().unflatten(-1, (-1, 32))
    d = (b.abs().amax(-1) / torch.full((), 127.0, device="cuda")).half()
    q = torch.where(d[..., None] > 0, torch.round(b / d.float()[..., None]), 0.0).clamp(-127, 127)
    return (q.double() * d.double()[..., None]).flatten(-2)


@pytest.mark.parametrize("fmt", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("dt,H,D,page,off", [("f32", 7, 128, 16, 0), ("f16", 13, 64, 64, 0), ("bf16", 5, 96, 8, 0), ("f32", 3, 256, 32, 1),
                                             ("f16", 9, 160, 16, 1)])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("rope", [None, ("half", 1.0), ("half", 0.5), ("interleaved", 1.0), ("interleaved", 0.25)])
def test_store_and_load(Q, fmt, dt, H, D, page, off, group, rope):
    """`group` heads a thread where H has that many: the smallest T that gets there and a few tokens more."""
    import torch
    rot = 0 if rope is None else int(rope[1] * D) // 2 * 2
    pairs = rope is not None and rope[0] == "half" and rot == D and D % 64 == 0 and off == 0
    per_thread = 16 if pairs else 8
    T = -(-group * sms() * 4 * 256 // (2 * (D // per_thread) * H)) + 5
    pages = (T + page - 1) // page + 2
    buf = randn((T, 2 * H, D + off), dt, T) * 3
    k, v = buf[:, :H, off:], buf[:, H:, off:]
    slots = place(T, page, pages, T)
    slots[T // 2] = -1
    at = torch.from_numpy(slots).cuda()
    kc, vc = Q.qkv_cache(fmt, pages, page, H, D)
    kw = {}
    if rope:
        pos = torch.arange(11, 11 + T, dtype=torch.int32, device="cuda")
        kw = dict(positions=pos, turns=turns_of(freqs(rot)), layout=rope[0], mscale=0.75)
    Q.qkv_store(fmt, k, v, at, kc, vc, page, **kw)
    live = at >= 0
    rows = [U.cache_values(fmt, c, page, H, D)[at[live] // page, :, at[live] % page] for c in (kc, vc)]
    assert torch.equal(rows[1], stored(fmt, v[live]))
    if not rope:
        assert torch.equal(rows[0], stored(fmt, k[live]))
    else:
        want, tol = rotated(k[live], pos[live], freqs(rot), 0.75, rope[0])
        if fmt == "q8_0":   # half a step of the block's scale, the scale's own rounding, and the rotation's error twice
            step = want.abs().unflatten(-1, (-1, 32)).amax(-1) / 127
            tol = 2 * tol + step.repeat_interleave(32, -1) * (0.5 + 128 * 2.0 ** -11) + 2.0 ** -24
        else:
            tol = tol + U.UNIT[fmt] * want.abs() + U.TINY[fmt]
        assert bool(((rows[0] - want).abs() <= tol).all())
    untouched = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    untouched[at[live]] = False
    rest = torch.nonzero(untouched).flatten()
    for c in (kc, vc):
        assert not bool(U.cache_values(fmt, c, page, H, D)[rest // page, :, rest % page].any())
    for out in ("f32", "f16"):
        got = Q.qkv_load(fmt, at, kc, vc, page, H, D, dtype=U.dtype(out))
        for g, r in zip(got, rows):
            assert torch.equal(g[live], r.float().to(U.dtype(out))) and not bool(g[T // 2].any())
    assert Q.check_device_error() == 0


def test_positions_and_slots_of_a_whole_context(Q):
    """8 heads a thread and one left over, offsets past 2^31 bytes in K and V."""
    import torch
    T, H, D, page = 262144, 9, 128, 64
    kv = torch.empty((T, 2 * H, D), device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    at = torch.randperm(T, generator=torch.Generator().manual_seed(2)).cuda()
    kc, vc = Q.qkv_cache("f16", T // page, page, H, D)
    Q.qkv_store("f16", kv[:, :H], kv[:, H:], at, kc, vc, page)
    K, V = Q.qkv_load("f16", at, kc, vc, page, H, D, dtype=torch.float16)
    assert torch.equal(K, kv[:, :H].half()) and torch.equal(V, kv[:, H:].half())
    assert math.prod(kv.shape) * 4 > 2 ** 31 and Q.check_device_error() == 0
