"""The q4_0 cache: qkv_store's bytes by definition, keys rotated on the way,
qkv_load's values, skipped and bad slots, blocks at the ends of the range."""
import math

import numpy as np
import pytest

from tests import kv_util as U
from tests import layer_util as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def Q():
    import torch  # noqa: F401
    from gemv_mul_mm_gb300 import build as qbuild
    from gemv_mul_mm_gb300 import qmm
    qbuild.build()
    return qmm


def randn(shape, dt, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(U.dtype(dt))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,H,D,page,off", [(1, 1, 32, 8, 0), (3, 8, 128, 16, 0), (37, 5, 96, 8, 0), (130, 2, 64, 32, 1),
                                            (700, 3, 256, 64, 0), (2, 1, 1024, 4096, 3), (5000, 8, 128, 64, 0)])
def test_store_and_load(Q, dt, T, H, D, page, off):
    import torch
    pages = (T + page - 1) // page + 2
    buf = randn((T, 2 * H, D + off), dt, T + D) * 3
    k, v = buf[:, :H, off:], buf[:, H:, off:]
    k[0, 0, :32] = 0                                                  # a block of zeros
    if T > 2:                                                         # values of a few levels: equal magnitudes of both signs
        k[1], v[2] = torch.round(k[1]), torch.round(v[2] * 2) / 2
    slots = np.random.RandomState(T).permutation(pages * page)[:T].astype(np.int64)
    if T > 2:
        slots[T // 2] = -1
    kc, vc = Q.qkv_cache("q4_0", pages, page, H, D)
    kc.fill_(0x55), vc.fill_(0x55)
    Q.qkv_store("q4_0", k, v, torch.from_numpy(slots).cuda(), kc, vc, page)
    assert Q.last_path() == Q.PATH_KV_STORE
    at = np.flatnonzero(slots >= 0)
    pg, row = slots[at] // page, slots[at] % page
    for src, cache in ((k, kc), (v, vc)):
        raw = cache.cpu().numpy().reshape(pages, H, -1)
        want = np.full_like(raw, 0x55)
        codes = want[:, :, :page * D // 2].reshape(pages, H, page, D // 2)
        scales = want[:, :, page * D // 2:].reshape(pages, H, page, D // 16)
        q, d = L.quantise4(src.float().cpu().numpy()[at])
        codes[pg, :, row], scales[pg, :, row] = L.nibbles(q), d.view(np.uint8).reshape(len(at), H, -1)
        want = np.concatenate([codes.reshape(pages, H, -1), scales.reshape(pages, H, -1)], -1)
        assert np.array_equal(raw, want)                              # every byte, those not written too
    for out in ("f32", "f16", "bf16"):
        K, V = Q.qkv_load("q4_0", torch.from_numpy(slots).cuda(), kc, vc, page, H, D, dtype=U.dtype(out))
        assert Q.last_path() == Q.PATH_KV_LOAD
        for got, cache in ((K, kc), (V, vc)):
            vals = L.q4_values(cache, page, H, D)[torch.from_numpy(pg).cuda(), :, torch.from_numpy(row).cuda()]
            # values are exact in fp32; one rounding to the output's type
            assert torch.equal(got[torch.from_numpy(at).cuda()], vals.float().to(U.dtype(out)))
            if T > 2:
                assert bool((got[T // 2] == 0).all())
    assert Q.check_device_error() == 0


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot,dt", [(128, 128, "f32"), (96, 96, "f16"), (64, 24, "bf16"), (128, 64, "f16"), (32, 10, "f32")])
def test_store_rotates_keys(Q, layout, D, rot, dt):
    import torch
    T, H, page = 19, 3, 8
    k, v = randn((T, H, D), dt, 5), randn((T, H, D), dt, 6)
    pos = torch.randint(0, 100000, (T,), dtype=torch.int32, generator=torch.Generator().manual_seed(1)).cuda()
    f = 10000.0 ** (-2.0 * np.arange(rot // 2) / rot)
    turns = torch.from_numpy(np.round(f / (2 * math.pi) * 2.0 ** 64).astype(np.uint64).view(np.int64)).cuda()
    kc, vc = Q.qkv_cache("q4_0", 4, page, H, D)
    at = torch.randperm(32, generator=torch.Generator().manual_seed(9))[:T].cuda()
    Q.qkv_store("q4_0", k, v, at, kc, vc, page, positions=pos, turns=turns, layout=layout, mscale=0.5)
    got = L.q4_values(kc, page, H, D)[at // page, :, at % page].cpu().numpy()
    xs = k.double().cpu().numpy()
    want = U.rotate(xs, pos.cpu().numpy(), f, 0.5, layout)
    # the rotation's error, half a step of the block's scale (a whole one where -8 has no opposite),
    # the scale's own rounding on eight of them, and the rotation's error in the scale
    step = np.repeat(np.abs(want).reshape(T, H, -1, 32).max(-1) / 8, 32, -1).reshape(want.shape)
    tol = 2 * U.rotate_tol(xs, f, 0.5, layout, "f32") + step * (np.where(np.abs(want) > 7.49 * step, 1.0, 0.5) + 9 * 2.0 ** -11) + 2.0 ** -24
    assert np.all(np.abs(got - want) <= tol)
    # the unrotated values, bit for bit
    q, d = L.quantise4(v.float().cpu().numpy())
    vals = (q.reshape(T, H, -1, 32).astype(np.float64) * d.astype(np.float64)[..., None]).reshape(T, H, D)
    assert np.array_equal(L.q4_values(vc, page, H, D)[at // page, :, at % page].cpu().numpy(), vals)


def test_extremes(Q):
    """NaN, Inf, scales beyond f16, subnormal and underflowing ones, opposite values
    of equal magnitude: the stored bytes by definition."""
    import torch
    D, page = 64, 16
    x = np.zeros((9, 1, D), np.float32)
    x[0, 0, 5] = np.nan
    x[1, 0, 40] = -np.inf
    x[2, 0, 3] = 1e6                                # 1e6 / 8 > 65504
    x[3, 0, :32] = np.linspace(-4e-7, 3e-7, 32)     # the scale is an f16 subnormal of one bit
    x[4, 0, :32] = 1e-8                             # the scale underflows to 0
    x[5, 0, :] = np.linspace(-8.4, 8.4, D)
    x[6, 0, :32], x[6, 0, 32:] = np.tile([3.0, -3.0], 16), np.tile([-3.0, 3.0], 16)
    x[7, 0, 31], x[7, 0, 8] = 5.0, -5.0             # equal ones in different lanes
    x[8, 0, :32] = (np.arange(32) - 16) / 2.0       # quotients at halves
    t = torch.from_numpy(x).cuda()
    kc, vc = Q.qkv_cache("q4_0", 1, page, 1, D)
    slots = torch.arange(9, device="cuda")
    Q.qkv_store("q4_0", t, -t, slots, kc, vc, page)
    for got, cache, src in zip(Q.qkv_load("q4_0", slots, kc, vc, page, 1, D), (kc, vc), (x, -x)):
        q, d = L.quantise4(src)
        want = (q.reshape(9, 1, 2, 32).astype(np.float64) * d.astype(np.float64)[..., None]).reshape(9, 1, D)
        assert np.array_equal(got.cpu().numpy().astype(np.float64), want, equal_nan=True)
        assert np.isnan(want[0, 0, :32]).all() and not np.isnan(want[0, 0, 32:]).any() and np.isnan(want[2, 0, :32]).all()
        raw = cache.cpu().numpy()[0]
        assert np.array_equal(raw[:9 * D // 2].reshape(9, 1, -1), L.nibbles(q))


def test_bad_slots(Q):
    import torch
    D, page, H = 64, 8, 2
    x = randn((4, H, D), "f16", 1)
    kc, vc = Q.qkv_cache("q4_0", 2, page, H, D)
    kc.fill_(0x88), vc.fill_(0x88)
    before = kc.clone()
    slots = torch.tensor([3, 16, -2, 15], device="cuda")
    Q.qkv_store("q4_0", x, x, slots, kc, vc, page)
    assert Q.check_device_error() == Q.STATUS_ID["QMM_ERR_BAD_SLOT"]
    touched = (kc != before).view(2, H, -1)
    codes = touched[:, :, :page * D // 2].reshape(2, H, page, -1).any(-1).any(1)
    assert codes.nonzero().tolist() == [[0, 3], [1, 7]]
    K, V = Q.qkv_load("q4_0", slots, kc, vc, page, H, D, dtype=torch.float16)
    assert Q.check_device_error() == Q.STATUS_ID["QMM_ERR_BAD_SLOT"]
    assert torch.isnan(K[1:3]).all() and torch.isnan(V[1:3]).all() and torch.isfinite(K[0]).all() and torch.equal(K[3], V[3])


@pytest.mark.parametrize("page", [16, 32])
def test_offsets_past_32_bits(Q, page):
    import torch
    H, D, fmt = 2, 64, "q4_0"
    nbytes = Q.qkv_page_bytes(fmt, page, H, D)
    stride = (1 << 31) + 4096
    big = torch.empty(2 * stride + 2 * nbytes, dtype=torch.uint8, device="cuda")
    kc = big.as_strided((3, nbytes), (stride, 1), 0)
    vc = big.as_strided((3, nbytes), (stride, 1), nbytes)
    x, y = randn((3 * page, H, D), "f32", 1), randn((3 * page, H, D), "f32", 2)
    slots = torch.randperm(3 * page, generator=torch.Generator().manual_seed(1)).cuda()
    Q.qkv_store(fmt, x, y, slots, kc, vc, page)
    small = Q.qkv_cache(fmt, 3, page, H, D)
    Q.qkv_store(fmt, x, y, slots, small[0], small[1], page)
    for a, b in zip(Q.qkv_load(fmt, slots, kc, vc, page, H, D), Q.qkv_load(fmt, slots, small[0], small[1], page, H, D)):
        assert torch.equal(a, b) and float(a.abs().max()) > 0
    q = randn((1, 4, D), "f16", 3)
    table, lens = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda"), torch.tensor([3 * page - 1], dtype=torch.int32, device="cuda")
    assert torch.equal(Q.qattn_decode(fmt, q, kc, vc, table, lens, page, H),
                       Q.qattn_decode(fmt, q, small[0], small[1], table, lens, page, H))
    assert Q.check_device_error() == 0
