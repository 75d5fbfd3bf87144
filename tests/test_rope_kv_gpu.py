"""qrope, qkv_store and qkv_load against 64-bit plain forms: every type, layout
and alignment class, strided views, in-place rotation, far positions, partial
heads; the cache's quantisation bit for bit, skipped and bad slots, bad values,
offsets past 32 bits."""
import math

import numpy as np
import pytest

from tests import kv_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def Q():
    import torch  # noqa: F401
    from gemv_mul_mm_gb300 import build as qbuild
    from gemv_mul_mm_gb300 import qmm
    qbuild.build()
    return qmm


def turns_of(freq):
    import torch
    return torch.from_numpy(np.round(np.asarray(freq) / (2 * math.pi) * 2.0 ** 64).astype(np.uint64).view(np.int64)).cuda()


def freqs(rot, base=10000.0):
    return base ** (-2.0 * np.arange(rot // 2) / rot)


def randn(shape, dt, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(U.dtype(dt))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,H,D,rot,pad", [
    (1, 1, 2, 2, 0), (1, 40, 128, 128, 0), (5, 3, 80, 80, 1), (7, 2, 96, 48, 8), (3, 5, 10, 6, 3), (33, 4, 128, 64, 0),
    (2, 1, 256, 20, 2), (301, 9, 64, 64, 4), (4, 70, 112, 28, 0)])
def test_rope(Q, dt, layout, T, H, D, rot, pad):
    import torch
    buf = randn((T, H + 1, D + pad), dt, T * 7 + D)
    x = buf[:, :H, :D] if not pad else buf[:, 1:, pad // 2: pad // 2 + D]     # a strided, possibly misaligned view
    pos = torch.randint(-50, 200000, (T,), dtype=torch.int32, generator=torch.Generator().manual_seed(T)).cuda()
    f = freqs(rot)
    y = Q.qrope(x, pos, turns_of(f), layout=layout, mscale=1.25)
    assert Q.last_path() == Q.PATH_ROPE and y.dtype == x.dtype and y.shape == x.shape
    xs = x.double().cpu().numpy()
    want = U.rotate(xs, pos.cpu().numpy(), f, 1.25, layout)
    err = np.abs(y.double().cpu().numpy() - want)
    # the table holds f to 2^-64 turns and f itself to a double: far below the tolerance
    assert np.all(err <= U.rotate_tol(xs, f, 1.25, layout, dt))
    # in place, on the view: the same bits, and nothing beside the view changes
    before = buf.clone()
    Q.qrope(x, pos, turns_of(f), layout=layout, mscale=1.25, out=x)
    assert torch.equal(x, y)
    x.copy_(before[:, :H, :D] if not pad else before[:, 1:, pad // 2: pad // 2 + D])
    assert torch.equal(buf, before)


def test_rope_far_positions_keep_fp32_accuracy(Q):
    import torch
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 1234567890, 0], dtype=torch.int32, device="cuda")
    x = randn((4, 1, 64), "f32", 3)
    f = freqs(64, 500000.0)
    turns = turns_of(f)
    y = Q.qrope(x, pos, turns).double().cpu().numpy()
    # the same table read as exact fractions of a turn
    phase = [[(int(p) * int(t)) % 2 ** 64 for t in turns.cpu().numpy().view(np.uint64)] for p in pos.cpu().numpy()]
    a = np.array([[p / 2.0 ** 64 * 2 * math.pi for p in row] for row in phase])
    xs = x.double().cpu().numpy()[:, 0]
    want = np.concatenate([xs[:, :32] * np.cos(a) - xs[:, 32:] * np.sin(a), xs[:, 32:] * np.cos(a) + xs[:, :32] * np.sin(a)], 1)
    assert np.all(np.abs(y[:, 0] - want) <= U.rotate_tol(xs[:, None], f, 1.0, "half", "f32")[:, 0])


def test_rope_gradient(Q):
    """The gradient of sum(w * rope(x)) is rope(w) at negated positions: against
    the formula's transpose and against differences."""
    import torch
    T, H, D, rot = 6, 2, 32, 24
    x, w = randn((T, H, D), "f32", 1), randn((T, H, D), "f32", 2)
    pos = torch.arange(5, 5 + T, dtype=torch.int32, device="cuda")
    f = freqs(rot)
    for layout in ("half", "interleaved"):
        g = Q.qrope(w, -pos, turns_of(f), layout=layout).double().cpu().numpy()
        ws, xs, ps = w.double().cpu().numpy(), x.double().cpu().numpy(), pos.cpu().numpy()
        assert np.all(np.abs(g - U.rotate(ws, -ps, f, 1.0, layout)) <= U.rotate_tol(ws, f, 1.0, layout, "f32"))
        for (t, h, d) in [(0, 0, 0), (3, 1, 13), (5, 1, 23), (2, 0, 30)]:
            e = np.zeros_like(xs)
            e[t, h, d] = 0.5
            up, dn = U.rotate(xs + e, ps, f, 1.0, layout), U.rotate(xs - e, ps, f, 1.0, layout)
            # the map is linear: the difference quotient is the derivative
            assert abs(np.sum(ws * (up - dn)) - g[t, h, d]) <= 1e-5


def place(T, page, pages, seed):
    rng = np.random.RandomState(seed)
    return rng.permutation(pages * page)[:T].astype(np.int64)


@pytest.mark.parametrize("fmt", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,H,D,page,off", [(1, 1, 32, 8, 0), (3, 8, 128, 16, 0), (37, 5, 96, 8, 0), (130, 2, 64, 32, 1),
                                            (700, 3, 256, 64, 0), (2, 1, 1024, 4096, 3)])
def test_store_and_load(Q, fmt, dt, T, H, D, page, off):
    import torch
    pages = (T + page - 1) // page + 2
    buf = randn((T, 2 * H, D + off), dt, T + D) * 3
    k, v = buf[:, :H, off:], buf[:, H:, off:]
    k[0, 0, :32] = 0                                                  # a block of zeros
    slots = place(T, page, pages, T)
    slots[T // 2] = -1 if T > 2 else slots[T // 2]
    kc, vc = Q.qkv_cache(fmt, pages, page, H, D)
    kc.fill_(0x55), vc.fill_(0x55)
    Q.qkv_store(fmt, k, v, torch.from_numpy(slots).cuda(), kc, vc, page)
    assert Q.last_path() == Q.PATH_KV_STORE
    for src, cache in ((k, kc), (v, vc)):
        x = src.float().cpu().numpy()
        raw = cache.cpu().numpy().reshape(pages, H, -1)
        want = np.full_like(raw, 0x55)
        for t, s in enumerate(slots):
            if s < 0:
                continue
            p, r = divmod(int(s), page)
            if fmt == "q8_0":
                q, d = U.quantise(x[t])
                want[p, :, r * D:(r + 1) * D] = q.view(np.uint8)
                at = page * D + r * (D // 16)
                want[p, :, at:at + D // 16] = d.view(np.uint8).reshape(H, -1)
            else:
                y = torch.from_numpy(x[t]).to(U.dtype(fmt)).view(torch.uint8).numpy()
                want[p, :, r * 2 * D:(r + 1) * 2 * D] = y.reshape(H, -1)
        assert np.array_equal(raw, want)                              # every byte, those not written too
    for out in ("f32", "f16", "bf16"):
        K, V = Q.qkv_load(fmt, torch.from_numpy(slots).cuda(), kc, vc, page, H, D, dtype=U.dtype(out))
        assert Q.last_path() == Q.PATH_KV_LOAD
        for got, cache in ((K, kc), (V, vc)):
            vals = U.cache_values(fmt, cache, page, H, D)
            for t, s in enumerate(slots):
                want = torch.zeros(H, D, dtype=torch.float64, device="cuda") if s < 0 else vals[s // page, :, s % page]
                # values are exact in fp32; one rounding to the output's type
                assert torch.equal(got[t], want.float().to(U.dtype(out)))
    assert Q.check_device_error() == 0


@pytest.mark.parametrize("fmt", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot,dt", [(128, 128, "f32"), (96, 96, "f16"), (64, 24, "bf16"), (128, 64, "f16"), (32, 10, "f32")])
def test_store_rotates_keys(Q, fmt, layout, D, rot, dt):
    import torch
    T, H, page = 19, 3, 8
    k, v = randn((T, H, D), dt, 5), randn((T, H, D), dt, 6)
    pos = torch.randint(0, 100000, (T,), dtype=torch.int32, generator=torch.Generator().manual_seed(1)).cuda()
    f = freqs(rot)
    kc, vc = Q.qkv_cache(fmt, 4, page, H, D)
    slots = place(T, page, 4, 9)
    Q.qkv_store(fmt, k, v, torch.from_numpy(slots).cuda(), kc, vc, page, positions=pos, turns=turns_of(f), layout=layout, mscale=0.5)
    at = torch.from_numpy(slots).cuda()
    got = U.cache_values(fmt, kc, page, H, D)[at // page, :, at % page].cpu().numpy()
    xs = k.double().cpu().numpy()
    want = U.rotate(xs, pos.cpu().numpy(), f, 0.5, layout)
    tol = U.rotate_tol(xs, f, 0.5, layout, "f32")
    if fmt == "q8_0":   # half a step of the block's scale, the scale's own rounding, and the rotation's error twice
        step = np.abs(want).reshape(T, H, -1, 32).max(-1) / 127
        tol = tol * 2 + np.repeat(step, 32, -1).reshape(want.shape) * (0.5 + 128 * 2.0 ** -11) + 2.0 ** -24
    else:
        tol = tol + U.UNIT[fmt] * np.abs(want) + U.TINY[fmt]
    assert np.all(np.abs(got - want) <= tol)
    # values are stored as they came
    vals = U.cache_values(fmt, vc, page, H, D)[at // page, :, at % page]
    plain = Q.qkv_cache(fmt, 4, page, H, D)
    Q.qkv_store(fmt, v, v, at, plain[0], plain[1], page)
    assert torch.equal(vals, U.cache_values(fmt, plain[1], page, H, D)[at // page, :, at % page])


def test_q8_0_extremes(Q):
    """Blocks with NaN or Inf, with a scale beyond f16, of subnormals and of the
    largest codes: the stored bytes by definition."""
    import torch
    D, page = 64, 8
    x = np.zeros((6, 1, D), np.float32)
    x[0, 0, 5] = np.nan
    x[1, 0, 40] = -np.inf
    x[2, 0, 3] = 1e7                                # 1e7 / 127 > 65504
    x[3, 0, :32] = np.linspace(-1e-6, 1e-6, 32)     # the scale is an f16 subnormal
    x[4, 0, :32] = 1e-9                             # the scale underflows to 0
    x[5, 0, :] = np.linspace(-127.4, 127.4, D)
    t = torch.from_numpy(x).cuda()
    kc, vc = Q.qkv_cache("q8_0", 1, page, 1, D)
    slots = torch.arange(6, device="cuda")
    Q.qkv_store("q8_0", t, -t, slots, kc, vc, page)
    K, V = Q.qkv_load("q8_0", slots, kc, vc, page, 1, D)
    for got, src in ((K, x), (V, -x)):
        q, d = U.quantise(src)
        want = q.reshape(6, 1, 2, 32).astype(np.float64) * d.astype(np.float64)[..., None]
        assert np.array_equal(got.cpu().numpy().astype(np.float64).reshape(want.shape), want, equal_nan=True)
        assert np.isnan(got.cpu().numpy()[0, 0, :32]).all() and not np.isnan(got.cpu().numpy()[0, 0, 32:]).any()


def test_bad_slots(Q):
    import torch
    D, page, H = 64, 8, 2
    x = randn((4, H, D), "f16", 1)
    kc, vc = Q.qkv_cache("f16", 2, page, H, D)
    slots = torch.tensor([3, 16, -2, 15], device="cuda")
    Q.qkv_store("f16", x, x, slots, kc, vc, page)
    assert Q.check_device_error() == Q.STATUS_ID["QMM_ERR_BAD_SLOT"]
    assert Q.check_device_error() == 0                                # read and cleared
    vals = U.cache_values("f16", kc, page, H, D)
    assert torch.equal(vals[0, :, 3], x[0].double()) and torch.equal(vals[1, :, 7], x[3].double())
    assert int((vals != 0).any(-1).sum()) == 2 * H
    K, V = Q.qkv_load("f16", slots, kc, vc, page, H, D, dtype=torch.float16)
    assert Q.check_device_error() == Q.STATUS_ID["QMM_ERR_BAD_SLOT"]
    assert torch.isnan(K[1:3]).all() and torch.isnan(V[1:3]).all() and torch.equal(K[0], x[0]) and torch.equal(V[3], x[3])


def test_offsets_past_32_bits(Q):
    """Pages far apart in one large buffer (layers sharing an allocation), keys
    and values side by side."""
    import torch
    page, H, D, fmt = 16, 2, 64, "q8_0"
    nbytes = Q.qkv_page_bytes(fmt, page, H, D)
    stride = (1 << 31) + 4096
    big = torch.empty(2 * stride + 2 * nbytes, dtype=torch.uint8, device="cuda")
    kc = big.as_strided((3, nbytes), (stride, 1), 0)
    vc = big.as_strided((3, nbytes), (stride, 1), nbytes)
    x, y = randn((3, H, D), "f32", 1), randn((3, H, D), "f32", 2)
    slots = torch.tensor([5, 16 + 7, 32 + 15], device="cuda")
    Q.qkv_store(fmt, x, y, slots, kc, vc, page)
    small = Q.qkv_cache(fmt, 3, page, H, D)
    Q.qkv_store(fmt, x, y, slots, small[0], small[1], page)
    for a, b in zip(Q.qkv_load(fmt, slots, kc, vc, page, H, D), Q.qkv_load(fmt, slots, small[0], small[1], page, H, D)):
        assert torch.equal(a, b) and float(a.abs().max()) > 0
    q = randn((1, 4, D), "f16", 3)
    table, lens = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda"), torch.tensor([48], dtype=torch.int32, device="cuda")
    for c in (kc, vc):
        for p in range(3):
            c[p].copy_(small[0][p] if c is kc else small[1][p])
    assert torch.equal(Q.qattn_decode(fmt, q, kc, vc, table, lens, page, H),
                       Q.qattn_decode(fmt, q, small[0], small[1], table, lens, page, H))
    assert Q.check_device_error() == 0


def test_binding_refuses_and_stays_usable(Q):
    import torch
    x = randn((4, 2, 64), "f16", 1)
    pos, turns = torch.zeros(4, dtype=torch.int32, device="cuda"), turns_of(freqs(64))
    kc, vc = Q.qkv_cache("f16", 2, 16, 2, 64)
    slots = torch.arange(4, device="cuda")
    for call, kind in (
            (lambda: Q.qrope(x.double(), pos, turns), TypeError), (lambda: Q.qrope("x", pos, turns), TypeError),
            (lambda: Q.qrope(x, pos.cpu(), turns), ValueError), (lambda: Q.qrope(x, pos[::2], turns), ValueError),
            (lambda: Q.qrope(x, pos, turns.int()), ValueError), (lambda: Q.qrope(x, pos, turns, out=x.float()), ValueError),
            (lambda: Q.qrope(x, pos, turns, layout="other"), KeyError), (lambda: Q.qrope(x, pos, turns, mscale="a"), TypeError),
            (lambda: Q.qkv_store("f16", x, x, slots, kc, vc.cpu(), 16), ValueError),
            (lambda: Q.qkv_store("f16", x, x, slots, kc, vc, 1 << 40), OverflowError),
            (lambda: Q.qkv_load("f16", slots, kc, vc, 16, 2, 64, dtype=torch.int32), TypeError),
            (lambda: Q.qkv_load("f16", slots, kc, vc, 16, -2, 64), ValueError),
            (lambda: Q.qattn_decode("f16", x, kc, vc, torch.zeros((4, 1), dtype=torch.int32, device="cuda"), pos, 16, 2,
                                    workspace=pos), ValueError)):
        with pytest.raises(kind):
            call()
    with pytest.raises(Q.QmmError) as e:
        Q.qkv_load("q8_0", slots, kc, vc, 16, 2, 80)
    assert e.value.name == "QMM_ERR_COLS_NOT_BLOCK_ALIGNED"
    assert torch.equal(Q.qrope(x, pos, turns), x)                     # position 0: no rotation


def test_on_another_stream_and_in_a_graph(Q):
    import torch
    x = randn((9, 4, 64), "f16", 4)
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    turns = turns_of(freqs(64))
    kc, vc = Q.qkv_cache("q8_0", 3, 16, 4, 64)
    slots = torch.arange(9, device="cuda")
    want = Q.qrope(x, pos, turns)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = Q.qrope(x, pos, turns)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Q.qrope(x, pos, turns, out=out)
        Q.qkv_store("q8_0", out, x, slots, kc, vc, 16)
    out.zero_(), kc.zero_(), vc.zero_()
    g.replay()
    torch.cuda.synchronize()
    ref = Q.qkv_cache("q8_0", 3, 16, 4, 64)
    Q.qkv_store("q8_0", want, x, slots, ref[0], ref[1], 16)
    assert torch.equal(out, want) and torch.equal(kc, ref[0]) and torch.equal(vc, ref[1])
