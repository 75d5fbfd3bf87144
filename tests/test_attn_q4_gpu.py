"""qattn_decode over a q4_0 cache against the 64-bit plain form: activation types,
head dims and groups, page sizes, lengths around every tile and page edge,
windows, softcaps; scales of either sign, garbage outside the range, empty
sequences, bad tables and lengths, splits, determinism, streams and graphs."""
import math

import numpy as np
import pytest

from tests import kv_util as U
from tests import layer_util as L

pytestmark = pytest.mark.gpu

FMT = "q4_0"
EDGES = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 127, 128, 129, 160, 200, 1000]


@pytest.fixture(scope="module")
def Q():
    import torch  # noqa: F401
    from gemv_mul_mm_gb300 import build as qbuild
    from gemv_mul_mm_gb300 import qmm
    qbuild.build()
    return qmm


def problem(Q, dt, D, Hkv, group, page, lens, seed, qscale=1.5):
    """Caches whose every unused row is NaN, tables whose unused entries are -1."""
    import torch
    rng = np.random.RandomState(seed)
    need = [(n + page - 1) // page for n in lens]
    width = max(1, max(need))
    order = rng.permutation(sum(need) + 2)
    table = np.full((len(lens), width), -1, np.int32)
    used = np.zeros((len(order), page), bool)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        j = np.arange(lens[b])
        used[table[b, j // page], j % page] = True
        at += n
    g = torch.Generator(device="cuda").manual_seed(seed)
    kc, vc = Q.qkv_cache(FMT, len(order), page, Hkv, D)
    for mask, make in ((used, lambda n, m: torch.randn((n, Hkv, D), generator=g, device="cuda") + m),
                       (~used, lambda n, m: torch.full((n, Hkv, D), math.nan, device="cuda"))):
        pg, row = np.nonzero(mask)
        if len(pg):
            slots = torch.from_numpy(pg.astype(np.int64) * page + row).cuda()
            Q.qkv_store(FMT, make(len(pg), 0.0), make(len(pg), 0.3), slots, kc, vc, page)
    q = (qscale * torch.randn((len(lens), Hkv * group, D), generator=g, device="cuda")).to(U.dtype(dt))
    return dict(dt=dt, page=page, Hkv=Hkv, D=D, q=q, kc=kc, vc=vc, table=torch.from_numpy(table).cuda(),
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), host=(table, lens))


def call(Q, p, **kw):
    return Q.qattn_decode(FMT, p["q"], p["kc"], p["vc"], p["table"], p["lens"], p["page"], p["Hkv"], **kw)


def check(Q, p, window=0, softcap=0.0, scale=None, **kw):
    import torch
    out, lse = call(Q, p, window=window, softcap=softcap, scale=scale, return_lse=True, **kw)
    assert Q.last_path() == Q.PATH_ATTN and Q.check_device_error() == 0
    assert out.dtype == p["q"].dtype and lse.dtype == torch.float32
    table, lens = p["host"]
    kv = [L.q4_values(c, p["page"], p["Hkv"], p["D"]) for c in (p["kc"], p["vc"])]
    for b, n in enumerate(lens):
        lo = max(0, n - window) if window else 0
        j = np.arange(lo, n)
        pg, row = torch.from_numpy(table[b, j // p["page"]].astype(np.int64)).cuda(), torch.from_numpy(j % p["page"]).cuda()
        K, V = (c[pg, :, row] for c in kv)
        want, wl, tol, ltol = U.attend(p["q"][b].double(), K, V, p["D"] ** -0.5 if scale is None else scale, softcap, p["dt"])
        err = (out[b].double() - want).abs()
        assert bool((err <= tol).all()), f"sequence {b} of length {n}: off by {float((err - tol).max())}"
        if n == 0:
            assert bool((out[b] == 0).all()) and bool((lse[b] == -math.inf).all())
        else:
            assert bool(((lse[b].double() - wl).abs() <= ltol).all())
    return out, lse


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("Hkv,group,page", [(2, 4, 16), (1, 13, 8), (1, 8, 64)])
def test_lengths_at_every_edge(Q, dt, D, Hkv, group, page):
    check(Q, problem(Q, dt, D, Hkv, group, page, EDGES, D + group))


@pytest.mark.parametrize("dt", ["f32", "f16"])
@pytest.mark.parametrize("Hkv,group", [(1, 1), (3, 1), (5, 7), (2, 8), (1, 9), (2, 16), (1, 17), (1, 40)])
def test_head_groups(Q, dt, Hkv, group):
    check(Q, problem(Q, dt, 128, Hkv, group, 32, [77, 300, 5], group))


@pytest.mark.parametrize("dt,D", [("f32", 128), ("f16", 64), ("bf16", 96), ("f16", 256)])
@pytest.mark.parametrize("page", [8, 16, 64, 512])
@pytest.mark.parametrize("window,softcap", [(1, 0.0), (13, 0.0), (16, 30.0), (100, 0.0), (5000, 2.0), (0, 10.0)])
def test_windows_softcaps_and_pages(Q, dt, D, page, window, softcap):
    check(Q, problem(Q, dt, D, 2, 3, page, [0, 1, 14, 16, 100, 117, 513, 1500], page + window), window, softcap)


@pytest.mark.parametrize("dt,D,group", [("f16", 128, 4), ("f32", 128, 8), ("bf16", 64, 2), ("f16", 96, 12), ("f32", 256, 1)])
def test_long_sequences_are_split_and_joined(Q, dt, D, group):
    import torch
    p = problem(Q, dt, D, 1, group, 64, [30011, 20000, 129], 3)
    need = Q.qattn_decode_workspace_bytes(FMT, U.dtype(dt), 3, group, 1, D, p["table"].shape[1] * 64)
    assert need > 0
    a = check(Q, p)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    b = call(Q, p, return_lse=True, workspace=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(Q.QmmError) as e:
        call(Q, p, workspace=ws[:-16])
    assert e.value.name == "QMM_ERR_WORKSPACE_TOO_SMALL"


@pytest.mark.parametrize("dt", ["f32", "f16"])
def test_many_sequences_and_a_long_one(Q, dt):
    lens = [int(v) for v in np.random.RandomState(1).randint(0, 700, 150)]
    lens[40] = 20000
    check(Q, problem(Q, dt, 128, 2, 4, 16, lens, 4))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_any_bytes_are_a_cache(Q, dt):
    """Random codes, scales of both signs over a wide range, the largest among small ones."""
    import torch
    p = problem(Q, dt, 128, 2, 4, 16, [500, 37, 1, 130], 11)
    g = torch.Generator(device="cuda").manual_seed(5)
    for i, c in enumerate((p["kc"], p["vc"])):
        u = c.view(c.shape[0], 2, -1)
        u[:, :, :16 * 64] = torch.randint(0, 256, u[:, :, :16 * 64].shape, generator=g, device="cuda", dtype=torch.uint8)
        s = u[:, :, 16 * 64:].view(torch.float16)
        e = torch.randint(-12, 1 if i == 0 else 6, s.shape, generator=g, device="cuda")
        s.copy_(torch.randn(s.shape, generator=g, device="cuda").sign() * 2.0 ** e * 0.3)
    check(Q, p, scale=0.02)


@pytest.mark.parametrize("dt", ["f32", "f16"])
@pytest.mark.parametrize("qscale", [1e-3, 30.0, 2000.0])
def test_small_and_large_scores(Q, dt, qscale):
    check(Q, problem(Q, dt, 128, 1, 4, 32, [400, 90], 6, qscale))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("group", [1, 2, 3, 4, 5])
def test_few_query_heads_over_small_and_large_pages(Q, dt, D, group):
    for page in (8, 32):
        check(Q, problem(Q, dt, D, 2, group, page, [1, 31, 33, 200, 0, 411], D + group + page))
    check(Q, problem(Q, dt, D, 2, group, 32, [90, 411], D + group), 40, 5.0)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("group", [4, 8, 16])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_query_without_a_value_stays_in_its_head(Q, dt, group, bad):
    import torch
    p = problem(Q, dt, 128, 2, group, 32, [300, 2, 5000], 3)
    want = call(Q, p)
    p["q"][:, 1, 7] = bad
    p["q"][:, group + group - 1, 100] = bad
    got = call(Q, p)
    hit = torch.zeros(2 * group, dtype=torch.bool, device="cuda")
    hit[[1, 2 * group - 1]] = True
    assert bool(torch.isnan(got[:, hit]).all()) and torch.equal(got[:, ~hit], want[:, ~hit])


def test_infinities_and_nan_in_range_show(Q):
    import torch
    p = problem(Q, "f16", 64, 1, 2, 16, [50, 50, 50], 8)
    want = call(Q, p)
    bad = torch.full((1, 1, 64), math.nan, device="cuda")
    ok = torch.zeros((1, 1, 64), device="cuda")
    table = p["host"][0]
    Q.qkv_store(FMT, bad, ok, torch.tensor([int(table[0, 1]) * 16 + 3], device="cuda"), p["kc"], p["vc"], 16)
    Q.qkv_store(FMT, ok, bad, torch.tensor([int(table[1, 2]) * 16], device="cuda"), p["kc"], p["vc"], 16)
    got = call(Q, p)
    assert torch.isnan(got[0]).all() and torch.isnan(got[1]).all() and torch.equal(got[2], want[2])


def test_bad_tables_and_lengths(Q):
    import torch
    p = problem(Q, "f16", 128, 2, 4, 16, [40, 40, 40, 40], 2)
    want = call(Q, p)
    for where, value in ((0, 1 << 20), (1, -7)):
        p["table"][where, 1] = value
    p["lens"][2] = 1000
    got, lse = call(Q, p, return_lse=True)
    assert Q.check_device_error() == Q.STATUS_ID["QMM_ERR_BAD_SLOT"]
    assert torch.isnan(got[:3]).all() and torch.isnan(lse[:3]).all() and torch.equal(got[3], want[3])


def test_views_streams_and_graphs(Q):
    import torch
    p = problem(Q, "f16", 128, 2, 4, 16, [300, 17, 0, 2000], 9)
    want = call(Q, p)
    wide = torch.zeros((4, 11, 128), dtype=torch.float16, device="cuda")
    wide[:, 2:10] = p["q"]
    assert torch.equal(call(Q, dict(p, q=wide[:, 2:10])), want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = call(Q, p)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(Q, p, out=out)
    p["lens"].copy_(torch.tensor([10, 0, 0, 1999], dtype=torch.int32))       # (sequence 2 has no pages)
    g.replay()
    torch.cuda.synchronize()
    again = call(Q, p, max_len=p["table"].shape[1] * 16)
    assert torch.equal(out, again) and not torch.equal(out, want) and bool((out[1] == 0).all())
    # in place of q
    q = p["q"].clone()
    assert call(Q, dict(p, q=q), out=q) is q and torch.equal(q, again)


def test_a_workspace_of_the_largest_sizes_serves_smaller_calls(Q):
    import torch
    for dt in ("f16", "f32"):
        for Hq, Hkv, D in ((8, 2, 128), (12, 1, 64), (4, 4, 256)):
            big = Q.qattn_decode_workspace_bytes(FMT, U.dtype(dt), 64, Hq, Hkv, D, 65536)
            for B in (1, 3, 17, 64):
                for n in (1, 100, 129, 1000, 8192, 40000, 65536):
                    for w in (0, 50, 5000):
                        assert Q.qattn_decode_workspace_bytes(FMT, U.dtype(dt), B, Hq, Hkv, D, n, w) <= big
    assert torch.cuda.is_available()


def test_head_dims_without_a_kernel_are_refused(Q):
    import torch
    kc, vc = Q.qkv_cache(FMT, 2, 16, 1, 160)
    with pytest.raises(Q.QmmError) as e:
        Q.qattn_decode(FMT, torch.zeros((1, 2, 160), device="cuda"), kc, vc, torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                       torch.ones(1, dtype=torch.int32, device="cuda"), 16, 1)
    assert e.value.name == "QMM_ERR_UNIMPLEMENTED"


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,group,page,n", [(128, 4, 32, 100), (64, 8, 16, 100), (128, 16, 64, 32), (96, 1, 8, 128), (256, 2, 32, 77),
                                            (128, 4, 64, 3000)])
@pytest.mark.parametrize("size", [30.0, 1.0, 0.1, 0.03, 0.003])
def test_keys_far_below_one_whose_value_is_zero(Q, dt, D, group, page, n, size):
    """One key takes nearly all of the softmax and has a value of zero: the output is made of
    the others, whose weights are 2^-12 to 2^-88 of its.

    fp32 queries: the plain form's tolerance, of sum |w v|. 16-bit ones: weights are held
    to 2^-25 as 2^14 e^(s - m), and so are their products with V's scale d, of which a block's largest is
    2^-3 or more: 2^-39 (1 / d + 1) of the largest weight and |v|, below 2^-35.8 a key, and
    2^-37 for what an MMA may cut off 24 bits below the largest weight's product: 2^-35."""
    import torch
    p = problem(Q, dt, D, 1, group, page, [n], 3)
    p["q"].fill_(1.0)
    g = torch.Generator(device="cuda").manual_seed(n + D)
    K, V = torch.zeros((n, 1, D), device="cuda"), size * torch.randn((n, 1, D), generator=g, device="cuda")
    K[7], V[7] = 1.0, 0.0
    j = np.arange(n)
    slots = torch.from_numpy(p["host"][0][0, j // page].astype(np.int64) * page + j % page).cuda()
    Q.qkv_store(FMT, K, V, slots, p["kc"], p["vc"], page)
    K, V = (L.q4_values(c, page, 1, D)[slots // page, :, slots % page] for c in (p["kc"], p["vc"]))
    assert bool((K[7] == 1).all()) and bool((V[7] == 0).all())
    if n <= 128:
        assert Q.qattn_decode_splits(FMT, U.dtype(dt), 1, group, 1, D, p["table"].shape[1] * page) == 1
    for below in (12, 20, 24, 28, 32, 33, 40, 56, 75, 88):
        scale = float(np.float32(below * math.log(2) / D))
        out = call(Q, p, scale=scale)
        want, _, tol, _ = U.attend(p["q"][0].double(), K, V, scale, 0.0, dt)
        if dt != "f32":
            tol = tol + n * 2.0 ** -35 * float(V.abs().max())
        err = (out[0].double() - want).abs()
        worst = float((err / tol).max())
        assert worst <= 1, f"2^-{below} of the largest: {worst} of the tolerance"
