"""qattn_decode against the 64-bit plain form (tests/kv_util.py): cache formats,
activation types, head dims and groups, page sizes, lengths around every tile
and page edge, windows, softcaps; garbage outside the range, empty sequences,
bad tables and lengths, splits, determinism, streams and graphs."""
import math

import numpy as np
import pytest

from tests import kv_util as U

pytestmark = pytest.mark.gpu

EDGES = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 200, 1000]


@pytest.fixture(scope="module")
def Q():
    import torch  # noqa: F401
    from gemv_mul_mm_gb300 import build as qbuild
    from gemv_mul_mm_gb300 import qmm
    qbuild.build()
    return qmm


def problem(Q, fmt, dt, D, Hkv, group, page, lens, seed, qscale=1.5, garbage=True):
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
        for j in range(lens[b]):
            used[table[b, j // page], j % page] = True
        at += n
    g = torch.Generator(device="cuda").manual_seed(seed)
    kc, vc = Q.qkv_cache(fmt, len(order), page, Hkv, D)
    pg, row = np.nonzero(used)
    if len(pg):
        slots = torch.from_numpy(pg.astype(np.int64) * page + row).cuda()
        K = torch.randn((len(pg), Hkv, D), generator=g, device="cuda")
        V = torch.randn((len(pg), Hkv, D), generator=g, device="cuda") + 0.3
        Q.qkv_store(fmt, K, V, slots, kc, vc, page)
    if garbage:
        pg, row = np.nonzero(~used)
        slots = torch.from_numpy(pg.astype(np.int64) * page + row).cuda()
        bad = torch.full((len(pg), Hkv, D), math.nan, device="cuda")
        Q.qkv_store(fmt, bad, bad, slots, kc, vc, page)
    q = (qscale * torch.randn((len(lens), Hkv * group, D), generator=g, device="cuda")).to(U.dtype(dt))
    return dict(fmt=fmt, dt=dt, page=page, Hkv=Hkv, D=D, q=q, kc=kc, vc=vc, table=torch.from_numpy(table).cuda(),
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), host=(table, lens))


def call(Q, p, **kw):
    return Q.qattn_decode(p["fmt"], p["q"], p["kc"], p["vc"], p["table"], p["lens"], p["page"], p["Hkv"], **kw)


def check(Q, p, window=0, softcap=0.0, scale=None, **kw):
    import torch
    out, lse = call(Q, p, window=window, softcap=softcap, scale=scale, return_lse=True, **kw)
    assert Q.last_path() == Q.PATH_ATTN and Q.check_device_error() == 0
    assert out.dtype == p["q"].dtype and lse.dtype == torch.float32
    table, lens = p["host"]
    kv = [U.cache_values(p["fmt"], c, p["page"], p["Hkv"], p["D"]) for c in (p["kc"], p["vc"])]
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


@pytest.mark.parametrize("fmt", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("Hkv,group,page", [(2, 4, 16), (1, 13, 8)])
def test_lengths_at_every_edge(Q, fmt, dt, D, Hkv, group, page):
    check(Q, problem(Q, fmt, dt, D, Hkv, group, page, EDGES, D + group))


@pytest.mark.parametrize("fmt", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("group,page,window", [(4, 16, 0), (11, 8, 0), (2, 32, 50)])
def test_head_dim_192(Q, fmt, dt, group, page, window):
    check(Q, problem(Q, fmt, dt, 192, 2, group, page, EDGES + [9000], group), window)


@pytest.mark.parametrize("fmt,dt", [("f16", "f16"), ("bf16", "bf16"), ("q8_0", "f32")])
@pytest.mark.parametrize("Hkv,group", [(1, 1), (3, 1), (5, 7), (2, 8), (1, 9), (2, 16), (1, 17), (1, 40)])
def test_head_groups(Q, fmt, dt, Hkv, group):
    check(Q, problem(Q, fmt, dt, 128, Hkv, group, 32, [77, 300, 5], group))


@pytest.mark.parametrize("fmt,dt,D", [("f16", "f32", 128), ("bf16", "f16", 64), ("q8_0", "bf16", 96), ("q8_0", "f16", 256)])
@pytest.mark.parametrize("page", [8, 16, 64, 512])
@pytest.mark.parametrize("window,softcap", [(1, 0.0), (13, 0.0), (16, 30.0), (100, 0.0), (5000, 2.0), (0, 10.0)])
def test_windows_softcaps_and_pages(Q, fmt, dt, D, page, window, softcap):
    check(Q, problem(Q, fmt, dt, D, 2, 3, page, [0, 1, 14, 16, 100, 117, 513, 1500], page + window), window, softcap)


@pytest.mark.parametrize("fmt,dt,D,group", [("f16", "f16", 128, 4), ("q8_0", "f32", 128, 8), ("bf16", "bf16", 64, 2),
                                            ("q8_0", "f16", 96, 12), ("f16", "bf16", 256, 1)])
def test_long_sequences_are_split_and_joined(Q, fmt, dt, D, group):
    import torch
    p = problem(Q, fmt, dt, D, 1, group, 64, [30011, 20000, 129], 3)
    need = Q.qattn_decode_workspace_bytes(fmt, U.dtype(dt), 3, group, 1, D, p["table"].shape[1] * 64)
    assert need > 0
    a = check(Q, p)
    # deterministic, whatever the workspace held; the caller's workspace of just
    # the size asked for
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    b = call(Q, p, return_lse=True, workspace=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(Q.QmmError) as e:
        call(Q, p, workspace=ws[:-16])
    assert e.value.name == "QMM_ERR_WORKSPACE_TOO_SMALL"


def test_many_sequences_are_not_split_below_their_need(Q):
    check(Q, problem(Q, "q8_0", "f16", 128, 2, 4, 16, [int(v) for v in np.random.RandomState(1).randint(0, 700, 150)], 4))


@pytest.mark.parametrize("fmt,dt", [("f16", "f16"), ("q8_0", "f16"), ("bf16", "f32"), ("q8_0", "f32")])
def test_one_long_sequence_among_many_short_ones(Q, fmt, dt):
    """A batch large enough that nothing has to be split to fill the GPU: the
    sums over a long sequence keep their accuracy all the same. Against the
    result's 2-norm: 16-bit outputs their own rounding and the 2^-16 of the
    weights, fp32 outputs the score error 2.5 delta of the derived tolerance,
    of which a sum over many keys shows far less (2e-6)."""
    lens = [1 + i % 3 for i in range(300)] + [40000]
    p = problem(Q, fmt, dt, 64, 2, 2, 64, lens, 11)
    out, _ = check(Q, p)
    table = p["host"][0]
    import torch
    j = np.arange(lens[-1])
    pg, row = torch.from_numpy(table[-1, j // 64].astype(np.int64)).cuda(), torch.from_numpy(j % 64).cuda()
    K, V = (U.cache_values(fmt, c, 64, 2, 64)[pg, :, row] for c in (p["kc"], p["vc"]))
    want = U.attend(p["q"][-1].double(), K, V, 0.125, 0.0, dt)[0]
    rel = float((out[-1].double() - want).norm() / want.norm())
    assert rel < (2e-6 if dt == "f32" else 2.0 ** -11 + 2.0 ** -16)


def test_strided_query_and_explicit_scale(Q):
    import torch
    p = problem(Q, "f16", "f16", 64, 2, 2, 16, [50, 3], 8)
    big = torch.zeros((2, 9, 64 + 8), dtype=torch.float16, device="cuda")
    view = big[:, 3:7, 4:68]                       # 8-byte aligned rows
    view.copy_(p["q"])
    p["q"] = view
    check(Q, p, scale=0.03)


@pytest.mark.parametrize("qscale", [1e-4, 40.0, 3000.0])
def test_sharp_and_flat_softmax(Q, qscale):
    """One key takes all the weight, or all share it; scores up to thousands."""
    for fmt, dt in (("f16", "f32"), ("q8_0", "f32"), ("bf16", "f32"), ("f16", "bf16"), ("q8_0", "f16")):
        check(Q, problem(Q, fmt, dt, 128, 1, 4, 16, [333, 40], 9, qscale=qscale))


def test_rising_scores_move_the_maximum_every_tile(Q):
    import torch
    p = problem(Q, "f16", "f16", 64, 1, 1, 16, [400], 5)
    slots = torch.from_numpy((p["host"][0][0, np.arange(400) // 16].astype(np.int64) * 16 + np.arange(400) % 16)).cuda()
    K = torch.zeros((400, 1, 64), device="cuda")
    K[:, 0, 0] = torch.linspace(-60, 60, 400, device="cuda")
    p["q"].zero_()
    p["q"][:, :, 0] = 8.0
    V = torch.randn((400, 1, 64), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    Q.qkv_store("f16", K, V, slots, p["kc"], p["vc"], 16)
    check(Q, p)


def test_keys_of_minus_infinity_are_masked_and_all_of_them_give_nan(Q):
    import torch
    p = problem(Q, "f16", "f16", 64, 1, 1, 16, [40, 20], 5)
    vals = p["kc"].view(torch.float16).view(-1, 1, 16, 64)
    p["q"].fill_(1.0)
    table = p["host"][0]
    vals[int(table[0, 1]), 0, 4, 0] = -math.inf                       # one key of the first sequence
    for j in range(20):
        vals[int(table[1, j // 16]), 0, j % 16, 0] = -math.inf        # every key of the second
    out, lse = call(Q, p, return_lse=True)
    K, V = (U.cache_values("f16", c, 16, 1, 64) for c in (p["kc"], p["vc"]))
    j = np.array([i for i in range(40) if i != 20])
    pg, row = torch.from_numpy(table[0, j // 16].astype(np.int64)).cuda(), torch.from_numpy(j % 16).cuda()
    want, wl, tol, ltol = U.attend(p["q"][0].double(), K[pg, :, row], V[pg, :, row], 0.125, 0.0, "f16")
    assert bool(((out[0].double() - want).abs() <= tol).all()) and bool(((lse[0].double() - wl).abs() <= ltol).all())
    assert bool(torch.isnan(out[1]).all()) and bool((lse[1] == -math.inf).all())
    assert Q.check_device_error() == 0


def test_enormous_scores(Q):
    """Scores near the ends of fp32's range: no reference value of the softmax
    is mistaken for them."""
    import torch
    p = problem(Q, "bf16", "f32", 64, 1, 2, 16, [100], 3)
    p["q"].mul_(1e34)
    out, lse = call(Q, p, return_lse=True)
    K, V = (U.cache_values("bf16", c, 16, 1, 64) for c in (p["kc"], p["vc"]))
    j = np.arange(100)
    pg, row = torch.from_numpy(p["host"][0][0, j // 16].astype(np.int64)).cuda(), torch.from_numpy(j % 16).cuda()
    s = torch.einsum("hd,nd->hn", p["q"][0].double(), K[pg, 0, row]) * 0.125
    best = s.argmax(-1)                                               # scores lie 1e33 apart: one key takes all
    assert bool(((out[0].double() - V[pg, 0, row][best]).abs() <= 2.0 ** -22 * V[pg, 0, row][best].abs() + 1e-30).all())
    assert bool(((lse[0].double() / s.amax(-1) - 1).abs() < 1e-5).all())


def test_nan_in_one_sequence_stays_there(Q):
    import torch
    p = problem(Q, "bf16", "bf16", 64, 2, 2, 16, [40, 33], 6)
    p["q"][0, 1, 3] = math.nan
    out = call(Q, p)
    assert bool(torch.isnan(out[0, 1]).all())
    out[0, 1] = 0
    assert bool(torch.isfinite(out).all())


def test_bad_pages_and_lengths(Q):
    import torch
    bad_slot = Q.STATUS_ID["QMM_ERR_BAD_SLOT"]
    for lens in ([40, 33, 20], [9000, 12000, 20]):                    # whole and split sequences
        p = problem(Q, "f16", "f16", 64, 1, 2, 16, lens, 7)
        good = call(Q, p)
        for wrong in (-1, p["kc"].shape[0], 2 ** 31 - 1):
            t = p["table"].clone()
            t[1, 1] = wrong
            out, lse = call(Q, {**p, "table": t}, return_lse=True)
            assert Q.check_device_error() == bad_slot
            assert bool(torch.isnan(out[1]).all()) and bool(torch.isnan(lse[1]).all())
            assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
        for wrong in (-5, p["table"].shape[1] * 16 + 1, 2 ** 31 - 1, -2 ** 31):
            n = p["lens"].clone()
            n[0] = wrong
            out = call(Q, {**p, "lens": n})
            assert Q.check_device_error() == bad_slot
            assert bool(torch.isnan(out[0]).all()) and torch.equal(out[1:], good[1:])
    out = call(Q, p, max_len=10000)                                   # 12000 is beyond the caller's own bound
    assert Q.check_device_error() == bad_slot
    assert bool(torch.isnan(out[1]).all()) and not bool(torch.isnan(out[0]).any())


def test_streams_and_graphs(Q):
    import torch
    p = problem(Q, "q8_0", "f16", 128, 2, 4, 16, [5000, 70, 0], 8)
    want = call(Q, p)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = call(Q, p)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(p["q"])
    ws = torch.empty(Q.qattn_decode_workspace_bytes("q8_0", torch.float16, 3, 8, 2, 128, p["table"].shape[1] * 16),
                     dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(Q, p, out=out, workspace=ws)
    for lens in ([5000, 70, 0], [17, 4000, 1]):                       # lengths are read on the device
        p["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        if lens[1] == 4000:
            p["table"][1] = p["table"][0]
            p["table"][2, 0] = p["table"][0, 3]
        out.fill_(7)
        g.replay()
        assert torch.equal(out, call(Q, p))
    assert Q.check_device_error() == 0


def test_stream_given_by_handle_does_not_share_memory_with_the_current_one(Q):
    """Outputs and workspaces of a call on another stream come from that
    stream's memory: work on the current stream, which allocates and fills
    blocks of the same sizes all the time, does not touch them."""
    import torch
    p = problem(Q, "f16", "f16", 128, 1, 8, 64, [30000, 300], 4)
    want = call(Q, p)
    need = Q.qattn_decode_workspace_bytes("f16", torch.float16, 2, 8, 1, 128, p["table"].shape[1] * 64)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    for _ in range(50):
        got.append(call(Q, p, stream=side.cuda_stream))
        for size in (need, want.numel() * 2):                         # what a freed block would be handed out to
            torch.full((size,), 0xff, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    with torch.cuda.stream(side):                                     # and the default stream from another one
        y = call(Q, p, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_back_to_back_calls_share_a_workspace_on_one_stream(Q):
    import torch
    p, r = (problem(Q, "f16", "f16", 128, 1, 8, 64, [n, 300], s) for n, s in ((9000, 1), (7000, 2)))
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    want = [call(Q, x) for x in (p, r)]
    for _ in range(20):
        got = [call(Q, x, workspace=ws) for x in (p, r)]
    assert all(torch.equal(a, b) for a, b in zip(got, want))
