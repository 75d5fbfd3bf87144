"""qmoe_route against its 64-bit plain form: ids equal, weights to fp32; scores,
biases, groups, expert counts, ties, values that fp32 cannot tell apart, infinite
and NaN logits, streams and graphs, and the layer that takes its outputs."""
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


def randn(shape, dt, seed, by=1.5):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (by * torch.randn(shape, generator=g, device="cuda")).to(U.dtype(dt))


def check(Q, x, k, score="softmax", bias=None, groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0):
    import torch
    ids, w = Q.qmoe_route(x, k, score=score, bias=bias, groups=groups, top_groups=top_groups, group_top=group_top, renorm=renorm,
                          scale=scale)
    assert Q.last_path() == Q.PATH_ROUTE and ids.dtype == torch.int32 and w.dtype == torch.float32
    assert ids.shape == w.shape == (x.shape[0], k)
    want, ww, _ = L.route(x.double().cpu().numpy(), k, score, None if bias is None else bias.cpu().numpy(), groups, top_groups,
                          group_top, renorm, scale)
    assert np.array_equal(ids.cpu().numpy(), want)
    # exponentials and quotients to 2 ulp each, x - top rounded (at most 2^-24 of 100 or so,
    # in the exponent), a sum of up to 32 (all E: 37 steps) terms, the scale
    err = np.abs(w.double().cpu().numpy() - ww)
    most = x[torch.isfinite(x)].double().abs().max().item() if bool(torch.isfinite(x).any()) else 0.0
    assert np.all(err <= np.abs(ww) * 2.0 ** -24 * (80 + 2 * most) + 2.0 ** -126)
    return ids, w


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,k,groups,top_groups,group_top", [
    (128, 8, 1, 1, 1), (256, 8, 8, 4, 2), (64, 6, 8, 3, 1), (160, 6, 8, 3, 1), (160, 6, 8, 3, 2), (8, 2, 1, 1, 1), (1, 1, 1, 1, 1),
    (7, 7, 1, 1, 1), (45, 4, 3, 2, 2), (33, 32, 1, 1, 1), (512, 10, 16, 5, 2), (1000, 32, 4, 1, 2), (1024, 8, 32, 32, 2),
    (384, 8, 1, 1, 1), (64, 4, 32, 2, 2)])
def test_forms(Q, dt, score, biased, E, k, groups, top_groups, group_top):
    import torch
    for T, renorm in ((1, True), (77, False), (700, True)):
        bias = 0.2 * randn((E,), "f32", E) if biased else None
        check(Q, randn((T, E), dt, T + E), k, score, bias, groups, top_groups, group_top, renorm, 2.5)
    # rows of a wider product, unaligned
    x = randn((19, E + 3), dt, 5)[:, 1:1 + E]
    check(Q, x, k, score, bias, groups, top_groups, group_top)
    assert not torch.equal(x[0], x[1])


def test_many_tokens(Q):
    check(Q, randn((20000, 256), "f32", 1), 8, "sigmoid", 0.1 * randn((256,), "f32", 2), 8, 4, 2, True, 2.5)
    check(Q, randn((20000, 128), "bf16", 3), 8)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("E,k,groups,top_groups,group_top,score,biased", [
    (128, 8, 1, 1, 1, "softmax", False), (64, 6, 1, 1, 1, "sigmoid", True), (128, 8, 4, 2, 2, "softmax", True),
    (256, 8, 8, 4, 2, "sigmoid", True), (256, 1, 8, 1, 1, "softmax", False), (192, 7, 2, 1, 2, "sigmoid", False),
    (160, 5, 5, 3, 2, "softmax", True), (48, 8, 3, 2, 1, "sigmoid", False), (40, 3, 1, 1, 1, "softmax", True)])
def test_batches_of_four_tokens_a_warp(Q, dt, E, k, groups, top_groups, group_top, score, biased):
    """Large calls, not a multiple of four tokens, with rows of equal values among them."""
    import torch
    x = randn((9731, E), dt, E)
    x[17::501] = 0
    x[40::333, ::3] = x[40::333, :1]
    check(Q, x, k, score, 0.2 * randn((E,), "f32", 2) if biased else None, groups, top_groups, group_top)


@pytest.mark.parametrize("times", [1, 300])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top_groups,group_top,k", [(64, 1, 1, 1, 8), (64, 8, 4, 2, 8), (96, 4, 2, 1, 5), (1024, 1, 1, 1, 32),
                                                             (256, 8, 3, 2, 32), (256, 8, 3, 2, 8)])
def test_equal_values_go_to_the_lower_index(Q, score, E, groups, top_groups, group_top, k, times):
    import torch
    if times > 1 and E == 1024:
        times = 3
    x = torch.zeros((40, E), device="cuda")                         # padded rows: all equal
    g = torch.Generator(device="cuda").manual_seed(E)
    x[10:20] = torch.randint(0, 2, (10, E), generator=g, device="cuda").float()
    x[20:30] = torch.randint(-3, 3, (10, E), generator=g, device="cuda").float()
    x[30:, : E // 2], x[30:35, E // 2:] = -0.0, 0.0
    x = x.repeat(times, 1)
    for bias in (None, torch.zeros(E, device="cuda"), torch.full((E,), 0.25, device="cuda"),
                 torch.randint(0, 2, (E,), generator=g, device="cuda").float()):
        check(Q, x, k, score, bias, groups, top_groups, group_top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_top", [1, 2])
def test_values_that_fp32_cannot_tell_apart(Q, score, group_top):
    """Biases that bring scores within a few 2^-24 of one another, in exact
    arithmetic on either side: the ids are those of the real numbers."""
    import torch
    E, T = 64, 200
    x = randn((T, E), "f32", 7)
    for t in range(0, T, 10):
        xs = x[t].double().cpu().numpy()
        s = 1 / (1 + np.exp(-xs)) if score == "sigmoid" else np.exp(xs) / np.exp(xs).sum()
        bias = torch.from_numpy((1.0 - s).astype(np.float32)).cuda()   # every c within 2^-24 of 1
        check(Q, x[t:t + 1], 8, score, bias)
        check(Q, x[t:t + 1], 8, score, bias, 8, 4, group_top)
        check(Q, x[t:t + 10], 8, score, bias, 4, 2, group_top)
        if t % 50 == 0:                                             # four tokens a warp
            many = x[t:t + 1].expand(8000, -1) + 0.0
            check(Q, many, 8, score, bias)
            check(Q, many, 8, score, bias, 4, 2, group_top)


@pytest.mark.parametrize("times", [1, 1000])
def test_infinite_and_nan_logits(Q, times):
    import torch
    inf, nan = math.inf, math.nan
    x = randn((8, 40), "f32", 1)
    x[0, 5:] = -inf                                                 # fewer finite logits than chosen
    x[1] = -inf
    x[2, 7] = x[2, 3] = inf
    x[3, 30] = nan
    x[4] = nan
    x[5, ::2] = -inf
    x[6] = -200.0                                                   # sigmoids of all zero in fp32
    x = x.repeat(times, 1)
    for score in ("softmax", "sigmoid"):
        for bias in (None, 0.1 * randn((40,), "f32", 2)):
            for groups in (1, 4):
                ids, w = Q.qmoe_route(x, 8, score=score, bias=bias, groups=groups, top_groups=2 if groups > 1 else 1,
                                      group_top=2 if groups > 1 else 1)
                i = ids.cpu().numpy()
                assert i.min() >= 0 and i.max() < 40 and all(len(set(r)) == 8 for r in i)
                assert bool(torch.isfinite(w[7]).all() and torch.isfinite(w[5]).all() and torch.isfinite(w[0]).all())
                # all zero scores (chosen in a kept group or not)
                assert bool((w[1] == 0).all())
                assert bool(torch.isnan(w[4]).all())
    for score in ("softmax", "sigmoid"):
        check(Q, x[[0, 1, 5, 7]], 8, score)
        check(Q, x[[0, 1, 5, 7]], 8, score, 0.1 * randn((40,), "f32", 2))
        ids, w = Q.qmoe_route(x, 2, score=score)
        assert ids[2].tolist() == [3, 7] and int(ids[3, 0]) == 30
        assert bool(torch.isnan(w[3]).all()) and bool(torch.isnan(w[2]).all()) == (score == "softmax")
    bias = torch.zeros(40, device="cuda")
    bias[:30] = -inf                                                # experts switched off
    check(Q, x[[5, 7]], 10, "sigmoid", bias)
    bias[3] = inf
    check(Q, x[[0, 5, 7]], 10, "softmax", bias)


@pytest.mark.parametrize("T", [5, 8002])
@pytest.mark.parametrize("groups,top_groups,group_top", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
@pytest.mark.parametrize("renorm", [True, False])
def test_rows_without_a_finite_logit(Q, T, groups, top_groups, group_top, renorm):
    """A row of only -Inf has scores of zero, also where they are not renormalised."""
    x = randn((T, 64), "f32", 1)
    x[::3] = -math.inf
    for bias in (None, 0.1 * randn((64,), "f32", 2)):
        check(Q, x, 6, "softmax", bias, groups, top_groups, group_top, renorm)


@pytest.mark.parametrize("T", [5, 8002])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("groups,group_top", [(1, 1), (4, 1), (4, 2)])
@pytest.mark.parametrize("renorm", [True, False])
def test_a_softmax_without_a_value_gives_nan_weights(Q, T, bad, groups, group_top, renorm):
    """The infinite or NaN logit makes all of the token's scores NaN, chosen or not."""
    import torch
    x = randn((T, 64), "f32", 1)
    x[1::3, 61] = bad
    for bias in (None, 0.1 * randn((64,), "f32", 2)):
        ids, w = Q.qmoe_route(x, 6, bias=bias, groups=groups, top_groups=min(2, groups), group_top=group_top, renorm=renorm)
        nan = torch.isnan(w)
        assert bool(nan[1::3].all()) and not bool(nan[::3].any()) and not bool(nan[2::3].any())
        i = ids.cpu().numpy()
        assert i.min() >= 0 and i.max() < 64 and all(len(set(r)) == 6 for r in i)


@pytest.mark.parametrize("T", [150, 8002])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("by", [50.0, 3e5])
def test_biases_of_either_sign_that_cancel_in_a_group(Q, T, score, by):
    """The two largest of each group are near by and -by: fp32 has rounded the scores
    in both, the sums of the real numbers are theirs."""
    import torch
    bias = torch.full((64,), -by, device="cuda")
    bias[::8] = by
    check(Q, randn((T, 64), "f32", 3), 4, score, bias, 8, 4, 2)


@pytest.mark.parametrize("T", [3, 8002])
@pytest.mark.parametrize("groups", [1, 2])
@pytest.mark.parametrize("same", [2, 12])
def test_equal_inputs_at_the_border_with_a_larger_value_behind(Q, T, groups, same):
    """Equal inputs take the last place and the next in fp32, and another expert of the same fp32
    value behind them is the larger: 22 + (1 - 9e-14) against 22 + (1 - 4e-8)."""
    import torch
    x = randn((T, 64), "f32", 1)
    bias = torch.zeros(64, device="cuda")
    bias[:7] = 30.0
    bias[10:10 + same] = bias[31] = 22.0
    x[:, 10:10 + same], x[:, 31] = 17.0, 30.0
    ids, _ = check(Q, x, 8, "sigmoid", bias, groups, 1, 2)
    assert bool((ids[:, 7] == 31).all())


def test_sigmoids_below_the_normal_range(Q):
    """Scores of 2^-126 and less, whose sum has no fp32 inverse."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    for T in (7, 8002):
        x = -88.5 + torch.rand((T, 64), generator=g, device="cuda")
        check(Q, x, 2, "sigmoid")
        check(Q, x, 2, "sigmoid", 0.1 * randn((64,), "f32", 2))


def test_refusals(Q):
    import torch
    x = randn((4, 64), "f32", 1)
    b = torch.zeros(64, device="cuda")
    for call, kind in (
            (lambda: Q.qmoe_route(x.double(), 2), TypeError), (lambda: Q.qmoe_route(x[0], 2), ValueError),
            (lambda: Q.qmoe_route(x.t(), 2), ValueError), (lambda: Q.qmoe_route(x, 2, score="other"), KeyError),
            (lambda: Q.qmoe_route(x, 2, bias=b.half()), ValueError), (lambda: Q.qmoe_route(x, 2, bias=b[:9]), ValueError),
            (lambda: Q.qmoe_route(x, -1), ValueError), (lambda: Q.qmoe_route(x, 2, ids=torch.zeros((4, 2), device="cuda")), ValueError),
            (lambda: Q.qmoe_route(x.cpu(), 2), ValueError)):
        with pytest.raises(kind):
            call()
    for kw, name in (
            (dict(top_k=0), "QMM_ERR_EMPTY_SHAPE"), (dict(top_k=65), "QMM_ERR_BAD_ARGUMENT"), (dict(top_k=33), "QMM_ERR_UNIMPLEMENTED"),
            (dict(top_k=2, groups=3), "QMM_ERR_BAD_ARGUMENT"), (dict(top_k=2, groups=0), "QMM_ERR_BAD_ARGUMENT"),
            (dict(top_k=9, groups=8, top_groups=1), "QMM_ERR_BAD_ARGUMENT"), (dict(top_k=2, groups=4, top_groups=5), "QMM_ERR_BAD_ARGUMENT"),
            (dict(top_k=2, groups=64, top_groups=4), "QMM_ERR_UNIMPLEMENTED"), (dict(top_k=2, group_top=3), "QMM_ERR_BAD_ARGUMENT"),
            (dict(top_k=2, groups=64, top_groups=4, group_top=2), "QMM_ERR_BAD_ARGUMENT"),
            (dict(top_k=2, scale=math.inf), "QMM_ERR_BAD_ARGUMENT")):
        with pytest.raises(Q.QmmError) as e:
            Q.qmoe_route(x, **kw)
        assert e.value.name == name
    with pytest.raises(Q.QmmError) as e:
        Q.qmoe_route(x, 2, weights=x.view(-1)[:8])                  # over the logits
    assert e.value.name == "QMM_ERR_BAD_ARGUMENT"
    with pytest.raises(Q.QmmError) as e:
        Q.qmoe_route(torch.zeros((2, 1025), device="cuda"), 2)
    assert e.value.name == "QMM_ERR_UNIMPLEMENTED"


def test_on_another_stream_and_in_a_graph(Q):
    import torch
    x, bias = randn((50, 128), "f16", 1), 0.1 * randn((128,), "f32", 2)
    want = Q.qmoe_route(x, 6, score="sigmoid", bias=bias)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = Q.qmoe_route(x, 6, score="sigmoid", bias=bias)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ids, w = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Q.qmoe_route(x, 6, score="sigmoid", bias=bias, ids=ids, weights=w)
    ids.zero_(), w.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(ids, want[0]) and torch.equal(w, want[1])


def test_experts_take_the_routing(Q, orc):
    """Logits, routing, expert products: the layer of the routed ids against the oracle's."""
    import torch
    from gemv_mul_mm_gb300 import synth
    from tests.gpu_util import dev
    p = synth.moe_layer_problem(8)
    x = dev(p["x"])
    router = randn((p["n_experts"], p["d_model"]), "f32", 4, p["d_model"] ** -0.5)
    ids, w = check(Q, x @ router.T, 8)
    y = Q.qmoe_ffn(p["kind"], dev(p["w_gu"]), p["gu_stride"], dev(p["w_down"]), p["down_stride"], p["n_experts"], x, ids, w,
                   p["d_model"], p["d_ff"])
    assert Q.check_device_error() == 0
    want, tol = orc.moe_ffn(p["kind"], p["w_gu"], p["gu_stride"], p["w_down"], p["down_stride"], p["n_experts"], p["x"],
                            ids.cpu().numpy(), w.cpu().numpy(), p["d_model"], p["d_ff"], nthreads=8)
    assert np.all(np.abs(y.double().cpu().numpy() - want) <= tol)
    assert isinstance(y, torch.Tensor)


@pytest.mark.parametrize("T", [7, 8002])
@pytest.mark.parametrize("E,k,groups,top_groups,group_top", [(64, 2, 1, 1, 1), (64, 8, 1, 1, 1), (64, 6, 4, 2, 2), (128, 8, 8, 3, 1), (45, 9, 3, 2, 2)])
@pytest.mark.parametrize("renorm", [True, False])
def test_sigmoids_whose_exponential_passes_fp32(Q, T, E, k, groups, top_groups, group_top, renorm):
    """Logits below -88.7: the score is not a normal float, and the renormalised weights are its ratios."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    for lo, hi in ((-89.5, -88.0), (-110.0, -60.0), (-690.0, -100.0), (-200.0, 20.0)):
        x = lo + (hi - lo) * torch.rand((T, E), generator=g, device="cuda")
        x[::3, ::2] = -200.0
        x[1::4] = -200.0
        x[2::5, 3:] = -math.inf
        check(Q, x, k, "sigmoid", None, groups, top_groups, group_top, renorm)
        check(Q, x, k, "sigmoid", 0.1 * randn((E,), "f32", 2), groups, top_groups, group_top, renorm)
    x = torch.full((T, E), -1e4, device="cuda")
    ids, w = Q.qmoe_route(x, k, score="sigmoid", groups=groups, top_groups=top_groups, group_top=group_top, renorm=renorm)
    assert bool((w == (1 / k if renorm else 0.0)).all() if k in (2, 8) else ((w - (1 / k if renorm else 0.0)).abs() <= 2.0 ** -24).all())


@pytest.mark.parametrize("T", [5, 8002])
@pytest.mark.parametrize("groups,top_groups,group_top", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
def test_softmax_scores_down_to_the_end_of_64_bits(Q, T, groups, top_groups, group_top):
    """With a bias of zeros the order is that of the scores, e^-703 and less but one."""
    import torch
    x = torch.arange(64, device="cuda", dtype=torch.float32) / 2 - 741.5      # -741.5 .. -710, ascending
    x[:16] = torch.arange(16, device="cuda") * 3.0 - 748.0                    # -748 .. -703
    x[3] = 0.0
    x = x.expand(T, 64) + 0.0
    x[1::2] = x[1::2].flip(1)
    check(Q, x, 6, "softmax", torch.zeros(64, device="cuda"), groups, top_groups, group_top)


@pytest.mark.parametrize("T", [5, 8002])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_that_64_bits_cannot_tell_apart_go_to_the_lower_index(Q, T, score):
    """With a bias, also one of zeros, values are compared in 64 bits: logits of 45 and 50 have the same sigmoid there,
    and scores below 2^-53 of the bias are lost in it. Without one the logits decide."""
    import torch
    x = randn((T, 64), "f32", 3, 0.1)
    if score == "sigmoid":
        x[:, 10:14] = torch.tensor([45.0, 50.0, 60.0, 47.0], device="cuda")
        bias = torch.zeros(64, device="cuda")
    else:
        x[:, 20] = 90.0                                                       # the others' scores: e^-90
        bias = torch.full((64,), 0.5, device="cuda")
    ids, _ = check(Q, x, 3, score, bias)
    assert ids[0].tolist() == ([10, 11, 12] if score == "sigmoid" else [20, 0, 1])
    ids, _ = check(Q, x, 3, score)
    if score == "sigmoid":
        assert ids[0].tolist() == [12, 11, 13]
