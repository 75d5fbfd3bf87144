"""qrmsnorm against its 64-bit plain form: types of input, residual and output,
row sizes from one value to rows no block holds, odd ones and unaligned views,
heads of a projection, Q8_0 rows bit for bit, in place, streams and graphs."""
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


def randn(shape, dt, seed, by=1.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (by * torch.randn(shape, generator=g, device="cuda")).to(U.dtype(dt))


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def check(Q, x, w, residual, out, offset=0.0, eps=1e-6):
    import torch
    r0 = None if residual is None else residual.clone()
    x0 = x.clone()
    y = Q.qrmsnorm(x, w, eps=eps, residual=residual, out_dtype=U.dtype(out), weight_offset=offset)
    assert Q.last_path() == Q.PATH_NORM and y.shape == x.shape and y.dtype == U.dtype(out) and y.is_contiguous()
    want, _ = L.norm(f64(x), f64(r0), f64(w), offset, eps)
    assert np.all(np.abs(f64(y) - want) <= L.norm_tol(want, out))
    assert torch.equal(x, x0)
    if residual is not None:                 # the fp32 sum, rounded once: bit for bit
        assert torch.equal(residual, (x.float() + r0.float()).to(residual.dtype))
    return y


@pytest.mark.parametrize("x,r,out", [(a, b, c) for a in U.UNIT for b in [None, *U.UNIT] for c in U.UNIT])
@pytest.mark.parametrize("T,D", [(3, 4096), (5, 200), (2, 77)])
def test_types(Q, x, r, out, T, D):
    check(Q, randn((T, D), x, D), randn((D,), "f32", 1), None if r is None else randn((T, D), r, 2, 3.0), out)


@pytest.mark.parametrize("T,D", [(1, 1), (7, 2), (3, 8), (40, 24), (1, 31), (2, 33), (9, 255), (4, 256), (4, 264), (1, 511), (3, 513),
                                 (300, 512), (2, 1000), (1, 2048), (3, 4639), (2, 5120), (2, 8191), (1, 8200), (1, 16384),
                                 (1, 20001), (2, 32768), (1, 40000), (1, 100003), (1, 1 << 18)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_sizes(Q, T, D, dt):
    check(Q, randn((T, D), dt, D), randn((D,), "f32", 1) * 0.2, randn((T, D), dt, 2), "f32", offset=1.0)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,H,D,pad", [(1, 1, 128, 0), (5, 40, 128, 0), (3, 7, 80, 8), (2, 3, 96, 1), (4, 5, 64, 3), (301, 9, 192, 0),
                                       (6, 2, 256, 0), (2, 4, 3000, 8)])
def test_heads_of_a_projection(Q, dt, T, H, D, pad):
    """Strided rows, aligned and not; in place on the view nothing beside it changes."""
    import torch
    buf = randn((T, H + 2, D + pad), dt, T + D)
    x = buf[:, 1:1 + H, pad // 2: pad // 2 + D]
    w = randn((D,), "f32", 3)
    y = check(Q, x, w, None, dt)
    res = randn((T, H, D + pad), "f32", 4)[..., :D]
    check(Q, x, w, res, dt)
    before = buf.clone()
    # sums go in another order where the arrays' rows begin unalike: both are within the tolerance
    want, _ = L.norm(f64(x), None, f64(w), 0.0, 1e-6)
    assert Q.qrmsnorm(x, w, out=x) is x
    assert np.all(np.abs(f64(x) - want) <= L.norm_tol(want, dt))
    x.copy_(before[:, 1:1 + H, pad // 2: pad // 2 + D])
    assert torch.equal(buf, before)
    # an output that is a view
    to = torch.full((T, H, 2 * D), 7.0, dtype=U.dtype(dt), device="cuda")
    Q.qrmsnorm(x, w, out=to[..., D:])
    assert np.all(np.abs(f64(to[..., D:]) - want) <= L.norm_tol(want, dt)) and bool((to[..., :D] == 7).all())
    assert torch.equal(y, Q.qrmsnorm(x, w))


@pytest.mark.parametrize("x,r,out", [("f32", None, "f16"), ("bf16", "f32", "bf16"), ("f16", "bf16", "f32"), ("bf16", "bf16", "bf16")])
@pytest.mark.parametrize("T,D,off", [(5, 33, 0), (700, 35, 1), (9, 63, 5), (4000, 129, 0), (3, 257, 7), (800, 511, 2), (6, 1001, 3),
                                     (700, 1001, 0), (5, 4639, 6), (700, 4639, 1), (3, 8191, 4), (2, 32763, 1), (1, 40001, 3)])
def test_rows_of_odd_sizes(Q, x, r, out, T, D, off):
    """Rows that begin anywhere on the 16-byte grid, alike in all arrays: contiguous
    ones of odd sizes, from an offset on; nothing beside them changes."""
    import torch
    n = T * D
    X, w = randn((n + 16,), x, D)[off:off + n].view(T, D), randn((D,), "f32", 1)
    R = None if r is None else randn((n + 16,), r, 2, 3.0)
    r0 = None if r is None else R.clone()
    Y = torch.full((n + 16,), 7.0, dtype=U.dtype(out), device="cuda")
    Q.qrmsnorm(X, w, residual=None if r is None else R[off:off + n].view(T, D), out=Y[off:off + n].view(T, D))
    want, _ = L.norm(f64(X), None if r is None else f64(r0[off:off + n].view(T, D)), f64(w), 0.0, 1e-6)
    assert np.all(np.abs(f64(Y[off:off + n].view(T, D)) - want) <= L.norm_tol(want, out))
    assert bool((Y[:off] == 7).all() and (Y[off + n:] == 7).all())
    if r is not None:
        r0[off:off + n] = (X.float() + r0[off:off + n].view(T, D).float()).to(U.dtype(r)).view(-1)
        assert torch.equal(R, r0)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,D,pad", [(1, 32, 0), (3, 64, 0), (5, 288, 0), (2, 512, 0), (1, 544, 0), (700, 2048, 0), (2, 4096, 8),
                                     (3, 1056, 1), (2, 8192, 0), (1, 33024, 0), (2, 65568, 0), (1, 40992, 3)])
def test_q8_0_rows(Q, dt, T, D, pad):
    """The bytes are the blocks of the fp32 output, by definition, and qdequant reads them."""
    import torch
    x, w = randn((T, D + pad), dt, D)[:, pad:], randn((D,), "f32", 1)
    x[0, :32] = 0
    y = check(Q, x, w, None, "f32")
    rows = Q.qrmsnorm(x, w, out_dtype="q8_0")
    assert rows.dtype == torch.uint8 and rows.shape == (T, D // 32 * 34)
    want = L.blocks_q8(y.cpu().numpy())
    assert np.array_equal(rows.cpu().numpy(), want)
    # in a larger buffer, at an address of no more than 2 bytes' alignment
    buf = torch.full((T, want.shape[1] + 6), 0x55, dtype=torch.uint8, device="cuda")
    Q.qrmsnorm(x, w, out=buf[:, 2:2 + want.shape[1]])
    got = buf.cpu().numpy()
    assert np.array_equal(got[:, 2:-4], want) and (got[:, :2] == 0x55).all() and (got[:, -4:] == 0x55).all()
    vals = Q.qdequant("Q8_0", rows, T, D).cpu().numpy()
    step = np.abs(y.cpu().numpy().reshape(T, -1, 32)).max(-1) / 127
    assert np.all(np.abs(vals - y.cpu().numpy()).reshape(T, -1, 32) <= (step * (0.5 + 128 * 2.0 ** -11) + 2.0 ** -24)[..., None])


def test_q8_0_rows_as_weights_of_a_product(Q):
    """Normed rows kept as blocks, scored against queries by the quantized product."""
    import torch
    T, D, N = 96, 512, 3
    x, w = randn((T, D), "f32", 1), randn((D,), "f32", 2)
    rows = Q.qrmsnorm(x, w, out_dtype="q8_0")
    q = randn((N, D), "f32", 3)
    got = f64(Q.qgemm("Q8_0", rows, q, T, D, N))
    vals = f64(Q.qdequant("Q8_0", rows, T, D))
    want = f64(q) @ vals.T
    assert np.all(np.abs(got - want) <= 1e-3 * (np.abs(f64(q)) @ np.abs(vals).T) + 1e-6)


def test_values_at_the_ends_of_the_range(Q):
    import torch
    D = 256
    x = torch.zeros((7, D), device="cuda")
    x[1] = 1e-30                              # eps decides
    x[2, 3], x[3, 9] = math.inf, math.nan
    x[4] = 1e18                               # squares near the top of fp32
    x[5] = 1e30                               # squares past it
    x[6, 0] = 1e4                             # one large value
    y = f64(Q.qrmsnorm(x, None))
    want, _ = L.norm(f64(x)[[0, 1, 4, 6]], None, None, 0.0, 1e-6)
    assert np.all(np.abs(y[[0, 1, 4, 6]] - want) <= L.norm_tol(want, "f32"))
    assert np.isnan(y[2, 3]) and np.isnan(y[3]).all() and (y[5] == 0).all()
    b = Q.qdequant("Q8_0", Q.qrmsnorm(x, None, out_dtype="q8_0"), 7, D).cpu().numpy()
    assert np.isnan(b[2, :32]).all() and np.isnan(b[3]).all() and (b[0] == 0).all()


def test_the_sum_goes_elsewhere(Q):
    import torch
    x, r, w = randn((9, 640), "f16", 1), randn((9, 640), "f32", 2), randn((640,), "f32", 3)
    r0, to = r.clone(), torch.full((9, 650), 3.0, device="cuda")
    y = Q.qrmsnorm(x, w, residual=r, residual_out=to[:, :640])
    assert torch.equal(r, r0) and torch.equal(to[:, :640], x.float() + r) and bool((to[:, 640:] == 3).all())
    assert torch.equal(y, Q.qrmsnorm(x, w, residual=r.clone()))
    a = randn((9, 640), "f32", 4)             # into X's place
    want = Q.qrmsnorm(a, w, residual=r.clone())
    s = a + r
    assert torch.equal(Q.qrmsnorm(a, w, residual=r, residual_out=a), want) and torch.equal(a, s) and torch.equal(r, r0)
    one = randn((640,), "f32", 5).expand(9, 640)       # one row added to all
    assert torch.equal(Q.qrmsnorm(x, w, residual=one, residual_out=to[:, :640]),
                       Q.qrmsnorm(x, w, residual=one.contiguous()))


def test_refusals(Q):
    import torch
    x, w = randn((4, 64), "f16", 1), randn((64,), "f32", 2)
    r = randn((4, 64), "f32", 3)
    for call, kind in (
            (lambda: Q.qrmsnorm(x.double(), w), TypeError), (lambda: Q.qrmsnorm(x[0], w), ValueError),
            (lambda: Q.qrmsnorm(x.t(), w), ValueError), (lambda: Q.qrmsnorm(x, w.half()), ValueError),
            (lambda: Q.qrmsnorm(x, w[:63]), ValueError), (lambda: Q.qrmsnorm(x, w.cpu()), ValueError),
            (lambda: Q.qrmsnorm(x, w, residual=r[:3]), ValueError), (lambda: Q.qrmsnorm(x, w, residual_out=r), ValueError),
            (lambda: Q.qrmsnorm(x, w, residual=r, residual_out=r.half()), ValueError),
            (lambda: Q.qrmsnorm(x, w, out=x.float(), out_dtype=torch.float16), ValueError),
            (lambda: Q.qrmsnorm(x, w, out_dtype="q4_0"), TypeError), (lambda: Q.qrmsnorm(x, w, eps="a"), TypeError)):
        with pytest.raises(kind):
            call()
    buf = randn((8, 64), "f16", 4)
    wide = randn((4, 128), "f32", 5)
    for call, name in (
            (lambda: Q.qrmsnorm(x, w, eps=-1.0), "QMM_ERR_BAD_ARGUMENT"),
            (lambda: Q.qrmsnorm(buf[:4], w, out=buf[1:5]), "QMM_ERR_BAD_ARGUMENT"),
            (lambda: Q.qrmsnorm(x, w, out=buf[:1].expand(4, 64)), "QMM_ERR_BAD_ARGUMENT"),
            (lambda: Q.qrmsnorm(r, w, residual=r, residual_out=r, out=r), "QMM_ERR_BAD_ARGUMENT"),
            (lambda: Q.qrmsnorm(x, w, residual=r[:1].expand(4, 64)), "QMM_ERR_BAD_ARGUMENT"),
            (lambda: Q.qrmsnorm(wide[:, :64], w, out=wide[:, 32:96]), "QMM_ERR_BAD_ARGUMENT"),
            (lambda: Q.qrmsnorm(x[:, :40], None, out_dtype="q8_0"), "QMM_ERR_COLS_NOT_BLOCK_ALIGNED"),
            (lambda: Q.qrmsnorm(x[:0], w), "QMM_ERR_EMPTY_SHAPE")):
        with pytest.raises(Q.QmmError) as e:
            call()
        assert e.value.name == name
    Q.qrmsnorm(wide[:, :64], w, out=wide[:, 64:])       # rows beside one another
    assert Q.check_device_error() == 0


def test_on_another_stream_and_in_a_graph(Q):
    import torch
    x, r, w = randn((33, 1536), "bf16", 1), randn((33, 1536), "f32", 2), randn((1536,), "f32", 3)
    r0 = r.clone()
    want = Q.qrmsnorm(x, w, residual=r)
    after = r.clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    r.copy_(r0)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        got = Q.qrmsnorm(x, w, residual=r)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(r, after)
    r.copy_(r0)
    torch.cuda.synchronize()
    got = Q.qrmsnorm(x, w, residual=r, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Q.qrmsnorm(x, w, residual=r, out=out)
        Q.qrmsnorm(out, w, out=out)
    r.copy_(r0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(r, after) and torch.equal(out, Q.qrmsnorm(want, w))


@pytest.mark.parametrize("out", ["f32", "f16", "q8_0"])
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("T,D,pad", [(5, 64, 0), (5, 256, 0), (5, 1024, 0), (5, 4096, 0), (700, 2048, 0), (3, 40960, 0), (2, 70016, 0), (5, 4640, 1)])
def test_an_infinite_value_takes_its_row(Q, out, res, T, D, pad):
    """h / sqrt(mean h^2): an Inf makes its own element NaN and the others zeros, in Q8_0 rows its block
    NaN and the others zeros; other rows are as they are without it."""
    import torch
    x = randn((T, D + pad), "f32", D)[:, pad:]
    r = randn((T, D), "f32", 2) if res else None
    to = "q8_0" if out == "q8_0" else U.dtype(out)
    want = Q.qrmsnorm(x, None, residual=None if r is None else r.clone(), out_dtype=to)
    x[1, D - 7] = -math.inf
    y = Q.qrmsnorm(x, None, residual=r, out_dtype=to)
    others = [i for i in range(T) if i != 1]
    assert torch.equal(y[others], want[others])
    if out == "q8_0":
        v = Q.qdequant("Q8_0", y[1:2].contiguous(), 1, D)[0]
        assert bool(torch.isnan(v[D - 32:]).all() and (v[:D - 32] == 0).all())
    else:
        hit = torch.zeros(D, dtype=torch.bool, device="cuda")
        hit[D - 7] = True
        assert torch.equal(torch.isnan(y[1]), hit) and bool((y[1][~hit] == 0).all())
    if r is not None:
        assert float(r[1, D - 7]) == -math.inf
