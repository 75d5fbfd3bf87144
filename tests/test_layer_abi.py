"""The norm, the router and the q4_0 cache on the CPU: every refusal by name
before a launch (no GPU needed: none of these calls reaches one)."""
import pytest

from gemv_mul_mm_gb300 import build as qbuild
from gemv_mul_mm_gb300 import qmm

FAKE = 0x100000  # never dereferenced: every call below is refused before a launch
FAR = 0x8000000
S = qmm.STATUS_ID


@pytest.fixture(scope="module")
def L():
    qbuild.build()
    return qmm.lib()


def norm(L, **kw):
    a = dict(X=FAKE, xd=1, xn=4 * 64, xt=64, xh=0, R=0, rd=0, rn=0, rt=0, rh=0, RO=0, ron=0, rot=0, roh=0, W=FAR, wn=64, off=0.0,
             eps=1e-6, Y=2 * FAR, yf=1, yn=4 * 64, yt=64, yh=0, T=4, H=1, D=64)
    a.update(kw)
    return L.qrmsnorm(*[a[k] for k in ("X", "xd", "xn", "xt", "xh", "R", "rd", "rn", "rt", "rh", "RO", "ron", "rot", "roh", "W", "wn",
                                       "off", "eps", "Y", "yf", "yn", "yt", "yh", "T", "H", "D")], None)


RES = dict(R=3 * FAR, rd=0, rn=256, rt=64)


@pytest.mark.parametrize("args,status", [
    (dict(xd=3), "QMM_ERR_BAD_DTYPE"), (dict(yf=3), "QMM_ERR_BAD_DTYPE"), (dict(RES, rd=5), "QMM_ERR_BAD_DTYPE"),
    (dict(T=-1), "QMM_ERR_BAD_ARGUMENT"), (dict(T=0), "QMM_ERR_EMPTY_SHAPE"), (dict(D=0), "QMM_ERR_EMPTY_SHAPE"),
    (dict(H=0), "QMM_ERR_EMPTY_SHAPE"), (dict(xt=-1), "QMM_ERR_BAD_ARGUMENT"), (dict(yh=1 << 41), "QMM_ERR_BAD_ARGUMENT"),
    (dict(D=(1 << 20) + 1), "QMM_ERR_BAD_ARGUMENT"), (dict(T=1 << 31), "QMM_ERR_BAD_ARGUMENT"),
    (dict(eps=-1e-6), "QMM_ERR_BAD_ARGUMENT"), (dict(eps=float("nan")), "QMM_ERR_BAD_ARGUMENT"),
    (dict(off=float("inf")), "QMM_ERR_BAD_ARGUMENT"), (dict(RO=4 * FAR, ron=256, rot=64), "QMM_ERR_BAD_ARGUMENT"),
    (dict(X=0), "QMM_ERR_NULL_POINTER"), (dict(Y=0), "QMM_ERR_NULL_POINTER"), (dict(X=FAKE + 1), "QMM_ERR_MISALIGNED"),
    (dict(W=FAR + 2), "QMM_ERR_MISALIGNED"), (dict(yf=0, Y=2 * FAR + 2), "QMM_ERR_MISALIGNED"),
    (dict(yf=16, Y=2 * FAR + 1, yn=4 * 68, yt=68), "QMM_ERR_MISALIGNED"), (dict(yf=16, yn=4 * 69, yt=69), "QMM_ERR_MISALIGNED"),
    (dict(yf=16, D=48, xt=48), "QMM_ERR_COLS_NOT_BLOCK_ALIGNED"), (dict(xn=255), "QMM_ERR_ACTIVATIONS_TOO_SMALL"),
    (dict(wn=63), "QMM_ERR_ACTIVATIONS_TOO_SMALL"), (dict(RES, rn=255), "QMM_ERR_ACTIVATIONS_TOO_SMALL"),
    (dict(yn=255), "QMM_ERR_OUTPUT_TOO_SMALL"), (dict(yf=16, yn=4 * 68 - 1, yt=68), "QMM_ERR_OUTPUT_TOO_SMALL"),
    (dict(RES, RO=4 * FAR, ron=255, rot=64), "QMM_ERR_OUTPUT_TOO_SMALL"),
    # outputs over one another or over inputs
    (dict(yt=63), "QMM_ERR_BAD_ARGUMENT"), (dict(Y=FAKE + 2), "QMM_ERR_BAD_ARGUMENT"), (dict(Y=FAKE, yf=2), "QMM_ERR_BAD_ARGUMENT"),
    (dict(Y=FAR), "QMM_ERR_BAD_ARGUMENT"), (dict(RES, Y=3 * FAR, yf=0), "QMM_ERR_BAD_ARGUMENT"),
    (dict(RES, RO=2 * FAR, ron=256, rot=64), "QMM_ERR_BAD_ARGUMENT"), (dict(RES, RO=FAKE, ron=256, rot=64), "QMM_ERR_BAD_ARGUMENT"),
    (dict(RES, RO=3 * FAR + 4, ron=256, rot=64), "QMM_ERR_BAD_ARGUMENT"), (dict(RES, RO=4 * FAR, ron=256, rot=0), "QMM_ERR_BAD_ARGUMENT"),
    (dict(RES, RO=FAR, ron=256, rot=64), "QMM_ERR_BAD_ARGUMENT")])
def test_norm_refusals(L, args, status):
    assert norm(L, **args) == S[status]


@pytest.mark.parametrize("args,status", [
    (dict(dt=4), "QMM_ERR_BAD_DTYPE"), (dict(T=0), "QMM_ERR_EMPTY_SHAPE"), (dict(E=0), "QMM_ERR_EMPTY_SHAPE"),
    (dict(k=0), "QMM_ERR_EMPTY_SHAPE"), (dict(k=-1), "QMM_ERR_BAD_ARGUMENT"), (dict(score=2), "QMM_ERR_BAD_ARGUMENT"),
    (dict(groups=5), "QMM_ERR_BAD_ARGUMENT"), (dict(groups=8, top=9), "QMM_ERR_BAD_ARGUMENT"), (dict(gt=0), "QMM_ERR_BAD_ARGUMENT"),
    (dict(groups=8, top=1, k=9), "QMM_ERR_BAD_ARGUMENT"), (dict(scale=float("nan")), "QMM_ERR_BAD_ARGUMENT"),
    (dict(E=1056, n=4 * 1056, st=1056), "QMM_ERR_UNIMPLEMENTED"), (dict(k=40), "QMM_ERR_UNIMPLEMENTED"),
    (dict(groups=64, top=8), "QMM_ERR_UNIMPLEMENTED"), (dict(x=0), "QMM_ERR_NULL_POINTER"), (dict(ids=0), "QMM_ERR_NULL_POINTER"),
    (dict(w=0), "QMM_ERR_NULL_POINTER"), (dict(x=FAKE + 1), "QMM_ERR_MISALIGNED"), (dict(b=FAR + 2), "QMM_ERR_MISALIGNED"),
    (dict(n=255), "QMM_ERR_ACTIVATIONS_TOO_SMALL"), (dict(out=15), "QMM_ERR_OUTPUT_TOO_SMALL"),
    (dict(ids=3 * FAR, w=3 * FAR + 60), "QMM_ERR_BAD_ARGUMENT"), (dict(ids=FAKE), "QMM_ERR_BAD_ARGUMENT"),
    (dict(b=FAR, w=FAR + 8), "QMM_ERR_BAD_ARGUMENT")])
def test_route_refusals(L, args, status):
    a = dict(x=FAKE, dt=0, n=4 * 64, st=64, b=0, score=0, groups=1, top=1, gt=1, k=4, renorm=1, scale=1.0, ids=2 * FAR, w=3 * FAR,
             out=16, T=4, E=64)
    a.update(args)
    assert L.qmoe_route(a["x"], a["dt"], a["n"], a["st"], a["b"], a["score"], a["groups"], a["top"], a["gt"], a["k"], a["renorm"],
                        a["scale"], a["ids"], a["w"], a["out"], a["T"], a["E"], None) == S[status]


def test_q4_0_pages(L):
    q4 = qmm.KV_FORMATS["q4_0"]
    assert qmm.qkv_page_bytes("q4_0", 16, 8, 128) == 16 * 8 * 4 * 18      # four 18-byte blocks a row
    assert qmm.qkv_page_bytes("q4_0", 8, 1, 96) == 8 * 3 * 18
    for bad in ((q4, 12, 8, 128), (q4, 16, 8, 80), (q4, 16, 0, 128), (3, 16, 8, 128), (5, 16, 8, 128)):
        assert qmm.qkv_page_bytes(*bad) == 0
    page = 16 * 2 * 2 * 18
    a = [q4, FAKE, 1000, 128, 64, FAKE, 1000, 128, 64, 1, FAKE, 0, 0, 0, 0, 1.0, FAR, 2 * FAR, 3 * page - 1, 3, page, 16, 4, 2, 64, None]
    assert L.qkv_store(*a) == S["QMM_ERR_CACHE_TOO_SMALL"]
    a[18], a[20] = 3 * page, page - 16
    assert L.qkv_store(*a) == S["QMM_ERR_CACHE_TOO_SMALL"]


def test_binding_argument_counts(L):
    m = qmm._calls()
    for name, n in (("qrmsnorm", 9), ("qmoe_route", 12)):
        for k in (0, 1, n - 1, n + 1):
            with pytest.raises(TypeError):
                getattr(m, name)(*[None] * k)


def test_bindings_refuse_host_tensors():
    import torch
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        qmm.qrmsnorm(x, torch.ones(64))
    with pytest.raises(ValueError):
        qmm.qmoe_route(x, 2)
    with pytest.raises(TypeError):
        qmm.qrmsnorm(x.int(), torch.ones(64))
    with pytest.raises(TypeError):
        qmm.qmoe_route(x.int(), 2)
