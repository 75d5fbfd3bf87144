"""The rotary, cache and attention entry points on the CPU: the frequency table
against its definition, page sizes, and every refusal by name before a launch
(no GPU needed: none of these calls reaches one)."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

from gemv_mul_mm_gb300 import build as qbuild
from gemv_mul_mm_gb300 import qmm

FAKE = 0x10000  # never dereferenced: every call below is refused before a launch
S = qmm.STATUS_ID


@pytest.fixture(scope="module")
def L():
    qbuild.build()
    return qmm.lib()


def test_page_bytes(L):
    assert qmm.qkv_page_bytes("f16", 16, 8, 128) == 16 * 8 * 256
    assert qmm.qkv_page_bytes("q8_0", 16, 8, 128) == 16 * 8 * 4 * 34     # four 34-byte blocks a row
    assert qmm.qkv_page_bytes("bf16", 8, 1, 96) == 8 * 192
    for bad in (("f16", 12, 8, 128), ("f16", 4, 8, 128), ("f16", 8192, 8, 128), ("f16", 16, 0, 128), ("q8_0", 16, 8, 80),
                (7, 16, 8, 128)):
        assert qmm.qkv_page_bytes(*bad) == 0


def freqs(base, rot, scaling, factor, orig, fast, slow):
    out = []
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        if scaling == "linear":
            f /= factor
        if scaling == "ramp":
            at = lambda r: rot * math.log(orig / (r * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
            lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), rot - 1)
            x = min(max((i - lo) / max(hi - lo, 0.001), 0), 1)
            f = f / factor * x + f * (1 - x)
        if scaling == "bands":
            x = min(max((orig * f / (2 * math.pi) - slow) / (fast - slow), 0), 1)
            f = f / factor * (1 - x) + f * x
        out.append(f)
    return out


@pytest.mark.parametrize("base,rot,scaling,factor", [
    (10000.0, 128, "plain", 1.0), (500000.0, 64, "linear", 4.0), (10000.0, 96, "base", 8.0),
    (1000000.0, 128, "ramp", 16.0), (500000.0, 128, "bands", 8.0), (10000.0, 2, "plain", 1.0)])
def test_turns_table(L, base, rot, scaling, factor):
    fast = {"ramp": 32.0, "bands": 4.0}.get(scaling, 4.0)
    turns, m = qmm.qrope_turns(rot, base, scaling, factor, 4096.0, fast, 1.0, device="cpu")
    got = turns.numpy().view(np.uint64)
    want = freqs(base, rot, scaling, factor, 4096.0, fast, 1.0)
    assert len(got) == rot // 2
    for g, f in zip(got, want):
        turn = Fraction(f) / Fraction(2 * math.pi)
        # two doubles' roundings of pow and of the quotients, and half a unit of 2^-64
        assert abs(Fraction(int(g), 2 ** 64) - turn) <= turn * 16 * Fraction(1, 2 ** 53) + Fraction(1, 2 ** 64)
    assert m == pytest.approx(0.1 * math.log(factor) + 1 if scaling == "ramp" else 1.0, rel=1e-7)


@pytest.mark.parametrize("args", [
    dict(rot=0), dict(rot=-2), dict(rot=3), dict(base=1.0), dict(base=float("inf")), dict(base=float("nan")), dict(scaling=5),
    dict(scaling=-1), dict(scaling=1, factor=0.5), dict(scaling=1, factor=float("nan")), dict(scaling=2, rot=2),
    dict(scaling=3, orig=0.0), dict(scaling=3, fast=1.0), dict(scaling=4, slow=0.0)])
def test_turns_refusals(L, args):
    a = dict(base=10000.0, rot=8, scaling=0, factor=2.0, orig=4096.0, fast=4.0, slow=1.0)
    a.update(args)
    out, m = (ctypes.c_uint64 * 8)(), ctypes.c_float()
    assert L.qrope_turns(a["base"], a["rot"], a["scaling"], a["factor"], a["orig"], a["fast"], a["slow"], out,
                         ctypes.byref(m)) == S["QMM_ERR_BAD_ARGUMENT"]


def test_turns_null(L):
    assert L.qrope_turns(1e4, 8, 0, 1.0, 0.0, 0.0, 0.0, None, ctypes.byref(ctypes.c_float())) == S["QMM_ERR_NULL_POINTER"]


@pytest.mark.parametrize("args,status", [
    (dict(dt=3), "QMM_ERR_BAD_DTYPE"), (dict(T=0), "QMM_ERR_EMPTY_SHAPE"), (dict(H=0), "QMM_ERR_EMPTY_SHAPE"),
    (dict(T=-1), "QMM_ERR_BAD_ARGUMENT"), (dict(xts=-4), "QMM_ERR_BAD_ARGUMENT"), (dict(rot=130), "QMM_ERR_BAD_ARGUMENT"),
    (dict(rot=7), "QMM_ERR_BAD_ARGUMENT"), (dict(rot=0), "QMM_ERR_BAD_ARGUMENT"), (dict(layout=2), "QMM_ERR_BAD_ARGUMENT"),
    (dict(m=float("inf")), "QMM_ERR_BAD_ARGUMENT"), (dict(X=0), "QMM_ERR_NULL_POINTER"),
    (dict(turns=0), "QMM_ERR_NULL_POINTER"), (dict(X=FAKE + 1), "QMM_ERR_MISALIGNED"),
    (dict(turns=FAKE + 4), "QMM_ERR_MISALIGNED"), (dict(xn=3 * 512 + 3 * 128 + 127), "QMM_ERR_ACTIVATIONS_TOO_SMALL"),
    (dict(yn=4 * 512 - 1), "QMM_ERR_OUTPUT_TOO_SMALL")])
def test_rope_refusals(L, args, status):
    a = dict(X=FAKE, dt=1, xn=4 * 512, xts=512, xhs=128, pos=FAKE, turns=FAKE, rot=128, layout=0, m=1.0, Y=FAKE, yn=4 * 512,
             yts=512, yhs=128, T=4, H=4, D=128)
    a.update(args)
    assert L.qrope(a["X"], a["dt"], a["xn"], a["xts"], a["xhs"], a["pos"], a["turns"], a["rot"], a["layout"], a["m"], a["Y"],
                   a["yn"], a["yts"], a["yhs"], a["T"], a["H"], a["D"], None) == S[status]


CACHE_REFUSALS = [
    (dict(fmt=3), "QMM_ERR_BAD_KIND"), (dict(dt=-1), "QMM_ERR_BAD_DTYPE"), (dict(ps=24), "QMM_ERR_BAD_ARGUMENT"),
    (dict(ps=4), "QMM_ERR_BAD_ARGUMENT"), (dict(pages=0), "QMM_ERR_EMPTY_SHAPE"), (dict(pages=-1), "QMM_ERR_BAD_ARGUMENT"),
    (dict(kc=0), "QMM_ERR_NULL_POINTER"), (dict(vc=FAKE + 8), "QMM_ERR_MISALIGNED"), (dict(stride=4 * 4096 + 8), "QMM_ERR_MISALIGNED"),
    (dict(stride=4 * 4096 - 16), "QMM_ERR_CACHE_TOO_SMALL"), (dict(bytes=10 * 4 * 4096 - 1), "QMM_ERR_CACHE_TOO_SMALL")]


@pytest.mark.parametrize("args,status", CACHE_REFUSALS + [
    (dict(T=0), "QMM_ERR_EMPTY_SHAPE"), (dict(D=80), "QMM_ERR_COLS_NOT_BLOCK_ALIGNED"), (dict(slots=0), "QMM_ERR_NULL_POINTER"),
    (dict(slots=FAKE + 4), "QMM_ERR_MISALIGNED"), (dict(K=FAKE + 1), "QMM_ERR_MISALIGNED"),
    (dict(kn=2 * 512 + 511), "QMM_ERR_ACTIVATIONS_TOO_SMALL"), (dict(vn=0), "QMM_ERR_ACTIVATIONS_TOO_SMALL"),
    (dict(pos=FAKE), "QMM_ERR_NULL_POINTER"), (dict(pos=FAKE, turns=FAKE, rot=256), "QMM_ERR_BAD_ARGUMENT")])
def test_store_refusals(L, args, status):
    a = dict(fmt=0, K=FAKE, kn=3 * 512, kts=512, khs=128, V=FAKE, vn=3 * 512, vts=512, vhs=128, dt=1, slots=FAKE, pos=0, turns=0,
             rot=128, layout=0, m=1.0, kc=FAKE, vc=FAKE, bytes=10 * 4 * 4096, pages=10, stride=4 * 4096, ps=16, T=3, H=4, D=128)
    a.update(args)
    assert L.qkv_store(a["fmt"], a["K"], a["kn"], a["kts"], a["khs"], a["V"], a["vn"], a["vts"], a["vhs"], a["dt"], a["slots"],
                       a["pos"], a["turns"], a["rot"], a["layout"], a["m"], a["kc"], a["vc"], a["bytes"], a["pages"],
                       a["stride"], a["ps"], a["T"], a["H"], a["D"], None) == S[status]


@pytest.mark.parametrize("args,status", CACHE_REFUSALS + [
    (dict(T=0), "QMM_ERR_EMPTY_SHAPE"), (dict(K=0), "QMM_ERR_NULL_POINTER"), (dict(V=FAKE + 2), "QMM_ERR_MISALIGNED"),
    (dict(n=3 * 512 - 1), "QMM_ERR_OUTPUT_TOO_SMALL")])
def test_load_refusals(L, args, status):
    a = dict(fmt=0, slots=FAKE, kc=FAKE, vc=FAKE, bytes=10 * 4 * 4096, pages=10, stride=4 * 4096, ps=16, K=FAKE, V=FAKE, dt=0,
             n=3 * 512, T=3, H=4, D=128)
    a.update(args)
    assert L.qkv_load(a["fmt"], a["slots"], a["kc"], a["vc"], a["bytes"], a["pages"], a["stride"], a["ps"], a["K"], a["V"],
                      a["dt"], a["n"], a["T"], a["H"], a["D"], None) == S[status]


@pytest.mark.parametrize("args,status", CACHE_REFUSALS + [
    (dict(B=0), "QMM_ERR_EMPTY_SHAPE"), (dict(maxlen=0), "QMM_ERR_EMPTY_SHAPE"), (dict(Hq=6), "QMM_ERR_BAD_ARGUMENT"),
    (dict(window=-1), "QMM_ERR_BAD_ARGUMENT"), (dict(cap=-1.0), "QMM_ERR_BAD_ARGUMENT"),
    (dict(cap=float("nan")), "QMM_ERR_BAD_ARGUMENT"), (dict(scale=float("nan")), "QMM_ERR_BAD_ARGUMENT"),
    (dict(maxlen=81), "QMM_ERR_BAD_ARGUMENT"), (dict(D=160, stride=4 * 16 * 320, bytes=1 << 30), "QMM_ERR_UNIMPLEMENTED"),
    (dict(q=0), "QMM_ERR_NULL_POINTER"), (dict(lens=0), "QMM_ERR_NULL_POINTER"), (dict(q=FAKE + 1), "QMM_ERR_MISALIGNED"),
    (dict(lse=FAKE + 2), "QMM_ERR_MISALIGNED"), (dict(qn=2 * 1024 - 1), "QMM_ERR_ACTIVATIONS_TOO_SMALL"),
    (dict(tn=9), "QMM_ERR_ACTIVATIONS_TOO_SMALL"), (dict(on=2 * 1024 - 1), "QMM_ERR_OUTPUT_TOO_SMALL")])
def test_attention_refusals(L, args, status):
    a = dict(fmt=0, q=FAKE, dt=1, qn=2 * 1024, qbs=1024, qhs=128, kc=FAKE, vc=FAKE, bytes=10 * 4 * 4096, pages=10,
             stride=4 * 4096, ps=16, table=FAKE, tn=10, ts=5, width=5, lens=FAKE, maxlen=80, B=2, Hq=8, H=4, D=128, scale=0.1,
             window=0, cap=0.0, out=FAKE, on=2 * 1024, lse=0, ws=0, wsb=0)
    a.update(args)
    assert L.qattn_decode(a["fmt"], a["q"], a["dt"], a["qn"], a["qbs"], a["qhs"], a["kc"], a["vc"], a["bytes"], a["pages"],
                          a["stride"], a["ps"], a["table"], a["tn"], a["ts"], a["width"], a["lens"], a["maxlen"], a["B"],
                          a["Hq"], a["H"], a["D"], a["scale"], a["window"], a["cap"], a["out"], a["on"], a["lse"], a["ws"],
                          a["wsb"], None) == S[status]


def test_new_status_strings(L):
    for code in (S["QMM_ERR_CACHE_TOO_SMALL"], S["QMM_ERR_BAD_SLOT"]):
        assert L.qmm_status_str(code) != b"unknown status"


def test_binding_refuses_wrong_tensors():
    import torch
    x = torch.zeros(4, 2, 64)
    pos, turns = torch.zeros(4, dtype=torch.int32), torch.zeros(32, dtype=torch.int64)
    with pytest.raises(TypeError):
        qmm.qrope(x.double(), pos, turns)
    with pytest.raises(ValueError):
        qmm.qrope(x[0], pos, turns)
    with pytest.raises(ValueError):
        qmm.qrope(x, pos.long(), turns)
    with pytest.raises(ValueError):
        qmm.qrope(x.transpose(1, 2), pos, turns)
    with pytest.raises(ValueError):
        qmm.qrope(x, pos[:3], turns)
    kc = torch.zeros(3, qmm.qkv_page_bytes("f16", 16, 2, 64), dtype=torch.uint8)
    slots = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        qmm.qkv_store("f16", x, x[:2], slots, kc, kc, 16)
    with pytest.raises(ValueError):
        qmm.qkv_store("f16", x, x, slots, kc, kc[:2], 16)
    with pytest.raises(ValueError):
        qmm.qkv_store("f16", x, x, slots, kc, kc, 16, positions=pos)
    with pytest.raises(ValueError):
        qmm.qattn_decode("f16", x, kc, kc, torch.zeros(4, 2), pos, 16, 2)
    with pytest.raises(ValueError):
        qmm.qattn_decode("f16", x, kc, kc, torch.zeros(3, 2, dtype=torch.int32), pos, 16, 2)
    with pytest.raises(ValueError):
        qmm.qkv_cache("q8_0", 4, 16, 2, 80, device="cpu")
