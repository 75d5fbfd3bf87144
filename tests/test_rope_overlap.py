"""qrope refuses outputs that overlap themselves or their input, before a launch
(no GPU needed), by exactly the calls in which an element would be touched twice."""
import itertools
import random

import pytest

from gemv_mul_mm_gb300 import build as qbuild
from gemv_mul_mm_gb300 import qmm

BASE = 0x100000  # never dereferenced without a GPU; only refused calls are made where there is one
BAD = qmm.STATUS_ID["QMM_ERR_BAD_ARGUMENT"]


@pytest.fixture(scope="module")
def L():
    qbuild.build()
    return qmm.lib()


def refused(L, T, H, D, x, xts, xhs, y, yts, yhs):
    """Offsets x and y in elements (f16)."""
    return L.qrope(BASE + 2 * x, 1, 1 << 40, xts, xhs, BASE, BASE, 2, 0, 1.0, BASE + 2 * y, 1 << 40, yts, yhs, T, H, D, None) == BAD


def elements(T, H, D, at, ts, hs):
    return [at + t * ts + h * hs + d for t in range(T) for h in range(H) for d in range(D)]


FAR = 1 << 30


@pytest.mark.parametrize("T,H,D,ts,hs", [
    (4, 3, 8, 0, 8), (4, 3, 8, 24, 0), (4, 3, 8, 0, 0), (2, 1, 8, 7, 8), (1, 2, 8, 0, 7), (3, 2, 8, 8, 8), (3, 2, 8, 16, 24 - 1),
    (2, 65536, 64, 64, 64), (1 << 20, 2, 64, 64, 64 * ((1 << 20) - 1))])
def test_outputs_that_overlap_themselves(L, T, H, D, ts, hs):
    assert refused(L, T, H, D, 0, H * D, D, FAR, ts, hs)


def test_in_place_and_shifted(L):
    T, H, D = 5, 4, 16
    for shift in (1, 15, 16, 48, H * D, (T - 1) * H * D):
        assert refused(L, T, H, D, 0, H * D, D, shift, H * D, D)
        assert refused(L, T, H, D, shift, H * D, D, 0, H * D, D)
    assert refused(L, T, H, D, 0, H * D, D, 0, 2 * H * D, D)            # the same address, other strides
    assert refused(L, T, H, D, 0, 48 * D, D, 3 * D, 48 * D, D)          # a head too many of a fused row
    assert refused(L, T, H, D, 0, 48 * D, 2 * D, D, 48 * D, D)


@pytest.mark.skipif("__import__('torch').cuda.is_available()", reason="accepted calls on made-up addresses would launch")
def test_exactly_the_calls_that_touch_an_element_twice(L):
    """Against sets of elements. (Without a GPU an accepted call ends in QMM_ERR_CUDA.)"""
    rng = random.Random(5)
    seen = set()
    for _ in range(20000):
        T, H, D = rng.randint(1, 4), rng.randint(1, 4), rng.choice([2, 3, 4])
        n = lambda: rng.choice([0, 1, D - 1, D, D + 1, 2 * D, H * D, H * D + 1, T * D, 2 * H * D, 3 * H * D, rng.randint(0, 40)])  # noqa: E731
        xts, xhs = n(), n()
        yts, yhs = (xts, xhs) if rng.random() < 0.5 else (xts, n()) if rng.random() < 0.7 else (n(), n())
        y = rng.choice([0, D, H * D, rng.randint(-30, 60), 500])
        xe, ye = elements(T, H, D, 0, xts, xhs), elements(T, H, D, y, yts, yhs)
        same = y == 0 and (T == 1 or xts == yts) and (H == 1 or xhs == yhs)
        bad = len(set(ye)) < len(ye) or (not same and bool(set(xe) & set(ye)))
        unclear = T > 1 and xts != yts and max(xe) >= min(ye) and max(ye) >= min(xe)   # refused, overlap or not
        assert refused(L, T, H, D, 0, xts, xhs, y, yts, yhs) == (bad or unclear)
        seen.add((bad, unclear, same))
    assert len(seen) >= 5


@pytest.mark.skipif("__import__('torch').cuda.is_available()", reason="accepted calls on made-up addresses would launch")
def test_usual_calls_are_not_refused(L):
    for T, H, D in itertools.product((1, 7, 8192), (1, 40, 65536), (2, 80, 128)):
        for x, xts, y, yts in ((0, H * D, 0, H * D), (0, H * D, T * H * D, H * D), (0, 3 * H * D, H * D, 3 * H * D),
                               (0, 3 * H * D, 1 << 40, H * D)):
            assert not refused(L, T, H, D, x, xts, D, y, yts, D)
        assert not refused(L, T, H, D, 0, D, T * D, 1 << 45, D, T * D)    # heads outermost
