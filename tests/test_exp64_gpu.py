"""The short exponential and inverse in 64 bits that the router decides by (csrc/exp64.cuh), against
wider host arithmetic and CUDA's own exponential and division."""
import ctypes
import subprocess

import numpy as np
import pytest

from gemv_mul_mm_gb300 import build as qbuild

pytestmark = pytest.mark.gpu

SOURCE = """
#include "exp64.cuh"
__global__ void k(const double* x, double* y, long n, int which) {
    const long i = blockIdx.x * 256l + threadIdx.x;
    if (i >= n) return;
    y[i] = which == 0 ? qmm::exp_mid(x[i]) : which == 1 ? exp(x[i]) : which == 2 ? qmm::inverse(x[i]) : 1.0 / x[i];
}
extern "C" int run(const double* x, double* y, long n, int which) {
    k<<<static_cast<unsigned>((n + 255) / 256), 256>>>(x, y, n, which);
    const cudaError_t e = cudaGetLastError();
    return static_cast<int>(e != cudaSuccess ? e : cudaDeviceSynchronize());
}
"""


@pytest.fixture(scope="module")
def values(tmp_path_factory):
    import torch
    folder = tmp_path_factory.mktemp("exp64")
    src, lib = folder / "exp64.cu", folder / "exp64.so"
    src.write_text(SOURCE)
    subprocess.run([qbuild.nvcc(), *qbuild.ARCH, "-O3", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-I", qbuild.CSRC, str(src),
                    "-o", str(lib)], check=True, capture_output=True)
    run = ctypes.CDLL(str(lib)).run
    run.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_long, ctypes.c_int]

    def of(x, which):
        d = torch.from_numpy(x).cuda()
        y = torch.empty_like(d)
        torch.cuda.synchronize()
        assert run(d.data_ptr(), y.data_ptr(), len(x), which) == 0
        return y.cpu().numpy()
    return of


def ulps(got, want):
    """|got - want| in units of the last place of want (80 bits or more)."""
    if np.finfo(np.longdouble).eps > 2.0 ** -60:
        pytest.skip("no wider host type")
    return np.abs(got.astype(np.longdouble) - want) / np.spacing(np.abs(want.astype(np.float64)))


def points(seed):
    """Exponents over the whole range, near multiples of ln 2 and of half of it, and the ends."""
    rng = np.random.RandomState(seed)
    near = np.concatenate([np.arange(-2019, 2020) * (np.log(2) / 2) + d for d in (0.0, 1e-13, -1e-13, 1e-6, -1e-6)])
    x = np.concatenate([rng.uniform(-700, 700, 200000), rng.uniform(-2, 2, 100000), rng.randn(1000) * 1e-9, near, [0.0, 700.0, -700.0, 1.0, -1.0]])
    return x[np.abs(x) <= 700]


def test_exponential(values):
    x = points(1)
    got = values(x, 0)
    assert float(ulps(got, np.exp(x.astype(np.longdouble))).max()) <= 2
    # CUDA's is within 1 ulp by its documentation
    assert float(ulps(got, values(x, 1).astype(np.longdouble)).max()) <= 3
    assert values(np.array([0.0]), 0)[0] == 1.0


def test_inverse(values):
    rng = np.random.RandomState(2)
    d = np.concatenate([2.0 ** rng.uniform(0, 126, 200000), 1.0 + np.abs(rng.randn(100000)), 1.0 + 2.0 ** rng.uniform(-53, 0, 100000),
                        2.0 ** np.arange(0, 127), np.arange(1.0, 2000.0)])
    got = values(d, 2)
    assert float(ulps(got, 1 / d.astype(np.longdouble)).max()) <= 1
    assert float(ulps(got, values(d, 3).astype(np.longdouble)).max()) <= 1.5     # 1 / d rounds by half an ulp
    assert np.array_equal(got[-2126:-1999], 1 / d[-2126:-1999])                   # powers of two
