"""qattn_decode's workspace: sized once for the largest batch and bound, it
serves every smaller call, though those may be split more often."""
import pytest

from tests import kv_util as U
from tests.test_attn_decode_gpu import Q, call, problem  # noqa: F401

pytestmark = pytest.mark.gpu

LENGTHS = sorted({int(16 * 1.07 ** i) for i in range(160)} | {1216, 1280, 1344, 7360, 9536, 9728, 131072})


@pytest.mark.parametrize("fmt,dt", [("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("q8_0", "f16"), ("q8_0", "f32")])
@pytest.mark.parametrize("Hkv,group,D", [(8, 4, 128), (1, 1, 64), (4, 16, 96), (2, 17, 128), (5, 7, 256)])
def test_size_grows_with_batch_bound_and_window(Q, fmt, dt, Hkv, group, D):
    def size(B, n, window=0):
        return Q.qattn_decode_workspace_bytes(fmt, U.dtype(dt), B, Hkv * group, Hkv, D, n, window)
    for B in (1, 2, 3, 7, 16, 64, 300):
        s = [size(B, n) for n in LENGTHS]
        assert s == sorted(s)
        s = [size(B, 131072, w) for w in LENGTHS if w < 131072] + [size(B, 131072)]
        assert s == sorted(s)
    for n in (64, 65, 1000, 9000, 131072):
        s = [size(B, n) for B in list(range(1, 40)) + [64, 100, 129, 500]]
        assert s == sorted(s)
        for B in (1, 3, 16, 100):                                     # and it holds every split's results
            k = Q.qattn_decode_splits(fmt, U.dtype(dt), B, Hkv * group, Hkv, D, n)
            assert k >= 1 and (k == 1 or size(B, n) >= B * Hkv * group * k * (4 * D + 8))


@pytest.mark.parametrize("fmt,dt,B,Hkv,group", [("f16", "f32", 16, 8, 2), ("q8_0", "f16", 16, 8, 4), ("f16", "f16", 1, 8, 4)])
def test_one_workspace_for_every_bound(Q, fmt, dt, B, Hkv, group):
    import torch
    p = problem(Q, fmt, dt, 64, Hkv, group, 64, [700] * B, 2, garbage=False)
    width = 10000 // 64
    p["table"] = torch.nn.functional.pad(p["table"], (0, width - p["table"].shape[1]), value=0)
    most = width * 64
    ws = torch.empty(Q.qattn_decode_workspace_bytes(fmt, U.dtype(dt), B, Hkv * group, Hkv, 64, most), dtype=torch.uint8, device="cuda")
    for max_len in (most, 9728, 9536, 7360, 1344, 1280, 1216, 704, 700):
        got = call(Q, p, workspace=ws, max_len=max_len)
        assert torch.equal(got, call(Q, p, max_len=max_len))
        assert Q.check_device_error() == 0
    r = {**p, "q": p["q"][:B // 2 + 1], "table": p["table"][:B // 2 + 1], "lens": p["lens"][:B // 2 + 1]}
    assert torch.equal(call(Q, r, workspace=ws), call(Q, r))


def test_an_unsplit_call_needs_none(Q):
    import torch
    p = problem(Q, "f16", "f16", 64, 8, 2, 64, [60] * 200, 2, garbage=False)
    n = p["table"].shape[1] * 64
    assert Q.qattn_decode_splits("f16", torch.float16, 200, 16, 8, 64, n) == 1
    assert torch.equal(call(Q, p, workspace=torch.empty(0, dtype=torch.uint8, device="cuda")), call(Q, p))
    assert Q.qattn_decode_splits("f16", torch.float16, 200, 15, 8, 64, n) == 0
