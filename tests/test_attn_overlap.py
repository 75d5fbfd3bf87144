"""qattn_decode's output: q itself where that is contiguous, else apart from it."""
import pytest

from gemv_mul_mm_gb300 import build as qbuild
from gemv_mul_mm_gb300 import qmm
from tests.test_attn_decode_gpu import Q, call, problem  # noqa: F401

FAKE = 0x100000  # never dereferenced: every call below is refused before a launch
B, H, D = 3, 8, 64


@pytest.mark.parametrize("shift,q_bs,q_hs", [
    (1, H * D, D), (D, H * D, D), (H * D, H * D, D), (-2 * H * D, H * D, D),   # out and q shifted against each other
    (0, 2 * H * D, D), (0, H * D, 0), (H * D, 3 * H * D, D)])                  # other strides over the same range
def test_partial_overlap_is_refused(shift, q_bs, q_hs):
    qbuild.build()
    page = qmm.qkv_page_bytes("f16", 16, 2, D)
    rc = qmm.lib().qattn_decode(0, FAKE, 1, 1 << 30, q_bs, q_hs, FAKE, FAKE, 4 * page, 4, page, 16, FAKE, 12, 4, 4, FAKE, 64, B, H, 2,
                                D, 0.1, 0, 0.0, FAKE + 2 * shift, 1 << 30, None, None, 0, None)
    assert rc == qmm.STATUS_ID["QMM_ERR_BAD_ARGUMENT"]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,dt,group", [("f16", "f16", 4), ("q8_0", "f32", 12), ("bf16", "bf16", 20)])
@pytest.mark.parametrize("lens", [[100, 33, 0], [9000, 0, 5, 700]])
def test_in_place(Q, fmt, dt, group, lens):
    import torch
    p = problem(Q, fmt, dt, 128, 2, group, 16, lens, 4)
    want = call(Q, p)
    for _ in range(5):
        r = {**p, "q": p["q"].clone()}
        assert torch.equal(call(Q, r, out=r["q"]), want)


@pytest.mark.gpu
def test_rows_of_a_fused_product(Q):
    """q between the rows of something else, out in a buffer of its own."""
    import torch
    p = problem(Q, "f16", "f16", 64, 2, 4, 16, [50, 300], 8)
    big = torch.zeros((2, 12, 64), dtype=torch.float16, device="cuda")
    big[:, :8].copy_(p["q"])
    assert torch.equal(call(Q, {**p, "q": big[:, :8]}), call(Q, p))
    with pytest.raises(Q.QmmError) as e:
        call(Q, {**p, "q": big[:, :8]}, out=big.view(-1)[:2 * 8 * 64])
    assert e.value.name == "QMM_ERR_BAD_ARGUMENT"
