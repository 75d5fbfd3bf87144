"""The norms, the routing and the q4_0 cache together with the products, as
examples/moe_decoder_layer.py runs them: prompts, then decode steps replayed from
a CUDA graph, the last step against its 64-bit recomputation; and the 4-bit
cache in the attention half alone."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def built():
    from gemv_mul_mm_gb300 import build as qbuild
    qbuild.build()


# Activations between operators are f16 on both sides and may differ by one rounding (2^-11)
# where the value is near to a tie: the normed rows, the heads, the normed and the rotated
# query, the attention's output; the products' own bar is 1e-3 of the sums of magnitudes,
# three of them in a row, and random products' results are some 1/20 of those.
@pytest.mark.parametrize("fmt,kind,batch", [("q4_0", "Q4_0", 4), ("q4_0", "Q8_0", 1), ("q8_0", "Q4_K", 7), ("f16", "Q8_0", 9)])
def test_decode_steps(built, fmt, kind, batch):
    from examples.moe_decoder_layer import run
    err, us = run(steps=20, batch=batch, fmt=fmt, kind=kind, d_model=1024, q_heads=8, kv_heads=2, max_len=512, page=16)
    assert err < 5 * 2.0 ** -11 + 3e-3 and us > 0


@pytest.mark.parametrize("dim,page,batch", [(64, 8, 3), (128, 32, 4)])
def test_attention_half_over_q4_0(built, dim, page, batch):
    from examples.decode_layer import run
    err, _ = run(steps=5, batch=batch, fmt="q4_0", kind="Q8_0", d_model=512, q_heads=6, kv_heads=2, dim=dim, max_len=300, page=page)
    assert err < 4 * 2.0 ** -11 + 1e-3
