"""The rotary, cache and attention operators together with the quantized
products, as examples/decode_layer.py runs them: prompts, then decode steps
replayed from a CUDA graph, the last step against its 64-bit recomputation."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from gemv_mul_mm_gb300 import build as qbuild
    qbuild.build()
    spec = importlib.util.spec_from_file_location("decode_layer", os.path.join(ROOT, "examples", "decode_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


# the qkv product, the rotated query and the attention output are f16 on both
# sides and may differ by one rounding (2^-11 relative) where the fp32 value is
# near to a tie; the products' own bar is 1e-3
@pytest.mark.parametrize("fmt,kind,batch", [("q8_0", "Q4_0", 4), ("f16", "Q8_0", 1), ("bf16", "Q4_K", 9)])
def test_decode_steps(example, fmt, kind, batch):
    err, us = example.run(steps=40, batch=batch, fmt=fmt, kind=kind, d_model=1024, q_heads=8, kv_heads=2, max_len=512, page=16)
    assert err < 4 * 2.0 ** -11 + 1e-3 and us > 0


def test_attention_of_other_head_dims(example):
    err, _ = example.run(steps=5, batch=3, fmt="q8_0", kind="Q8_0", d_model=512, q_heads=6, kv_heads=2, dim=64, max_len=300, page=8)
    assert err < 4 * 2.0 ** -11 + 1e-3
