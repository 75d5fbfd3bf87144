"""examples/decode_layer.py notices a cache that does not hold what its prompts
and steps should have left: its own check of keys and values, with the layer's
store or prompt replaced by one that is wrong."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SIZES = dict(steps=5, batch=3, kind="Q8_0", d_model=512, q_heads=4, kv_heads=2, dim=64, max_len=128, page=16)


@pytest.fixture
def example():
    from gemv_mul_mm_gb300 import build as qbuild
    qbuild.build()
    spec = importlib.util.spec_from_file_location("decode_layer_check", os.path.join(ROOT, "examples", "decode_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def store_with(change):
    """AttentionLayer.store with (k, v, positions, slots) changed on the way."""
    def store(self, k, v, positions):
        from gemv_mul_mm_gb300 import qmm
        k, v, at, slots = change(k, v, positions.flatten().int().contiguous(), self.slots(positions))
        qmm.qkv_store(self.fmt, k, v, slots, self.k_cache, self.v_cache, self.page, positions=at, turns=self.turns,
                      mscale=self.mscale)
    return store


def skipped(k, v, at, slots):
    slots = slots.clone()
    slots[0] = -1
    return k, v, at, slots


WRONG = {
    "keys one position off": lambda k, v, at, slots: (k, v, at + 1, slots),
    "keys not rotated": lambda k, v, at, slots: (k, v, at * 0, slots),
    "keys and values exchanged": lambda k, v, at, slots: (v, k, at, slots),
    "a token skipped": skipped,
}


@pytest.mark.parametrize("fmt", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("what", sorted(WRONG))
def test_a_wrong_cache_is_noticed(example, monkeypatch, fmt, what):
    monkeypatch.setattr(example.AttentionLayer, "store", store_with(WRONG[what]))
    with pytest.raises(RuntimeError):
        example.run(fmt=fmt, **SIZES)


@pytest.mark.parametrize("fmt", ["f16", "bf16", "q8_0"])
def test_lost_lengths_are_noticed(example, monkeypatch, fmt):
    prompt = example.AttentionLayer.prompt

    def shorter(self, x, lens):
        prompt(self, x, lens)
        self.lens.clamp_(max=5)
    monkeypatch.setattr(example.AttentionLayer, "prompt", shorter)
    with pytest.raises(RuntimeError):
        example.run(fmt=fmt, **SIZES)


@pytest.mark.parametrize("fmt", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("kind", ["Q8_0", "Q4_0", "Q4_K"])
def test_a_right_one_passes(example, fmt, kind):
    err, _ = example.run(fmt=fmt, **{**SIZES, "kind": kind})
    assert err < 4 * 2.0 ** -11 + 1e-3
