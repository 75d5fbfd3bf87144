"""The attention half of a decoder layer's decode step on block-quantized weights
and a quantized, paged key-value cache: fused QKV projection, rotary positions,
cache write, attention of the new tokens, output projection.

    python examples/decode_layer.py [--steps 32] [--batch 4] [--fmt q8_0] [--kind Q4_0]

runs a batch of sequences of different lengths for some steps, replaying one
CUDA graph per step, checks the cache and the last step against a plain 64-bit
computation, and prints the time of a step.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from gemv_mul_mm_gb300 import qmm, synth  # noqa: E402


class AttentionLayer:
    """Weights, cache and page tables of one layer for `batch` sequences of up to
    `max_len` tokens. Pages are handed out in order as sequences grow."""

    def __init__(self, kind="Q4_0", fmt="q8_0", d_model=2048, q_heads=16, kv_heads=4, dim=128, batch=4, max_len=1024, page=32,
                 seed=1):
        self.kind, self.fmt, self.page, self.max_len = kind, fmt, page, max_len
        self.d_model, self.q_heads, self.kv_heads, self.dim, self.batch = d_model, q_heads, kv_heads, dim, batch
        self.rows = (q_heads + 2 * kv_heads) * dim
        self.w_qkv = torch.from_numpy(synth.quant_weights(kind, self.rows, d_model, seed)).cuda()
        self.w_out = torch.from_numpy(synth.quant_weights(kind, d_model, q_heads * dim, seed + 1)).cuda()
        self.turns, self.mscale = qmm.qrope_turns(dim, base=500000.0, scaling="bands", factor=8.0, orig_len=8192.0)
        width = (max_len + page - 1) // page
        self.k_cache, self.v_cache = qmm.qkv_cache(fmt, batch * width, page, kv_heads, dim)
        self.table = torch.randperm(batch * width, generator=torch.Generator().manual_seed(seed)).int().view(batch, width).cuda()
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")

    def slots(self, positions):
        """Cache slots of `positions` (batch, n) of each sequence, as (batch * n,)."""
        p = positions.long()
        return (torch.gather(self.table.long(), 1, p // self.page) * self.page + p % self.page).flatten()

    def heads(self, x):
        """Query, key and value heads of the rows of x, as views of one product."""
        y = qmm.qgemm(self.kind, self.w_qkv, x, self.rows, self.d_model, x.shape[0], weights_const=True,
                      out_dtype=torch.float16).view(x.shape[0], -1, self.dim)
        h, k = self.q_heads, self.kv_heads
        return y[:, :h], y[:, h:h + k], y[:, h + k:]

    def store(self, k, v, positions):
        """Keys (rotated) and values of `positions` (batch, n), rows in that order."""
        qmm.qkv_store(self.fmt, k, v, self.slots(positions), self.k_cache, self.v_cache, self.page,
                      positions=positions.flatten().int().contiguous(), turns=self.turns, mscale=self.mscale)

    def prompt(self, x, lens):
        """Fills the cache from prompts x (batch, n, d_model), of which the first
        lens[b] tokens count."""
        b, n, _ = x.shape
        _, k, v = self.heads(x.reshape(b * n, -1))
        self.store(k, v, torch.arange(n, device="cuda").expand(b, n))
        self.lens.copy_(lens)

    def step(self, x):
        """One new token per sequence: x (batch, d_model) to the layer's attention
        output (batch, d_model), fp32."""
        q, k, v = self.heads(x)
        self.store(k, v, self.lens[:, None])
        q = qmm.qrope(q, self.lens, self.turns, mscale=self.mscale)
        self.lens += 1
        o = qmm.qattn_decode(self.fmt, q, self.k_cache, self.v_cache, self.table, self.lens, self.page, self.kv_heads,
                             max_len=self.max_len)
        return qmm.qgemm(self.kind, self.w_out, o.view(self.batch, -1), self.d_model, self.q_heads * self.dim, self.batch,
                         weights_const=True)

    def plain_heads(self, x):
        """heads(x) of x (n, d_model) in 64 bits from the weights, rounded to f16 as there."""
        w = qmm.qdequant(self.kind, self.w_qkv, self.rows, self.d_model).double()
        y = (x.double() @ w.T).half().double().view(x.shape[0], -1, self.dim)
        h, k = self.q_heads, self.kv_heads
        return y[:, :h], y[:, h:h + k], y[:, h + k:]

    def plain_rotation(self, x, positions):
        """x (n, heads, dim) rotated at positions (n,), in 64 bits."""
        turns = self.turns.cpu().numpy().view("uint64").astype("float64") / 2.0 ** 64
        a = positions.double()[:, None, None] * torch.from_numpy(turns * 2 * math.pi).cuda()
        c, s = a.cos() * self.mscale, a.sin() * self.mscale
        x1, x2 = x.chunk(2, -1)
        return torch.cat([x1 * c - x2 * s, x2 * c + x1 * s], -1)

    def check_cache(self, x, lens, token, steps):
        """Raises unless prompts x of lens tokens and `steps` steps on token left the
        lengths and the rows that they should have: each head's key and value
        against the weights' 64-bit products, rotated in 64 bits. Of a row's norm the product may be off
        by 4e-3 and its f16 rounding by 2^-11, twice, the cache by its
        format's rounding (Q8_0: half a code, amax / 254, in each of 32 values; Q4_0: half a
        code, amax / 16, in 31 values, and where -8 has no opposite a whole one, of a
        value that counts for more in the norm)."""
        if not torch.equal(self.lens, lens + steps):
            raise RuntimeError(f"lengths are {self.lens.tolist()}, not {(lens + steps).tolist()}")
        bound = 4e-3 + 2 * 2.0 ** -11 + {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "q8_0": 32 ** 0.5 / 254 * (1 + 2.0 ** -9),
                                        "q4_0": 31 ** 0.5 / 16 * (1 + 2.0 ** -8)}[self.fmt]
        for b, n in enumerate(lens.tolist()):
            at = torch.arange(n + steps, device="cuda")
            _, k, v = self.plain_heads(torch.cat([x[b, :n], token[b].expand(steps, -1)]))
            slots = self.slots(at.expand(self.batch, -1)).view(self.batch, -1)[b].contiguous()
            got = qmm.qkv_load(self.fmt, slots, self.k_cache, self.v_cache, self.page, self.kv_heads, self.dim)
            for name, have, want in (("key", got[0], self.plain_rotation(k, at)), ("value", got[1], v)):
                off = (have.double() - want).norm(dim=-1) / want.norm(dim=-1)
                if not bool((off <= bound).all()):
                    raise RuntimeError(f"sequence {b}: a cached {name} is off by {float(off.max()):.1e} of its norm")

    def plain_step(self, x):
        """What step(x) returned, recomputed in 64 bits from the weights and the
        cache as it now is (check_cache says whether it is right); activations
        between operators are f16, as there."""
        w_out = qmm.qdequant(self.kind, self.w_out, self.d_model, self.q_heads * self.dim).double()
        q = self.plain_rotation(self.plain_heads(x)[0], self.lens - 1).half().double()
        out = []
        for b, n in enumerate(self.lens.tolist()):
            at = self.slots(torch.arange(n, device="cuda").expand(self.batch, n)).view(self.batch, n)[b].contiguous()
            k, v = (t.double() for t in qmm.qkv_load(self.fmt, at, self.k_cache, self.v_cache, self.page, self.kv_heads, self.dim))
            qb = q[b].view(self.kv_heads, -1, self.dim)
            p = torch.softmax(torch.einsum("hgd,nhd->hgn", qb, k) * self.dim ** -0.5, -1)
            out.append(torch.einsum("hgn,nhd->hgd", p, v).reshape(-1))
        return torch.stack(out).half().double() @ w_out.T


def run(steps=32, batch=4, fmt="q8_0", kind="Q4_0", **sizes):
    """(relative error of the last step against plain_step, microseconds per step)."""
    layer = AttentionLayer(kind, fmt, batch=batch, **sizes)
    prompt = 200 if layer.max_len > 400 else layer.max_len // 4
    if prompt < 1 or steps < 1 or prompt + 1 + steps > layer.max_len:   # a step of its own comes before the replayed ones
        raise ValueError(f"prompts of up to {prompt} tokens and 1 + {steps} steps do not fit {layer.max_len} tokens")
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((batch, prompt, layer.d_model), generator=gen, device="cuda").half()
    lens = torch.randint(1, prompt + 1, (batch,), generator=gen, device="cuda", dtype=torch.int32)
    layer.prompt(x, lens)
    token = torch.randn((batch, layer.d_model), generator=gen, device="cuda").half()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())   # the prompt and the token are still being made there
    with torch.cuda.stream(side):        # a first call outside the capture
        layer.step(token)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.step(token)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(steps):
        graph.replay()
    end.record()
    end.synchronize()
    if qmm.check_device_error():
        raise RuntimeError("a device error was latched")
    layer.check_cache(x, lens, token, 1 + steps)
    want = layer.plain_step(token)
    return float((y.double() - want).norm() / want.norm()), begin.elapsed_time(end) * 1e3 / steps


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--fmt", default="q8_0", choices=sorted(qmm.KV_FORMATS))
    ap.add_argument("--kind", default="Q4_0", choices=qmm.KINDS)
    a = ap.parse_args()
    err, us = run(a.steps, a.batch, a.fmt, a.kind)
    print(f"{a.batch} sequences, {a.kind} weights, {a.fmt} cache: {us:.1f} us per step, last step off by {err:.1e} (relative)")


if __name__ == "__main__":
    main()
