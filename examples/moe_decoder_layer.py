"""A whole decoder layer's decode step with a mixture of experts, on block-quantized
weights and a 4-bit key-value cache: RMS norm, the attention half of
decode_layer.py with normed query and key heads, RMS norm with the residual's
addition, router product, routing to experts, expert products, residual.

    python examples/moe_decoder_layer.py [--steps 32] [--batch 4] [--fmt q4_0] [--kind Q4_0]

runs a batch of sequences of different lengths for some steps, replaying one CUDA
graph per step, checks the last step against a plain 64-bit computation, and
prints the time of a step.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from examples.decode_layer import AttentionLayer  # noqa: E402
from gemv_mul_mm_gb300 import qmm, synth  # noqa: E402


class MoeDecoderLayer(AttentionLayer):
    """The attention half with norms, and the experts' half. The residual stream is fp32."""

    def __init__(self, kind="Q4_0", fmt="q4_0", d_model=1024, experts=32, top_k=4, d_ff=256, seed=1, **sizes):
        super().__init__(kind, fmt, d_model=d_model, seed=seed, **sizes)
        self.experts, self.top_k, self.d_ff = experts, top_k, d_ff
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def norm(n):
            return 1.0 + 0.2 * torch.randn(n, generator=gen, device="cuda")

        self.attn_norm, self.ffn_norm, self.q_norm, self.k_norm = norm(d_model), norm(d_model), norm(self.dim), norm(self.dim)
        self.bias = 0.02 * torch.randn(experts, generator=gen, device="cuda")
        self.w_router = torch.from_numpy(synth.quant_weights("Q8_0", experts, d_model, seed + 2)).cuda()
        self.w_gu = torch.from_numpy(synth.quant_weights(kind, experts * 2 * d_ff, d_model, seed + 3)).cuda()
        self.w_down = torch.from_numpy(synth.quant_weights(kind, experts * d_model, d_ff, seed + 4)).cuda()
        self.moe_ws = torch.empty(qmm.qmoe_ffn_workspace_bytes(self.batch, top_k, d_model, d_ff), dtype=torch.uint8, device="cuda")

    def normed_heads(self, x):
        """heads() of the normed rows of the residual x, with normed queries and keys."""
        q, k, v = self.heads(qmm.qrmsnorm(x, self.attn_norm, out_dtype=torch.float16))
        return qmm.qrmsnorm(q, self.q_norm, out=q), qmm.qrmsnorm(k, self.k_norm, out=k), v

    def prompt(self, x, lens):
        b, n, _ = x.shape
        _, k, v = self.normed_heads(x.reshape(b * n, -1))
        self.store(k, v, torch.arange(n, device="cuda").expand(b, n))
        self.lens.copy_(lens)

    def step(self, x):
        """One new token per sequence: x (batch, d_model) fp32, the residual stream, is updated in place and returned."""
        q, k, v = self.normed_heads(x)
        self.store(k, v, self.lens[:, None])
        q = qmm.qrope(q, self.lens, self.turns, mscale=self.mscale)
        self.lens += 1
        o = qmm.qattn_decode(self.fmt, q, self.k_cache, self.v_cache, self.table, self.lens, self.page, self.kv_heads,
                             max_len=self.max_len)
        o = qmm.qgemm(self.kind, self.w_out, o.view(self.batch, -1), self.d_model, self.q_heads * self.dim, self.batch, weights_const=True)
        h = qmm.qrmsnorm(o, self.ffn_norm, residual=x)                       # x += o, normed for the experts
        logits = qmm.qgemm("Q8_0", self.w_router, h, self.experts, self.d_model, self.batch, weights_const=True)
        ids, weights = qmm.qmoe_route(logits, self.top_k, score="sigmoid", bias=self.bias, groups=4, top_groups=2, group_top=2)
        self.routed = logits, ids, weights
        y = qmm.qmoe_ffn(self.kind, self.w_gu, self.w_gu.numel() // self.experts, self.w_down, self.w_down.numel() // self.experts,
                         self.experts, h, ids, weights, self.d_model, self.d_ff, workspace=self.moe_ws)
        return x.add_(y)

    @staticmethod
    def plain_norm(x, weight):
        x = x.double()
        return x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.double()

    def plain_step(self, x):
        """What step made of the residual x (as it was before), in 64 bits from the weights and
        the cache as it now is; activations between operators are rounded as there. The
        experts are those that step chose: check_routing says whether rightly."""
        q, _, _ = self.plain_heads(self.plain_norm(x, self.attn_norm).half())
        q = self.plain_norm(q, self.q_norm).half()
        q = self.plain_rotation(q, self.lens - 1).half().double()
        out = []
        for b, n in enumerate(self.lens.tolist()):
            at = self.slots(torch.arange(n, device="cuda").expand(self.batch, n)).view(self.batch, n)[b].contiguous()
            k, v = (t.double() for t in qmm.qkv_load(self.fmt, at, self.k_cache, self.v_cache, self.page, self.kv_heads, self.dim))
            qb = q[b].view(self.kv_heads, -1, self.dim)
            p = torch.softmax(torch.einsum("hgd,nhd->hgn", qb, k) * self.dim ** -0.5, -1)
            out.append(torch.einsum("hgn,nhd->hgd", p, v).reshape(-1))
        o = torch.stack(out).half().double() @ qmm.qdequant(self.kind, self.w_out, self.d_model, self.q_heads * self.dim).double().T
        x = x.double() + o
        h = self.plain_norm(x, self.ffn_norm)
        _, ids, weights = self.routed
        gu = qmm.qdequant(self.kind, self.w_gu, self.experts * 2 * self.d_ff, self.d_model).double().view(self.experts, 2 * self.d_ff, -1)
        down = qmm.qdequant(self.kind, self.w_down, self.experts * self.d_model, self.d_ff).double().view(self.experts, self.d_model, -1)
        for j in range(self.top_k):
            e = ids[:, j].long()
            g, u = torch.einsum("bfd,bd->bf", gu[e], h).chunk(2, -1)
            y = torch.einsum("bdf,bf->bd", down[e], g * torch.sigmoid(g) * u)
            x = x + weights[:, j:j + 1].double() * y
        return x

    def check_routing(self):
        """Raises unless the last step's experts and weights are those of its logits, by the definition in 64 bits."""
        logits, ids, weights = self.routed
        s = torch.sigmoid(logits.double())
        c = (s + self.bias.double()).view(self.batch, 4, -1)
        best = c.topk(2, -1).values.sum(-1).topk(2, -1).indices
        keep = torch.zeros(self.batch, 4, dtype=torch.bool, device="cuda").scatter_(1, best, True)
        want = c.masked_fill(~keep[..., None], float("-inf")).flatten(1).topk(self.top_k, -1).indices
        w = s.gather(1, want)
        w = w / w.sum(-1, keepdim=True)
        if not torch.equal(want.int(), ids) or not bool(((weights - w).abs() <= 2.0 ** -18 * w).all()):
            raise RuntimeError("the routing is not that of the logits")


def run(steps=32, batch=4, fmt="q4_0", kind="Q4_0", **sizes):
    """(relative error of what the last step added against plain_step, microseconds per step)."""
    layer = MoeDecoderLayer(kind, fmt, batch=batch, **sizes)
    prompt = 200 if layer.max_len > 400 else layer.max_len // 4
    if prompt < 1 or steps < 1 or prompt + 1 + steps > layer.max_len:   # a step of its own comes before the replayed ones
        raise ValueError(f"prompts of up to {prompt} tokens and 1 + {steps} steps do not fit {layer.max_len} tokens")
    gen = torch.Generator(device="cuda").manual_seed(3)
    layer.prompt(torch.randn((batch, prompt, layer.d_model), generator=gen, device="cuda"),
                 torch.randint(1, prompt + 1, (batch,), generator=gen, device="cuda", dtype=torch.int32))
    token = torch.randn((batch, layer.d_model), generator=gen, device="cuda")
    x = token.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())   # the prompt and the token are still being made there
    with torch.cuda.stream(side):        # a first call outside the capture
        layer.step(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.copy_(token)
        layer.step(x)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(steps):
        graph.replay()
    end.record()
    end.synchronize()
    if qmm.check_device_error():
        raise RuntimeError("a device error was latched")
    layer.check_routing()
    want = layer.plain_step(token)
    return float((x.double() - want).norm() / (want - token.double()).norm()), begin.elapsed_time(end) * 1e3 / steps


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--fmt", default="q4_0", choices=sorted(qmm.KV_FORMATS))
    ap.add_argument("--kind", default="Q4_0", choices=qmm.KINDS)
    a = ap.parse_args()
    err, us = run(a.steps, a.batch, a.fmt, a.kind)
    print(f"{a.batch} sequences, {a.kind} weights, {a.fmt} cache: {us:.1f} us per step, last step off by {err:.1e} (relative)")


if __name__ == "__main__":
    main()
