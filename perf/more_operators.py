"""The rest of a decoder layer's serving operators, as cases that can be timed and compared: the RMS norm with the
residual's addition, the routing of tokens to experts, and the key-value cache in 4 bits (written, read back, attended).

Each case names an operator ("op") and its sizes; ``run`` makes one pass, in plain torch operations or, where
``own`` is set, through the package's entry points.

A q4_0 cache is one byte buffer for keys and one for values, a row for each page; in a page each key-value head has
`page` * `dim` / 2 bytes of codes, [page][dim / 2] (element 2 j in the low half of byte j, 2 j + 1 in the high half, each
code plus 8), followed by `page` * `dim` / 32 scales (f16). A value is scale * code, code in [-8, 7].

A q8_0 row is dim / 32 blocks of an f16 scale and 32 int8 codes.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # one token of a decode step, before a projection on f16 activations: the smallest call, latency alone
        dict(name="norm one token", op="norm", tokens=1, heads=1, dim=4096, x="f32", residual="f32", out="f16", offset=0.0),
        # each query and key head of a batch, as a view of the fused projection
        dict(name="norm heads f16", op="norm", tokens=512, heads=40, dim=128, x="f16", residual="none", out="f16", offset=0.0),
        # a long prompt's residual stream
        dict(name="norm prompt bf16", op="norm", tokens=16384, heads=1, dim=4096, x="bf16", residual="bf16", out="bf16", offset=0.0),
        # rows in blocks with scales, as weights of a later product have them; weights held as 1 + w, an odd count
        dict(name="norm rows q8_0", op="norm", tokens=3001, heads=1, dim=2048, x="f32", residual="f32", out="q8_0", offset=1.0),
        # one token of a decode step
        dict(name="route one token", op="route", tokens=1, experts=128, top_k=8, score="softmax", bias=False, groups=1,
             top_groups=1, group_top=1, renorm=True, scale=1.0, dtype="f32"),
        # a prompt over many experts, balanced by a bias, limited to half of the groups
        dict(name="route groups f32", op="route", tokens=8192, experts=256, top_k=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, group_top=2, renorm=True, scale=2.5, dtype="f32"),
        # a long prompt, logits of a 16-bit product with many equal ones
        dict(name="route prompt bf16", op="route", tokens=65536, experts=128, top_k=8, score="softmax", bias=False, groups=1,
             top_groups=1, group_top=1, renorm=True, scale=1.0, dtype="bf16"),
        # a decode batch's keys and values, each token to a page of its own; read back
        dict(name="store batch q4_0", op="store", tokens=129, kv_heads=8, dim=128, page=16, dtype="f16", rope=True,
             layout="half", batch=True),
        # a long prompt's keys and values, from the products' fp32; read back
        dict(name="store prompt q4_0", op="store", tokens=16384, kv_heads=8, dim=128, page=64, dtype="f32", rope=True,
             layout="half", batch=False),
        # one user, a short chat: latency
        dict(name="attention one short", op="attention", batch=1, max_len=777, ragged=False, q_heads=32, kv_heads=8, dim=128,
             page=16, dtype="f16", window=0, softcap=0.0, lse=False),
        # one user with a very long context: the split over the length; fp32 activations
        dict(name="attention one long f32", op="attention", batch=1, max_len=131072, ragged=False, q_heads=32, kv_heads=8,
             dim=128, page=64, dtype="f32", window=0, softcap=0.0, lse=True),
        # the largest: a full server
        dict(name="attention large", op="attention", batch=128, max_len=8192, ragged=True, q_heads=32, kv_heads=8, dim=128,
             page=32, dtype="f16", window=0, softcap=0.0, lse=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "route", "route", "store", "attention", "attention"])
    types = ["f32", "f16", "bf16"]
    if op == "norm":
        heads = rng.choice([1, 1, 1, rng.randint(2, 48)])
        out = rng.choice(types + ["q8_0"]) if heads == 1 else rng.choice(types)
        if heads > 1:
            dim, tokens = rng.choice([64, 80, 96, 128, 192, 256]), _log(rng, 1, 4096)
        else:
            dim = 32 * _log(rng, 2, 512) if out == "q8_0" else rng.choice([_log(rng, 33, 16384), 64 * _log(rng, 1, 256)])
            tokens = _log(rng, 1, min(16384, (1 << 25) // dim))
        return dict(op=op, tokens=tokens, heads=heads, dim=dim, x=rng.choice(types),
                    residual=rng.choice(types + ["none"]) if heads == 1 else "none", out=out, offset=rng.choice([0.0, 0.0, 1.0]))
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * rng.choice([4, 8, 16, 20, 32, 45, 64])
        top_groups = rng.randint(1, groups)
        return dict(op=op, tokens=_log(rng, 1, 65536), experts=experts, top_k=rng.randint(1, min(10, top_groups * experts // groups)),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups, top_groups=top_groups,
                    group_top=rng.choice([1, 2]), renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]), dtype=rng.choice(types))
    dim, page, dtype = rng.choice([64, 96, 128, 128, 256]), rng.choice([8, 16, 32, 64, 128, 256]), rng.choice(types)
    if op == "store":
        batch = rng.random() < 0.5
        return dict(op=op, tokens=_log(rng, 1, 512) if batch else _log(rng, 8, 8192), kv_heads=rng.randint(1, 8), dim=dim,
                    page=page, dtype=dtype, rope=rng.random() < 0.6, layout=rng.choice(["half", "interleaved"]), batch=batch)
    kv_heads, group = rng.choice([1, 2, 4, 5, 8]), rng.choice([1, 2, 3, 4, 7, 8, 8, 12, 16])
    batch = _log(rng, 1, 128)
    # cached values of each kind: at most the largest listed case's; fewer where many heads share them
    most = (1 << (29 if group <= 8 else 28)) // (kv_heads * dim * batch)
    max_len = _log(rng, 16, min(131072, most))
    return dict(op=op, batch=batch, max_len=max_len, ragged=rng.random() < 0.7, q_heads=kv_heads * group, kv_heads=kv_heads,
                dim=dim, page=page, dtype=dtype, window=_log(rng, 16, max_len) if rng.random() < 0.25 else 0,
                softcap=rng.choice([0.0, 0.0, 0.0, 30.0]), lse=rng.random() < 0.5)


def _lens(case):
    """The lengths of a batch: a ragged one has its longest first and, from four sequences on, an empty one last."""
    n, top = case["batch"], case["max_len"]
    if not case["ragged"]:
        return [top] * n
    lens = np.random.RandomState(n * 7 + top).randint(1, top + 1, size=n)
    lens[0] = top
    if n >= 4:
        lens[-1] = 0
    return [int(v) for v in lens]


def work(case):
    op = case["op"]
    if op == "norm":
        n = case["tokens"] * case["heads"] * case["dim"]
        res = 0 if case["residual"] == "none" else 2 * n * SIZES[case["residual"]]
        out = n * 34 // 32 * 2 + 2 * n if case["out"] == "q8_0" else n * SIZES[case["out"]]  # blocks: written, read back as values
        return {"bytes": n * SIZES[case["x"]] + res + out + 4 * case["dim"], "flops": 5 * n}
    if op == "route":
        t, e = case["tokens"], case["experts"]
        return {"bytes": t * e * SIZES[case["dtype"]] + 8 * t * case["top_k"] + (4 * e if case["bias"] else 0), "flops": 4 * t * e}
    row = case["dim"] * 18 // 32
    if op == "store":
        rows = 2 * case["tokens"] * case["kv_heads"]
        return {"bytes": rows * (case["dim"] * SIZES[case["dtype"]] + 2 * row + 2 * case["dim"]) + 8 * case["tokens"],
                "flops": 4 * rows * case["dim"]}
    lens = [min(n, case["window"]) if case["window"] else n for n in _lens(case)]
    io = case["batch"] * case["q_heads"] * (2 * case["dim"] * SIZES[case["dtype"]] + (4 if case["lse"] else 0))
    return {"bytes": 2 * sum(lens) * case["kv_heads"] * row + io + sum(lens) // case["page"] * 4,
            "flops": 4 * sum(lens) * case["q_heads"] * case["dim"]}


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(DTYPES[dtype])


def _cache(case, gen, pages):
    """A q4_0 cache of keys or values with contents, as bytes."""
    h, p, d = case["kv_heads"], case["page"], case["dim"]
    c = torch.empty((pages, h, p * d * 18 // 32), device="cuda", dtype=torch.uint8)
    c[:, :, : p * d // 2].random_(0, 256, generator=gen)
    c[:, :, p * d // 2:].view(torch.float16).uniform_(-0.4, 0.4, generator=gen)
    return c.view(pages, -1)


def _parts(case, cache):
    """Views of a q4_0 cache: code bytes [page][head][row][dim / 2] and scales [page][head][row][dim / 32]."""
    h, p, d = case["kv_heads"], case["page"], case["dim"]
    u = cache.view(cache.shape[0], h, p * d * 18 // 32)
    return u[:, :, : p * d // 2].unflatten(2, (p, d // 2)), u[:, :, p * d // 2:].view(torch.float16).unflatten(2, (p, d // 32))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = np.random.RandomState(seed & 0x7FFFFFFF)
    s = {"case": case}
    op = case["op"]
    if op == "norm":
        t, h, d = case["tokens"], case["heads"], case["dim"]
        x = _normal(gen, (t, h + (8 if h > 1 else 0), d), case["x"])  # heads: the projection's rows hold the values too
        s["x"] = x[:, :h] if h > 1 else x[:, 0]
        if case["residual"] != "none":
            s["residual"] = (3.0 * _normal(gen, (t, d), "f32")).to(DTYPES[case["residual"]])
        s["weight"] = 1.0 - case["offset"] + 0.2 * _normal(gen, (d,), "f32")
        return s
    if op == "route":
        t, e = case["tokens"], case["experts"]
        s["logits"] = (1.5 * _normal(gen, (t, e), "f32")).to(DTYPES[case["dtype"]])
        s["bias"] = 0.1 * _normal(gen, (e,), "f32") if case["bias"] else None
        return s
    page = case["page"]
    if op == "store":
        t, h, d = case["tokens"], case["kv_heads"], case["dim"]
        if case["batch"]:  # a token for each sequence, somewhere in that sequence's last page
            pages = t + 3
            slots = host.permutation(pages)[:t].astype(np.int64) * page + host.randint(0, page, size=t)
            s["pos"] = torch.from_numpy(host.randint(0, 32768, size=t).astype(np.int32)).cuda()
        else:  # consecutive tokens over pages in any order, from the middle of a page on
            first = int(host.randint(0, page))
            pages = (first + t - 1) // page + 4
            at = np.arange(first, first + t)
            slots = host.permutation(pages)[at // page].astype(np.int64) * page + at % page
            s["pos"] = torch.arange(5000, 5000 + t, device="cuda", dtype=torch.int32)
        s["slots"] = torch.from_numpy(slots).cuda()
        s["k_cache"], s["v_cache"] = _cache(case, gen, pages), _cache(case, gen, pages)
        turns = 10000.0 ** (-2.0 * np.arange(d // 2) / d) / (2 * math.pi)  # turns per position, as 64-bit fractions
        s["turns"] = torch.from_numpy(np.round(turns * 2.0 ** 64).astype(np.uint64).view(np.int64)).cuda()
        kv = _normal(gen, (t, 2 * h, d), case["dtype"])  # the projection's rows: keys, then values
        s["k"], s["v"] = kv[:, :h], kv[:, h:]
        return s
    lens = _lens(case)
    width = max(1, (case["max_len"] + page - 1) // page)
    need = [(n + page - 1) // page for n in lens]
    order = host.permutation(sum(need) + 2)
    table = np.full((len(lens), width), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    s["table"] = torch.from_numpy(table).cuda()
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["q"] = (1.5 * _normal(gen, (len(lens), case["q_heads"], case["dim"]), "f32")).to(DTYPES[case["dtype"]])
    s["k_cache"], s["v_cache"] = _cache(case, gen, len(order)), _cache(case, gen, len(order))
    return s


def _norm(case, s):
    h = s["x"].float()
    if "residual" in s:
        h = h + s["residual"].float()
        s["residual"].copy_(h)
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * (s["weight"] + case["offset"])
    if case["out"] != "q8_0":
        return y.to(DTYPES[case["out"]])
    b = y.unflatten(-1, (-1, 32))
    most = b.abs().amax(-1, keepdim=True)
    d = (most / torch.full_like(most, 127.0)).half().float()
    code = torch.where(d > 0, torch.round(b / d), torch.zeros_like(b)).clamp(-127, 127)
    return (code * d).flatten(-2).half()


def _route(case, s):
    """In 64 bits: scores next to one another have to be told apart."""
    x = s["logits"].double()
    if case["score"] == "softmax":
        e = torch.exp(x - x.amax(-1, keepdim=True))
        score = e / e.sum(-1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    c = score if s["bias"] is None else score + s["bias"].double()
    if case["groups"] > 1:
        by = c.unflatten(-1, (case["groups"], -1))
        value = by.sort(dim=-1, descending=True).values[..., : case["group_top"]].sum(-1)
        best = value.sort(dim=-1, descending=True, stable=True).indices[..., : case["top_groups"]]
        keep = torch.zeros_like(value, dtype=torch.bool).scatter_(-1, best, True)
        c = by.masked_fill(~keep[..., None], float("-inf")).flatten(-2)
    ids = c.sort(dim=-1, descending=True, stable=True).indices[..., : case["top_k"]]
    w = torch.gather(score, -1, ids)
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return ids.int(), (w * case["scale"]).float()


def _rotate(x, pos, turns, layout):
    """Rotated x (32 bits): the phase is the top half of pos * turns."""
    a = ((pos.to(torch.int64)[:, None] * turns) >> 32).float() * (2 * math.pi / 2 ** 32)
    c, n = torch.cos(a)[:, None], torch.sin(a)[:, None]
    x = x.float()
    if layout == "half":
        x1, x2 = x.chunk(2, -1)
        return torch.cat([x1 * c - x2 * n, x2 * c + x1 * n], -1)
    x1, x2 = x[..., 0::2], x[..., 1::2]
    return torch.stack([x1 * c - x2 * n, x2 * c + x1 * n], -1).flatten(-2)


def _write(case, cache, rows, slots):
    page, at = slots // case["page"], slots % case["page"]
    b = rows.unflatten(-1, (-1, 32))
    first = b.abs().argmax(-1, keepdim=True)  # scales have the sign of the largest value
    scale = (torch.gather(b, -1, first) / -8.0).half()
    d = scale.float()
    code = torch.where(d != 0, torch.round(b / d), torch.zeros_like(b)).clamp(-8, 7) + 8
    code = code.flatten(-2).to(torch.uint8)
    codes, scales = _parts(case, cache)
    codes[page, :, at] = code[..., 0::2] | (code[..., 1::2] << 4)
    scales[page, :, at] = scale.squeeze(-1)


def _read(case, cache, slots):
    """Rows (32 bits) of `slots`, of any shape: [..., head, dim]."""
    page, at = slots // case["page"], slots % case["page"]
    codes, scales = _parts(case, cache)
    u = codes[page, :, at]
    v = torch.stack([u & 15, u >> 4], -1).flatten(-2).float() - 8.0
    return (v.unflatten(-1, (-1, 32)) * scales[page, :, at].float()[..., None]).flatten(-2)


def _attend(case, s):
    page, h = case["page"], case["kv_heads"]
    at = torch.arange(case["max_len"], device="cuda")
    lens = s["lens"].to(torch.int64)[:, None]
    valid = at < lens
    if case["window"]:
        valid &= at >= lens - case["window"]
    slots = s["table"].to(torch.int64)[:, at // page] * page + at % page
    slots = torch.where(valid, slots, torch.zeros_like(slots))
    k = _read(case, s["k_cache"], slots).transpose(1, 2)                   # [batch][head][position][dim]
    q = s["q"].float().unflatten(1, (h, -1))                               # [batch][head][group][dim]
    score = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(case["dim"])
    del k
    if case["softcap"]:
        score = case["softcap"] * torch.tanh(score / case["softcap"])
    score = score.masked_fill(~valid[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    v = torch.where(valid[:, None, :, None], _read(case, s["v_cache"], slots).transpose(1, 2), 0.0)
    o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    return o.flatten(1, 2).to(s["q"].dtype), (top + torch.log(total)).flatten(1)


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        from gemv_mul_mm_gb300 import qmm
        if op == "norm":
            out = "q8_0" if case["out"] == "q8_0" else DTYPES[case["out"]]
            y = qmm.qrmsnorm(s["x"], s["weight"], eps=1e-6, residual=s.get("residual"), out_dtype=out, weight_offset=case["offset"])
            if case["out"] == "q8_0":
                y = qmm.qdequant("Q8_0", y, case["tokens"], case["dim"]).half()
            return (y, s["residual"]) if "residual" in s else y
        if op == "route":
            return qmm.qmoe_route(s["logits"], case["top_k"], score=case["score"], bias=s["bias"], groups=case["groups"],
                                  top_groups=case["top_groups"], group_top=case["group_top"], renorm=case["renorm"],
                                  scale=case["scale"])
        if op == "store":
            rotary = dict(positions=s["pos"], turns=s["turns"], layout=case["layout"]) if case["rope"] else {}
            qmm.qkv_store("q4_0", s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], case["page"], **rotary)
            return qmm.qkv_load("q4_0", s["slots"], s["k_cache"], s["v_cache"], case["page"], case["kv_heads"], case["dim"],
                                dtype=torch.float16)
        return qmm.qattn_decode("q4_0", s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], case["page"],
                                case["kv_heads"], window=case["window"], softcap=case["softcap"], max_len=case["max_len"],
                                return_lse=case["lse"])
    if op == "norm":
        y = _norm(case, s)
        return (y, s["residual"]) if "residual" in s else y
    if op == "route":
        return _route(case, s)
    if op == "store":
        k = _rotate(s["k"], s["pos"], s["turns"], case["layout"]) if case["rope"] else s["k"].float()
        _write(case, s["k_cache"], k, s["slots"])
        _write(case, s["v_cache"], s["v"].float(), s["slots"])
        return _read(case, s["k_cache"], s["slots"]).half(), _read(case, s["v_cache"], s["slots"]).half()
    o, lse = _attend(case, s)
    return (o, lse) if case["lse"] else o


def _exact_rows(case, cache, slots):
    """Values of `slots` [n] in 64 bits, [n][head][dim], read from the bytes."""
    h, p, d = case["kv_heads"], case["page"], case["dim"]
    unit = cache.reshape(cache.shape[0], h, -1)
    page, row = torch.div(slots, p, rounding_mode="floor")[:, None, None], torch.remainder(slots, p)[:, None, None]
    head, i = torch.arange(h, device="cuda")[None, :, None], torch.arange(d, device="cuda")
    byte = unit[page, head, row * (d // 2) + torch.div(i, 2, rounding_mode="floor")].to(torch.int64)
    code = torch.div(byte, 16 ** (i % 2), rounding_mode="floor") % 16 - 8
    raw = unit[page, head, p * d // 2 + 2 * (row * (d // 32)) + torch.arange(d // 16, device="cuda")]
    return code.double() * torch.repeat_interleave(raw.view(torch.float16).double(), 32, dim=2)


def _exact_norm(case, s):
    h = s["x"].double() + (s["residual"].double() if "residual" in s else 0.0)
    y = h / torch.sqrt((h * h).sum(-1, keepdim=True) / case["dim"] + 1e-6) * (s["weight"].double() + case["offset"])
    if case["out"] == "q8_0":  # the nearest code of the stored scale
        b = y.reshape(y.shape[0], -1, 32)
        d = (b.abs().max(dim=-1, keepdim=True).values / 127).half().double()
        y = (torch.round(b / d).clamp(-127, 127) * d).reshape(y.shape)
    return (y, h) if "residual" in s else y


def _exact_route(case, s):
    """The selection by ranks: how many experts (or groups) come before each."""
    x = s["logits"].double()
    score = torch.softmax(x, -1) if case["score"] == "softmax" else torch.sigmoid(x)
    c = score + (0.0 if s["bias"] is None else s["bias"].double())
    t, e, g = case["tokens"], case["experts"], case["groups"]

    def rank(v):
        i = torch.arange(v.shape[1], device="cuda")
        return torch.stack([((v > v[:, j:j + 1]) | ((v == v[:, j:j + 1]) & (i < j))).sum(-1) for j in range(v.shape[1])], -1)

    by = c.reshape(t, g, e // g)
    value = torch.topk(by, min(case["group_top"], e // g), dim=-1).values.sum(-1)
    kept = (rank(value) < case["top_groups"])[:, :, None].expand(-1, -1, e // g).reshape(t, e)
    place = rank(torch.where(kept, c, torch.full_like(c, float("-inf"))))
    ids = place.argsort(-1)[:, : case["top_k"]]
    w = score.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return ids.int(), w * case["scale"]


def _exact_rotation(case, x, pos):
    n = case["dim"] // 2
    f = 10000.0 ** (-torch.arange(n, device="cuda", dtype=torch.float64) / n)
    angle = pos.double()[:, None, None] * f
    first, second = (slice(0, n), slice(n, 2 * n)) if case["layout"] == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    z = torch.complex(x.double()[..., first], x.double()[..., second]) * torch.polar(torch.ones_like(angle), angle)
    y = x.double().clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        return _exact_norm(case, s)
    if op == "route":
        return _exact_route(case, s)
    if op == "store":  # the nearest code of the stored scale
        got = []
        for x in (_exact_rotation(case, s["k"], s["pos"]) if case["rope"] else s["k"].double(), s["v"].double()):
            b = x.reshape(*x.shape[:2], -1, 32)
            high, low = b.max(dim=-1, keepdim=True).values, b.min(dim=-1, keepdim=True).values
            i = torch.arange(32, device="cuda")
            before = torch.where(b == high, i, 32).amin(-1, keepdim=True) < torch.where(b == low, i, 32).amin(-1, keepdim=True)
            m = torch.where((high > -low) | ((high == -low) & before), high, low)
            d = (m / -8).half().double()
            got.append((torch.where(d == 0, 0.0, torch.round(b / d)).clamp(-8, 7) * d).reshape(x.shape))
        return tuple(got)
    group = case["q_heads"] // case["kv_heads"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], float("-inf"), dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lens(case)):
        lo = max(0, n - case["window"]) if case["window"] else 0
        at = torch.arange(lo, n, device="cuda")
        if not len(at):
            continue
        slots = s["table"][b].long()[torch.div(at, case["page"], rounding_mode="floor")] * case["page"] + at % case["page"]
        k, v = (_exact_rows(case, s[c], slots) for c in ("k_cache", "v_cache"))
        q = s["q"][b].double().reshape(case["kv_heads"], group, case["dim"])
        x = torch.einsum("hgd,nhd->hgn", q, k) * case["dim"] ** -0.5
        if case["softcap"]:
            x = torch.tanh(x / case["softcap"]) * case["softcap"]
        lse[b] = torch.logsumexp(x, -1).reshape(-1)
        o[b] = torch.einsum("hgn,nhd->hgd", torch.softmax(x, -1), v).reshape(-1, case["dim"])
    return (o, lse) if case["lse"] else o
