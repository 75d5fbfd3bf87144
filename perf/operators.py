"""The serving operators around the attention of a decoder layer, as cases that can be timed and compared:
rotary positions, the paged key-value cache (written and read back) and the attention of one new token a
sequence over that cache.

Each case names an operator ("op") and its sizes; ``run`` makes one pass, in plain torch operations in 32 bits
or, where ``own`` is set, through the package's entry points.

The cache is one byte buffer for keys and one for values, a row for each page; in a page each key-value head
has `page` rows of `dim` values: f16 or bf16 as they are, q8_0 as `page` * `dim` codes (int8) followed by
`page` * `dim` / 32 scales (f16), a value being scale * code.

Rotary frequencies are held as turns per position, a 64-bit fraction: the phase of a position is an integer
product, exact at any position.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # one token's 32 query and 8 key heads, rotated as a view of the fused projection: the smallest call, latency alone
        dict(name="rope one token", op="rope", tokens=1, heads=40, dim=128, rot=128, layout="half", dtype="f16",
             base=500000.0, scaling="none", factor=1.0, strided=True, pos_max=32768),
        # a prompt's query heads, frequencies scaled for a long context
        dict(name="rope prompt bf16", op="rope", tokens=8192, heads=32, dim=128, rot=128, layout="half", dtype="bf16",
             base=10000.0, scaling="ramp", factor=16.0, strided=True, pos_max=131072),
        # two thirds of an odd head size rotated, interleaved pairs, fp32 as the products write by default
        dict(name="rope partial f32", op="rope", tokens=2999, heads=20, dim=96, rot=64, layout="interleaved", dtype="f32",
             base=10000.0, scaling="linear", factor=4.0, strided=False, pos_max=65536),
        # the new token of one sequence, rotated, quantised and written; read back
        dict(name="store one token q8_0", op="store", tokens=1, kv_heads=8, dim=128, page=16, fmt="q8_0", dtype="f16",
             rope=True, layout="half", batch=True),
        # a decode batch: each sequence's token goes to a page of its own
        dict(name="store batch bf16", op="store", tokens=129, kv_heads=4, dim=64, page=32, fmt="bf16", dtype="f32",
             rope=True, layout="interleaved", batch=True),
        # a long prompt's keys and values, from the products' fp32
        dict(name="store prompt q8_0", op="store", tokens=16384, kv_heads=8, dim=128, page=64, fmt="q8_0", dtype="f32",
             rope=True, layout="half", batch=False),
        # a short sequence's rows in fp32, an odd head size
        dict(name="load short q8_0", op="load", tokens=701, kv_heads=5, dim=96, page=16, fmt="q8_0", dtype="f32"),
        # a long context read back for a product or another machine
        dict(name="load long q8_0", op="load", tokens=65536, kv_heads=8, dim=128, page=64, fmt="q8_0", dtype="f16"),
        # one user, a short chat: latency
        dict(name="attention one short", op="attention", batch=1, max_len=777, ragged=False, q_heads=32, kv_heads=8, dim=128,
             page=16, fmt="f16", dtype="f16", window=0, softcap=0.0, lse=False),
        # a serving batch of many lengths, one slot empty, quantised cache, fp32 activations
        dict(name="attention batch q8_0 f32", op="attention", batch=24, max_len=8192, ragged=True, q_heads=32, kv_heads=4,
             dim=128, page=32, fmt="q8_0", dtype="f32", window=0, softcap=0.0, lse=True),
        # one user with a very long context: the split over the length
        dict(name="attention one long", op="attention", batch=1, max_len=131072, ragged=False, q_heads=32, kv_heads=8,
             dim=128, page=64, fmt="f16", dtype="f16", window=0, softcap=0.0, lse=False),
        # the largest: a full server
        dict(name="attention large bf16", op="attention", batch=128, max_len=8192, ragged=True, q_heads=32, kv_heads=8,
             dim=128, page=16, fmt="bf16", dtype="bf16", window=0, softcap=0.0, lse=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "store", "load", "attention", "attention"])
    if op == "rope":
        dim = rng.choice([64, 80, 96, 112, 128, 192, 256])
        return dict(op=op, tokens=_log(rng, 1, 8192), heads=rng.randint(1, 40 if dim < 128 else 16), dim=dim,
                    rot=rng.choice([dim, dim, dim // 2, dim // 4]), layout=rng.choice(["half", "interleaved"]),
                    dtype=rng.choice(["f32", "f16", "bf16"]), base=rng.choice([10000.0, 500000.0, 1000000.0]),
                    scaling=rng.choice(["none", "linear", "ramp"]), factor=rng.choice([2.0, 4.0, 8.0, 32.0]),
                    strided=rng.random() < 0.5, pos_max=_log(rng, 1000, 131072))
    dim, page = rng.choice([64, 96, 128, 128, 256]), rng.choice([8, 16, 32, 64, 128, 256])
    fmt, dtype = rng.choice(["f16", "bf16", "q8_0", "q8_0"]), rng.choice(["f32", "f16", "bf16"])
    if op == "store":
        batch = rng.random() < 0.5
        return dict(op=op, tokens=_log(rng, 1, 512) if batch else _log(rng, 8, 8192), kv_heads=rng.randint(1, 8), dim=dim,
                    page=page, fmt=fmt, dtype=dtype, rope=rng.random() < 0.6, layout=rng.choice(["half", "interleaved"]),
                    batch=batch)
    if op == "load":
        return dict(op=op, tokens=_log(rng, 1, 32768), kv_heads=rng.randint(1, 8), dim=dim, page=page, fmt=fmt, dtype=dtype)
    kv_heads, group = rng.choice([1, 2, 4, 5, 8]), rng.choice([1, 2, 3, 4, 7, 8, 8, 12, 16])
    batch = _log(rng, 1, 128)
    most = (1 << 30) // (kv_heads * dim * batch)  # cached values of each kind: at most the largest listed case's
    max_len = _log(rng, 16, min(131072, most))
    return dict(op=op, batch=batch, max_len=max_len, ragged=rng.random() < 0.7, q_heads=kv_heads * group, kv_heads=kv_heads,
                dim=dim, page=page, fmt=fmt, dtype=dtype, window=_log(rng, 16, max_len) if rng.random() < 0.25 else 0,
                softcap=rng.choice([0.0, 0.0, 0.0, 30.0]), lse=rng.random() < 0.5)


def _row_bytes(case):
    """Bytes of one head's row of a token."""
    return case["dim"] * 34 // 32 if case["fmt"] == "q8_0" else 2 * case["dim"]


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
    if op == "rope":
        n = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": 2 * n * SIZES[case["dtype"]] + 4 * case["tokens"] + 4 * case["rot"],
                "flops": 6 * case["tokens"] * case["heads"] * case["rot"] // 2}
    if op in ("store", "load"):
        rows = 2 * case["tokens"] * case["kv_heads"]
        dense, cached = rows * case["dim"] * SIZES[case["dtype"]], rows * _row_bytes(case)
        back = rows * (_row_bytes(case) + 2 * case["dim"]) if op == "store" and case["fmt"] == "q8_0" else 0
        return {"bytes": dense + cached + back + 8 * case["tokens"], "flops": 4 * rows * case["dim"]}
    lens = [min(n, case["window"]) if case["window"] else n for n in _lens(case)]
    io = case["batch"] * case["q_heads"] * (2 * case["dim"] * SIZES[case["dtype"]] + (4 if case["lse"] else 0))
    return {"bytes": 2 * sum(lens) * case["kv_heads"] * _row_bytes(case) + io + sum(lens) // case["page"] * 4,
            "flops": 4 * sum(lens) * case["q_heads"] * case["dim"]}


def _frequencies(case):
    """Radians per position of each rotated pair, in 64 bits, and the factor on the rotated values."""
    rot, base, factor = case.get("rot", case["dim"]), case.get("base", 10000.0), case.get("factor", 1.0)
    i = np.arange(rot // 2, dtype=np.float64)
    f = base ** (-2.0 * i / rot)
    scaling = case.get("scaling", "none")
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "ramp":  # frequencies that turn often in 4096 positions stay, slow ones are stretched, a ramp between
        pair = lambda t: rot * math.log(4096 / (t * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot - 1)
        keep = 1.0 - np.clip((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        return f / factor * (1.0 - keep) + f * keep, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _turns(case):
    f, m = _frequencies(case)
    return torch.from_numpy(np.round(f / (2 * math.pi) * 2.0 ** 64).astype(np.uint64).view(np.int64)).cuda(), m


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(DTYPES[dtype])


def _cache(case, gen, pages):
    """A cache of keys or values with contents, as bytes."""
    n = case["kv_heads"] * case["page"] * case["dim"]
    if case["fmt"] != "q8_0":
        c = torch.empty((pages, n), device="cuda", dtype=DTYPES[case["fmt"]]).normal_(generator=gen)
        return c.view(torch.uint8)
    c = torch.empty((pages, case["kv_heads"], case["page"] * _row_bytes(case)), device="cuda", dtype=torch.uint8)
    codes, scales = _parts(case, c.view(pages, -1))
    codes.random_(-127, 128, generator=gen)
    scales.uniform_(0.005, 0.02, generator=gen)
    return c.view(pages, -1)


def _parts(case, cache):
    """Views of a q8_0 cache: codes [page][head][row][dim] and scales [page][head][row][dim / 32]."""
    h, p, d = case["kv_heads"], case["page"], case["dim"]
    u = cache.view(cache.shape[0], h, p * _row_bytes(case))
    return (u[:, :, : p * d].view(torch.int8).unflatten(2, (p, d)),
            u[:, :, p * d:].view(torch.float16).unflatten(2, (p, d // 32)))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = np.random.RandomState(seed & 0x7FFFFFFF)
    s = {"case": case}
    op = case["op"]
    if op == "rope":
        t, h, d = case["tokens"], case["heads"], case["dim"]
        s["turns"], s["mscale"] = _turns(case)
        start = int(host.randint(0, max(1, case["pos_max"] - t)))
        s["pos"] = torch.arange(start, start + t, device="cuda", dtype=torch.int32)
        x = _normal(gen, (t, h + (8 if case["strided"] else 0), d), case["dtype"])
        s["x"] = x[:, :h]
        return s
    page = case["page"]
    if op in ("store", "load"):
        t, h, d = case["tokens"], case["kv_heads"], case["dim"]
        if op == "store" and case["batch"]:  # a token for each sequence, somewhere in that sequence's last page
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
        if op == "store":
            s["turns"], s["mscale"] = _turns(case)
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


def _rotate(x, pos, turns, mscale, layout):
    """Rotated x (32 bits): the phase is the top half of pos * turns."""
    rot = 2 * turns.shape[0]
    a = ((pos.to(torch.int64)[:, None] * turns) >> 32).float() * (2 * math.pi / 2 ** 32)
    c, n = (torch.cos(a) * mscale)[:, None], (torch.sin(a) * mscale)[:, None]
    x = x.float()
    if layout == "half":
        x1, x2 = x[..., : rot // 2], x[..., rot // 2: rot]
        return torch.cat([x1 * c - x2 * n, x2 * c + x1 * n, x[..., rot:]], -1)
    x1, x2 = x[..., 0:rot:2], x[..., 1:rot:2]
    return torch.cat([torch.stack([x1 * c - x2 * n, x2 * c + x1 * n], -1).flatten(-2), x[..., rot:]], -1)


def _write(case, cache, rows, slots):
    page, at = slots // case["page"], slots % case["page"]
    if case["fmt"] != "q8_0":
        typed = cache.view(DTYPES[case["fmt"]]).view(-1, case["kv_heads"], case["page"], case["dim"])
        typed[page, :, at] = rows.to(typed.dtype)
        return
    blocks = rows.unflatten(-1, (-1, 32))
    most = blocks.abs().amax(-1)
    scale = (most / torch.full_like(most, 127.0)).half()
    d = scale.float()[..., None]
    code = torch.where(d > 0, torch.round(blocks / d), torch.zeros_like(blocks)).clamp(-127, 127)
    codes, scales = _parts(case, cache)
    codes[page, :, at] = code.flatten(-2).to(torch.int8)
    scales[page, :, at] = scale


def _read(case, cache, slots):
    """Rows (32 bits) of `slots`, of any shape: [..., head, dim]."""
    page, at = slots // case["page"], slots % case["page"]
    if case["fmt"] != "q8_0":
        typed = cache.view(DTYPES[case["fmt"]]).view(-1, case["kv_heads"], case["page"], case["dim"])
        return typed[page, :, at].float()
    codes, scales = _parts(case, cache)
    return (codes[page, :, at].float().unflatten(-1, (-1, 32)) * scales[page, :, at].float()[..., None]).flatten(-2)


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
        if op == "rope":
            return qmm.qrope(s["x"], s["pos"], s["turns"], layout=case["layout"], mscale=s["mscale"])
        if op == "store":
            rotary = dict(positions=s["pos"], turns=s["turns"], layout=case["layout"]) if case["rope"] else {}
            qmm.qkv_store(case["fmt"], s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], case["page"], **rotary)
            if case["fmt"] == "q8_0":
                return qmm.qkv_load("q8_0", s["slots"], s["k_cache"], s["v_cache"], case["page"], case["kv_heads"],
                                    case["dim"], dtype=torch.float16)
            return s["k_cache"].view(DTYPES[case["fmt"]]), s["v_cache"].view(DTYPES[case["fmt"]])
        if op == "load":
            return qmm.qkv_load(case["fmt"], s["slots"], s["k_cache"], s["v_cache"], case["page"], case["kv_heads"],
                                case["dim"], dtype=DTYPES[case["dtype"]])
        return qmm.qattn_decode(case["fmt"], s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], case["page"],
                                case["kv_heads"], window=case["window"], softcap=case["softcap"],
                                max_len=case["max_len"], return_lse=case["lse"])
    if op == "rope":
        return _rotate(s["x"], s["pos"], s["turns"], s["mscale"], case["layout"]).to(s["x"].dtype)
    if op == "store":
        k = _rotate(s["k"], s["pos"], s["turns"], s["mscale"], case["layout"]) if case["rope"] else s["k"].float()
        _write(case, s["k_cache"], k, s["slots"])
        _write(case, s["v_cache"], s["v"].float(), s["slots"])
        if case["fmt"] == "q8_0":
            return _read(case, s["k_cache"], s["slots"]).half(), _read(case, s["v_cache"], s["slots"]).half()
        return s["k_cache"].view(DTYPES[case["fmt"]]), s["v_cache"].view(DTYPES[case["fmt"]])
    if op == "load":
        return tuple(_read(case, s[c], s["slots"]).to(DTYPES[case["dtype"]]) for c in ("k_cache", "v_cache"))
    o, lse = _attend(case, s)
    return (o, lse) if case["lse"] else o


def _exact_rows(case, cache, slots):
    """Values of `slots` [n] in 64 bits, [n][head][dim], read from the bytes."""
    h, p, d = case["kv_heads"], case["page"], case["dim"]
    unit = cache.reshape(cache.shape[0], h, -1)
    page, row = torch.div(slots, p, rounding_mode="floor"), torch.remainder(slots, p)
    head = torch.arange(h, device="cuda")[None, :, None]
    pg = page[:, None, None]
    if case["fmt"] != "q8_0":
        return unit.view(DTYPES[case["fmt"]])[pg, head, (row * d)[:, None, None] + torch.arange(d, device="cuda")].double()
    code = unit[pg, head, (row * d)[:, None, None] + torch.arange(d, device="cuda")].view(torch.int8).double()
    where = (p * d + 2 * (row * (d // 32)))[:, None, None] + torch.arange(d // 16, device="cuda")
    scale = unit[pg, head, where].view(torch.float16).double()
    return code * torch.repeat_interleave(scale, 32, dim=2)


def _exact_rotation(case, x, pos):
    f, m = _frequencies(case)
    angle = pos.double()[:, None, None] * torch.from_numpy(f).cuda()
    n = f.shape[0]
    first, second = (slice(0, n), slice(n, 2 * n)) if case["layout"] == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    z = torch.complex(x.double()[..., first], x.double()[..., second]) * torch.polar(torch.full_like(angle, m), angle)
    y = x.double().clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return _exact_rotation(case, s["x"], s["pos"])
    if op == "load":
        return tuple(_exact_rows(case, s[c], s["slots"]) for c in ("k_cache", "v_cache"))
    if op == "store":
        rows = (_exact_rotation(case, s["k"], s["pos"]) if case["rope"] else s["k"].double(), s["v"].double())
        if case["fmt"] == "q8_0":  # the nearest code of the stored scale
            got = []
            for x in rows:
                b = x.reshape(*x.shape[:2], -1, 32)
                d = (b.abs().max(dim=-1, keepdim=True).values / 127).half().double()
                got.append((torch.round(b / d).clamp(-127, 127) * d).reshape(x.shape))
            return tuple(got)
        out = []
        for c, x in (("k_cache", rows[0]), ("v_cache", rows[1])):
            full = s[c].view(DTYPES[case["fmt"]]).double().view(-1, case["kv_heads"], case["page"], case["dim"])
            full[torch.div(s["slots"], case["page"], rounding_mode="floor"), :, torch.remainder(s["slots"], case["page"])] = x
            out.append(full.reshape(s[c].shape[0], -1))
        return tuple(out)
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
