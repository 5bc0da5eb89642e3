"""Cases and plain forms of the token operators: attention of new tokens over a
paged key/value cache, writing and reading that cache in 8 bits, RMS
normalisation with the residual's addition and an 8-bit output, and products
with 4-bit weights.

`own` chooses between the plain forms (elementary torch operations in 32 bits)
and the package's kernels.  `exact` gives each operator's definition in 64 bits.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
# Position of weight k (mod 8) among the eight nibbles of its packed word.
_NIBBLE = (0, 4, 1, 5, 2, 6, 3, 7)


# ------------------------------------------------------------------ the cases
def _attention(name, batch, tokens, context, heads, kv_heads, head_dim, page, cache, causal=True, window=0, ragged=False):
    return dict(name=name, op="attention", batch=batch, tokens=tokens, context=context, heads=heads, kv_heads=kv_heads,
                head_dim=head_dim, page=page, cache=cache, causal=causal, window=window, ragged=ragged)


def _cache(name, batch, tokens, context, kv_heads, head_dim, page, cache, ragged=False):
    return dict(name=name, op="cache", batch=batch, tokens=tokens, context=context, kv_heads=kv_heads,
                head_dim=head_dim, page=page, cache=cache, ragged=ragged)


def _norm(name, rows, cols, dtype, residual, out):
    return dict(name=name, op="norm", rows=rows, cols=cols, dtype=dtype, residual=residual, out=out)


def _linear(name, rows, n, k, group, x, zeros, bias, silu, out):
    return dict(name=name, op="linear", rows=rows, n=n, k=k, group=group, x=x, zeros=zeros, bias=bias, silu=silu, out=out)


def listed():
    return [
        # One stream answering token by token over a short history: latency alone.
        _attention("attention 1 token", 1, 1, 1000, 32, 8, 128, 16, "bf16"),
        # A full server: 64 streams of differing long histories, each one token further, the cache in 8 bits.
        _attention("attention 64 streams int8", 64, 1, 8192, 32, 8, 128, 64, "int8", ragged=True),
        # The cells of 16 images' 20x20 feature maps, each image's cells seeing one another (no causal order).
        _attention("attention 20x20 maps", 16, 400, 400, 8, 8, 64, 16, "bf16", causal=False),
        # A chunk of a long prompt over what came before it.
        _attention("attention chunk of 2048", 1, 2048, 32768, 32, 8, 128, 64, "bf16"),
        # Chunks of odd lengths in one call, sliding window, cache in 8 bits.
        _attention("attention odd chunks int8", 5, 333, 5001, 24, 4, 64, 32, "int8", window=2000, ragged=True),
        # One new token of each of 16 streams into the 8-bit cache, and the histories read back.
        _cache("cache 16 tokens int8", 16, 1, 600, 8, 128, 16, "int8", ragged=True),
        # Prompt chunks written in 8 bits and read back whole, as for moving a cache elsewhere.
        _cache("cache chunks int8", 4, 2048, 16384, 8, 128, 64, "int8"),
        # A few rows of odd width in float, as a small head normalises its inputs.
        _norm("norm 3 rows", 3, 1000, "fp32", False, "same"),
        # A prompt chunk's residual stream, normalised to 8 bits for the products that follow.
        _norm("norm 8192 rows int8", 8192, 4096, "bf16", True, "int8"),
        # One token through a layer's fused query/key/value product, inputs in 8 bits.
        _linear("linear 1 token", 1, 6144, 4096, 128, "int8", False, False, False, "bf16"),
        # An odd output width with the finest groups, bias and SiLU.
        _linear("linear 5 tokens odd", 5, 1001, 2048, 32, "bf16", True, True, True, "fp32"),
        # A batch of streams through a wide layer; its weights do not fit the L2 cache between passes.
        _linear("linear 16 tokens wide", 16, 16384, 8192, 64, "bf16", True, False, False, "bf16"),
    ]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm (round ones are the listed cases')."""
    n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n - 1 if n % 1024 == 0 else n


def _scores(c):
    return c["batch"] * c["heads"] * c["tokens"] * c["context"]


def draw(rng):
    op = rng.choice(("attention", "attention", "cache", "norm", "linear"))
    if op == "attention":
        kv = rng.choice((1, 2, 4, 8))
        c = dict(op=op, batch=_log_int(rng, 1, 64), tokens=1 if rng.random() < 0.4 else _log_int(rng, 2, 2048),
                 context=_log_int(rng, 16, 32768), heads=kv * rng.choice((1, 2, 3, 4, 6, 8)), kv_heads=kv,
                 head_dim=rng.choice((64, 128)), page=rng.choice((16, 32, 64)), cache=rng.choice(("bf16", "int8")),
                 causal=rng.random() < 0.8, window=0, ragged=rng.random() < 0.7)
        c["tokens"] = min(c["tokens"], c["context"])
        if c["causal"] and rng.random() < 0.2:
            c["window"] = _log_int(rng, 64, 4096)
        # no more scores, and no larger a cache, than the largest listed cases'
        while _scores(c) > 32 * 2048 * 30000 or c["batch"] * c["context"] * kv > 64 * 8192 * 8:
            c["batch" if c["batch"] > 1 else "tokens"] = (c["batch"] if c["batch"] > 1 else c["tokens"]) // 2
        return c
    if op == "cache":
        kv = rng.choice((1, 2, 4, 8))
        c = dict(op=op, batch=_log_int(rng, 1, 64), tokens=1 if rng.random() < 0.4 else _log_int(rng, 2, 2048),
                 context=_log_int(rng, 16, 16384), kv_heads=kv, head_dim=rng.choice((64, 128)),
                 page=rng.choice((16, 32, 64)), cache=rng.choice(("bf16", "int8", "int8")), ragged=rng.random() < 0.7)
        c["tokens"] = min(c["tokens"], c["context"])
        while c["batch"] * c["context"] * kv > 4 * 16384 * 8:
            c["batch"] //= 2
        return c
    if op == "norm":
        dtype = rng.choice(("bf16", "bf16", "fp32"))
        rows, cols = _log_int(rng, 1, 8192), _log_int(rng, 256, 8192)
        return dict(op=op, rows=min(rows, 8192 * 4096 // cols), cols=cols, dtype=dtype, residual=rng.random() < 0.6,
                    out=rng.choice(("int8", "int8", "same")))
    group = rng.choice((32, 64, 128))
    return dict(op="linear", rows=_log_int(rng, 1, 32), n=_log_int(rng, 500, 16384),
                k=256 * _log_int(rng, 2, 32) + 128, group=group, x=rng.choice(("int8", "bf16")), zeros=rng.random() < 0.5,
                bias=rng.random() < 0.5, silu=rng.random() < 0.5, out=rng.choice(("bf16", "bf16", "fp32")))


def _lengths(c):
    """Each sequence's length, and how many of its last tokens are new."""
    b = c["batch"]
    if not c["ragged"]:
        return [c["context"]] * b, [c["tokens"]] * b
    lens = [max(1, c["context"] - (i * 977) % (c["context"] // 2 + 1)) for i in range(b)]
    new = [min(n, max(1, c["tokens"] - (i * 37) % (c["tokens"] // 2 + 1))) for i, n in enumerate(lens)]
    if b >= 4 and c["tokens"] > 1:
        new[-1] = 0  # a sequence of the batch that has nothing new in this call
    return lens, new


# ------------------------------------------------------------------ the inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows_of_8_bits(shape, g):
    """Codes and scales of rows quantised from normal values, largest value at 127."""
    codes = (torch.randn(shape, device="cuda", generator=g, dtype=torch.bfloat16) * 36).clamp_(-127, 127).to(torch.int8)
    scales = torch.rand(shape[:-1], device="cuda", generator=g) * 0.02 + 0.015
    return codes, scales


def _pages(c, g, s):
    """A pool of pages in an order of its own, the sequences' page table and lengths."""
    lens, new = _lengths(c)
    kv, d, page = c["kv_heads"], c["head_dim"], c["page"]
    count = [-(-n // page) for n in lens]
    pool = sum(count) + 3
    order = torch.randperm(pool, device="cuda", generator=g).to(torch.int32)
    table = torch.full((c["batch"], max(count)), -1, dtype=torch.int32, device="cuda")
    first = torch.tensor([sum(count[:i]) for i in range(c["batch"])], device="cuda")
    slot = torch.arange(max(count), device="cuda")
    used = slot[None] < torch.tensor(count, device="cuda")[:, None]
    table[used] = order[(first[:, None] + slot[None])[used]]
    s["table"] = table
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    starts = [sum(new[:i]) for i in range(c["batch"] + 1)]
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["total"], s["max_len"], s["max_new"] = starts[-1], max(lens), max(new)
    s["seq_of"] = torch.repeat_interleave(torch.arange(c["batch"], device="cuda"), torch.tensor(new, device="cuda"))
    s["index"] = torch.arange(starts[-1], device="cuda") - s["starts"].long()[s["seq_of"]]
    shape = (pool, kv, page, d)
    if c["cache"] == "int8":
        s["k"], s["k_scale"] = _rows_of_8_bits(shape, g)
        s["v"], s["v_scale"] = _rows_of_8_bits(shape, g)
    else:
        s["k"] = torch.randn(shape, device="cuda", generator=g, dtype=torch.bfloat16)
        s["v"] = torch.randn(shape, device="cuda", generator=g, dtype=torch.bfloat16)
        s["k_scale"] = s["v_scale"] = None


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": case}
    c = case
    if c["op"] == "attention":
        _pages(c, g, s)
        s["q"] = torch.randn((s["total"], c["heads"], c["head_dim"]), device="cuda", generator=g, dtype=torch.bfloat16)
    elif c["op"] == "cache":
        _pages(c, g, s)
        # keys and values as the last two thirds of a fused product's rows
        rows = torch.randn((s["total"], 3, c["kv_heads"], c["head_dim"]), device="cuda", generator=g, dtype=torch.bfloat16)
        s["k_new"], s["v_new"] = rows[:, 1], rows[:, 2]
    elif c["op"] == "norm":
        t = _TYPES[c["dtype"]]
        s["x"] = torch.randn((c["rows"], c["cols"]), device="cuda", generator=g).to(t)
        s["residual"] = torch.randn((c["rows"], c["cols"]), device="cuda", generator=g).mul_(4).to(t) if c["residual"] else None
        s["weight"] = torch.rand(c["cols"], device="cuda", generator=g) + 0.5
        s["eps"] = 1e-5
    else:
        n, k, group = c["n"], c["k"], c["group"]
        codes = (torch.randn((n, k), device="cuda", generator=g) * 2.5 + 8).round_().clamp_(0, 15).to(torch.uint8)
        by_nibble = codes.view(n, k // 8, 8)[:, :, [0, 2, 4, 6, 1, 3, 5, 7]]
        s["packed"] = (by_nibble[..., 0::2] | (by_nibble[..., 1::2] << 4)).reshape(n, k // 2).contiguous()
        s["scales"] = (torch.rand((k // group, n), device="cuda", generator=g) * 0.01 + 0.004).to(torch.bfloat16)
        s["zeros"] = torch.randint(5, 12, (k // group, n), device="cuda", generator=g, dtype=torch.uint8) if c["zeros"] else None
        s["bias"] = torch.randn(n, device="cuda", generator=g) if c["bias"] else None
        if c["x"] == "int8":
            s["x"], s["x_scale"] = _rows_of_8_bits((c["rows"], k), g)
        else:
            s["x"], s["x_scale"] = torch.randn((c["rows"], k), device="cuda", generator=g).to(torch.bfloat16), None
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program keeps between calls: the cache, the attention's plan and workspace, the packed layer."""
    from conv_bn_silu_gb300 import _binding as B
    from conv_bn_silu_gb300 import tokens
    c = s["case"]
    if c["op"] in ("attention", "cache"):
        s["cache"] = tokens.PagedCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    if c["op"] == "attention":
        s["attention"] = tokens.PagedAttention(s["cache"], batch=c["batch"], max_new=s["max_new"], max_len=s["max_len"],
                                               heads=c["heads"], causal=c["causal"], window=c["window"])
    if c["op"] == "linear":
        s["layer"] = tokens.LinearW4(s["packed"], s["scales"], c["group"], zeros=s["zeros"], bias=s["bias"],
                                     activation=B.CBS_ACT_SILU if c["silu"] else B.CBS_ACT_IDENTITY)


# ------------------------------------------------------------- the plain forms
def _values(pool, scale, table, length):
    """A paged pool's rows in the sequences' order, in float: [batch, kv_heads, length, head_dim]."""
    at = table.clamp(min=0).long()
    x = pool[at].float()
    if scale is not None:
        x = x * scale[at][..., None]
    b, p, kv, page, d = x.shape
    return x.transpose(1, 2).reshape(b, kv, p * page, d)[:, :, :length]


def _plain_attention(s):
    c = s["case"]
    b, h, kv, d, t, n = c["batch"], c["heads"], c["kv_heads"], c["head_dim"], s["max_new"], s["max_len"]
    key = torch.arange(n, device="cuda")
    lens = s["lens"].long()
    held = (key[None] < lens[:, None])[:, None, :, None]
    k = _values(s["k"], s["k_scale"], s["table"], n).masked_fill(~held, 0.0)
    v = _values(s["v"], s["v_scale"], s["table"], n).masked_fill(~held, 0.0)
    q = torch.zeros((b, t, h, d), device="cuda")
    q[s["seq_of"], s["index"]] = s["q"].float()
    q = q.view(b, t, kv, h // kv, d).permute(0, 2, 3, 1, 4).reshape(b, kv, h // kv * t, d)
    scores = (q @ k.transpose(-1, -2)).view(b, kv, h // kv, t, n).mul_(1.0 / math.sqrt(d))
    new = (s["starts"][1:] - s["starts"][:-1]).long()
    place = (lens - new)[:, None] + torch.arange(t, device="cuda")[None]
    seen = (key[None] < lens[:, None])[:, None, :].expand(b, t, n)
    if c["causal"]:
        seen = seen & (key[None, None] <= place[:, :, None])
    if c["window"]:
        seen = seen & (key[None, None] > place[:, :, None] - c["window"])
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(b, kv, h // kv * t, n) @ v).view(b, kv, h // kv, t, d)
    out = (out / total.masked_fill(total == 0.0, 1.0)).permute(0, 3, 1, 2, 4).reshape(b, t, h, d)
    return out[s["seq_of"], s["index"]].to(torch.bfloat16)


def _to_8_bits(x):
    """Rows in 8 bits: scale = max|x| / 127, code = the nearest whole number to x / scale."""
    scale = x.abs().amax(-1) / 127.0
    return (x / scale.masked_fill(scale == 0.0, 1.0)[..., None]).round().clamp(-127, 127), scale


def _plain_cache(s):
    c = s["case"]
    new = s["starts"][1:] - s["starts"][:-1]
    place = (s["lens"] - new).long()[s["seq_of"]] + s["index"]
    page, slot = s["table"][s["seq_of"], place // c["page"]].long(), place % c["page"]
    if c["cache"] == "int8":
        codes, scale = _to_8_bits(s["k_new"].float())
        s["k"][page, :, slot], s["k_scale"][page, :, slot] = codes.to(torch.int8), scale
        codes, scale = _to_8_bits(s["v_new"].float())
        s["v"][page, :, slot], s["v_scale"][page, :, slot] = codes.to(torch.int8), scale
    else:
        s["k"][page, :, slot], s["v"][page, :, slot] = s["k_new"], s["v_new"]
    held = (torch.arange(s["max_len"], device="cuda")[None] < s["lens"][:, None])[:, None, :, None]
    k = _values(s["k"], s["k_scale"], s["table"], s["max_len"]).masked_fill(~held, 0.0)
    v = _values(s["v"], s["v_scale"], s["table"], s["max_len"]).masked_fill(~held, 0.0)
    return {"k": k.transpose(1, 2).to(torch.bfloat16).contiguous(), "v": v.transpose(1, 2).to(torch.bfloat16).contiguous()}


def _plain_norm(s):
    c = s["case"]
    t = _TYPES[c["dtype"]]
    h = s["x"].float()
    if c["residual"]:
        h = h + s["residual"].float()
    r = 1.0 / torch.sqrt(h.square().mean(-1) + s["eps"])
    u = h * s["weight"]
    out = {"h": h.to(t)} if c["residual"] else {}
    if c["out"] == "int8":
        codes, scale = _to_8_bits(u)
        out["y"] = (codes * (scale * r)[:, None]).to(torch.bfloat16)
        out["scale"] = scale * r
    else:
        out["y"] = (u * r[:, None]).to(t)
    return out


def _plain_linear(s):
    c = s["case"]
    n, k, group = c["n"], c["k"], c["group"]
    w = torch.stack((s["packed"] & 15, s["packed"] >> 4), -1).view(n, k // 8, 8)[:, :, list(_NIBBLE)]
    w = w.reshape(n, k // group, group).float()
    w = w - (s["zeros"].t()[..., None].float() if c["zeros"] else 8.0)
    w = (w * s["scales"].t()[..., None].float()).view(n, k)
    x = s["x"].float()
    y = x @ w.t()
    if s["x_scale"] is not None:
        y = y * s["x_scale"][:, None]
    if c["bias"]:
        y = y + s["bias"]
    if c["silu"]:
        y = y / (1.0 + torch.exp(-y))
    return y.to(_TYPES[c["out"]])


def run(s):
    c = s["case"]
    if not own:
        return {"attention": _plain_attention, "cache": _plain_cache, "norm": _plain_norm, "linear": _plain_linear}[c["op"]](s)
    from conv_bn_silu_gb300 import tokens
    if c["op"] == "attention":
        return s["attention"](s["q"], s["starts"], s["lens"], s["table"])
    if c["op"] == "cache":
        s["cache"].write(s["k_new"], s["v_new"], s["starts"], s["lens"], s["table"])
        k, v = s["cache"].read(s["lens"], s["table"], s["max_len"])
        return {"k": k, "v": v}
    if c["op"] == "norm":
        r = tokens.rmsnorm(s["x"], s["weight"], s["eps"], residual=s["residual"], int8=c["out"] == "int8")
        out = {"h": r.h} if c["residual"] else {}
        if c["out"] == "int8":
            out["y"], out["scale"] = tokens.dequantize_rows(r.y, r.scale), r.scale
        else:
            out["y"] = r.y
        return out
    return s["layer"](s["x"], s["x_scale"], dtype=_TYPES[c["out"]])


# ------------------------------------------------------------- bytes and flops
def work(case):
    c = case
    if c["op"] in ("attention", "cache"):
        lens, new = _lengths(c)
        row = c["head_dim"] * (2 if c["cache"] == "bf16" else 1) + (4 if c["cache"] == "int8" else 0)
    if c["op"] == "attention":
        keys = scores = 0
        for n, t in zip(lens, new):
            lo, hi = n - t + 1, n  # the keys up to the first and up to the last new token
            if not t:
                continue
            if not c["causal"]:
                keys, scores = keys + n, scores + n * t
                continue
            w = c["window"] or n
            full = max(0, min(t, hi - max(lo, w) + 1))  # new tokens that see a whole window
            part = t - full
            scores += full * w + (lo + lo + part - 1) * part // 2
            keys += n - max(0, lo - w)
        io = 2 * sum(new) * c["heads"] * c["head_dim"] * 2
        return {"bytes": 2 * keys * c["kv_heads"] * row + io, "flops": 4 * scores * c["heads"] * c["head_dim"]}
    if c["op"] == "cache":
        written = 2 * sum(new) * c["kv_heads"]
        read = 2 * sum(lens) * c["kv_heads"]
        out = 2 * c["batch"] * max(lens) * c["kv_heads"] * c["head_dim"] * 2
        flops = (4 * written + read) * c["head_dim"] if c["cache"] == "int8" else 0
        return {"bytes": written * (c["head_dim"] * 2 + row) + read * row + out, "flops": flops}
    if c["op"] == "norm":
        e, count = (2 if c["dtype"] == "bf16" else 4), c["rows"] * c["cols"]
        moved = count * e * (3 if c["residual"] else 1) + c["cols"] * 4
        # in 8 bits: the codes written, and read again to give the values they stand for
        moved += count * 4 + c["rows"] * 8 if c["out"] == "int8" else count * e
        return {"bytes": moved, "flops": count * 8}
    n, k, m = c["n"], c["k"], c["rows"]
    weights = n * k // 2 + n * (k // c["group"]) * (3 if c["zeros"] else 2)
    x = m * (k + 4) if c["x"] == "int8" else m * k * 2
    return {"bytes": weights + x + m * n * (2 if c["out"] == "bf16" else 4) + (4 * n if c["bias"] else 0), "flops": 2 * m * n * k}


# ------------------------------------------------------- definitions in 64 bits
def _history(s, i, pool, scale):
    """Sequence i's rows of a pool, in 64 bits: [length, kv_heads, head_dim]."""
    n, page = int(s["lens"][i]), s["case"]["page"]
    pages = s["table"][i, : -(-n // page)].long()
    x = pool[pages].double()
    if scale is not None:
        x *= scale[pages].double().unsqueeze(-1)
    return x.permute(0, 2, 1, 3).flatten(0, 1)[:n]


def _exact_attention(s):
    c = s["case"]
    group = c["heads"] // c["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for i in range(c["batch"]):
        a, b = int(s["starts"][i]), int(s["starts"][i + 1])
        if a == b:
            continue
        keys, values = _history(s, i, s["k"], s["k_scale"]), _history(s, i, s["v"], s["v_scale"])
        n = keys.shape[0]
        place = torch.arange(n - (b - a), n, device="cuda").unsqueeze(1)
        key = torch.arange(n, device="cuda").unsqueeze(0)
        hidden = torch.zeros((b - a, n), dtype=torch.bool, device="cuda")
        if c["causal"]:
            hidden |= key > place
        if c["window"]:
            hidden |= key <= place - c["window"]
        empty = hidden.all(1)
        for h in range(c["heads"]):
            x = torch.mm(s["q"][a:b, h].double(), keys[:, h // group].t()) / c["head_dim"] ** 0.5
            x[hidden] = -math.inf
            x[empty] = 0.0
            y = torch.mm(torch.softmax(x, 1), values[:, h // group])
            y[empty] = 0.0
            out[a:b, h] = y
    return out


def _nearest_codes(x):
    step = x.abs().max(dim=-1).values / 127
    return torch.round(x / torch.where(step > 0, step, torch.ones_like(step)).unsqueeze(-1)), step


def _exact_cache(s):
    c = s["case"]
    out = {}
    for side in ("k", "v"):
        new = s[side + "_new"].double()
        if c["cache"] == "int8":
            codes, step = _nearest_codes(new)
            new = codes * step.unsqueeze(-1)
        whole = torch.zeros((c["batch"], s["max_len"], c["kv_heads"], c["head_dim"]), dtype=torch.float64, device="cuda")
        for i in range(c["batch"]):
            n, a, b = int(s["lens"][i]), int(s["starts"][i]), int(s["starts"][i + 1])
            whole[i, :n] = _history(s, i, s[side], s[side + "_scale"])
            whole[i, n - (b - a):n] = new[a:b]
        out[side] = whole
    return out


def _exact_norm(s):
    c = s["case"]
    h = s["x"].double() + (s["residual"].double() if c["residual"] else 0.0)
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + s["eps"]) * s["weight"].double()
    out = {"h": h} if c["residual"] else {}
    if c["out"] == "int8":
        codes, step = _nearest_codes(y)
        out["y"], out["scale"] = codes * step.unsqueeze(1), step
    else:
        out["y"] = y
    return out


def _exact_linear(s):
    c = s["case"]
    n, k, group = c["n"], c["k"], c["group"]
    w = torch.empty((n, k), dtype=torch.float64, device="cuda")
    for j in range(8):  # weight 8 i + j is one nibble of its word's four bytes
        byte = s["packed"].view(n, k // 8, 4)[:, :, _NIBBLE[j] // 2]
        w[:, j::8] = (byte >> 4 if _NIBBLE[j] % 2 else byte & 15).double()
    for i in range(k // group):
        block = w[:, i * group:(i + 1) * group]
        block -= s["zeros"][i].double().unsqueeze(1) if c["zeros"] else 8
        block *= s["scales"][i].double().unsqueeze(1)
    x = s["x"].double()
    if s["x_scale"] is not None:
        x = x * s["x_scale"].double().unsqueeze(1)
    y = torch.mm(x, w.t())
    if c["bias"]:
        y += s["bias"].double()
    return y * torch.sigmoid(y) if c["silu"] else y


def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _exact_attention, "cache": _exact_cache, "norm": _exact_norm, "linear": _exact_linear}[case["op"]](s)
