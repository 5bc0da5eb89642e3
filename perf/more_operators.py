"""Cases and plain forms of the token operators for many and long answers over
a few images: attention of sequences that share a prefix, attention that also
weighs the cache's positions, eviction of positions by that weight, and products
with 8-bit weights for prompts as for single tokens.

`own` chooses between the plain forms (elementary torch operations in 32 bits)
and the package's kernels.  `exact` gives each operator's definition in 64 bits.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases
def _shared(name, groups, each, tokens, prefix, context, heads, kv_heads, head_dim, page, cache, ragged=True):
    return dict(name=name, op="shared", groups=groups, each=each, tokens=tokens, prefix=prefix, context=context,
                heads=heads, kv_heads=kv_heads, head_dim=head_dim, page=page, cache=cache, ragged=ragged)


def _weighed(name, batch, tokens, context, heads, kv_heads, head_dim, page, cache, causal=True, window=0, decay=1.0,
             ragged=False):
    return dict(name=name, op="weighed", batch=batch, tokens=tokens, context=context, heads=heads, kv_heads=kv_heads,
                head_dim=head_dim, page=page, cache=cache, causal=causal, window=window, decay=decay, ragged=ragged)


def _evict(name, batch, context, keep, recent, kv_heads, head_dim, page, cache, ragged=False):
    return dict(name=name, op="evict", batch=batch, context=context, keep=keep, recent=recent, kv_heads=kv_heads,
                head_dim=head_dim, page=page, cache=cache, ragged=ragged)


def _linear(name, rows, n, k, bias, silu, out):
    return dict(name=name, op="linear", rows=rows, n=n, k=k, bias=bias, silu=silu, out=out)


def listed():
    return [
        # Six answers about one image, a token further each: its 20x20 cells are their prefix.  Latency alone.
        _shared("shared 6 answers on a map", 1, 6, 1, 400, 30, 8, 2, 64, 16, "int8"),
        # A server whose 64 streams begin with the same long instructions.
        _shared("shared 64 streams", 1, 64, 1, 8192, 1000, 32, 8, 128, 64, "bf16"),
        # Odd groups of questions on five documents, the questions' tokens in one call.
        _shared("shared odd questions int8", 5, 7, 40, 3001, 150, 24, 4, 64, 32, "int8"),
        # One stream's token over a short history, weights of this step alone.  Latency.
        _weighed("weighed 1 token", 1, 1, 1000, 32, 8, 128, 16, "bf16", decay=0.0),
        # 32 streams, each a token further, the weights summed up over the steps.
        _weighed("weighed 32 streams int8", 32, 1, 8192, 32, 8, 128, 64, "int8", ragged=True),
        # A chunk of a long prompt, after which the cache is to be thinned out.
        _weighed("weighed chunk of 1024", 1, 1024, 16384, 32, 8, 128, 64, "bf16"),
        # A short history to three fifths.  Latency.
        _evict("evict 1 stream", 1, 1000, 600, 64, 8, 128, 16, "bf16"),
        # Long histories of differing length to half.
        _evict("evict 16 streams int8", 16, 8192, 4096, 512, 8, 128, 64, "int8", ragged=True),
        # A long prompt of odd length to a small odd rest: the choice is most of the work.
        _evict("evict long prompt", 1, 65001, 4001, 100, 4, 64, 32, "bf16"),
        # One token through a layer's fused query/key/value product.
        _linear("linear 1 token", 1, 6144, 4096, False, False, "bf16"),
        # The 20x20 cells of one image through an odd output width, with bias and SiLU.
        _linear("linear 400 cells odd", 400, 1001, 2064, True, True, "fp32"),
        # A long prompt through a square layer.
        _linear("linear prompt", 8192, 8192, 8192, False, False, "bf16"),
    ]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm (round ones are the listed cases')."""
    n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n - 1 if n % 1024 == 0 else n


def draw(rng):
    op = rng.choice(("shared", "weighed", "evict", "linear"))
    kv = rng.choice((1, 2, 4, 8))
    common = dict(kv_heads=kv, head_dim=rng.choice((64, 128)), page=rng.choice((16, 32, 64)), cache=rng.choice(("bf16", "int8")),
                  ragged=rng.random() < 0.7)
    if op == "shared":
        c = dict(op=op, groups=_log_int(rng, 1, 8), each=_log_int(rng, 1, 64), tokens=1 if rng.random() < 0.5 else _log_int(rng, 2, 300),
                 prefix=_log_int(rng, 16, 16384), context=_log_int(rng, 1, 2000), heads=kv * rng.choice((1, 2, 3, 4, 6, 8)), **common)
        # no more scores than 2^30, and no more histories than the largest listed case's
        while c["groups"] * c["each"] > 64 or c["groups"] * c["each"] * (c["prefix"] + c["context"]) * kv > 64 * 9192 * 8:
            c["each" if c["each"] > 1 else "groups"] = max(1, c["each" if c["each"] > 1 else "groups"] // 2)
        c["context"] = max(c["context"], c["tokens"])
        while c["groups"] * c["each"] * c["tokens"] * c["heads"] * (c["prefix"] + c["context"]) > 1 << 28:
            c["tokens"] = max(1, c["tokens"] // 2)
            c["prefix"] = max(16, c["prefix"] * 3 // 4)
        return c
    if op == "weighed":
        c = dict(op=op, batch=_log_int(rng, 1, 32), tokens=1 if rng.random() < 0.5 else _log_int(rng, 2, 1024),
                 context=_log_int(rng, 16, 16384), heads=kv * rng.choice((1, 2, 3, 4, 6, 8)), causal=rng.random() < 0.8, window=0,
                 decay=rng.choice((0.0, 1.0, 0.75)), **common)
        c["tokens"] = min(c["tokens"], c["context"])
        if c["causal"] and rng.random() < 0.2:
            c["window"] = _log_int(rng, 64, 4096)
        while c["batch"] * c["heads"] * c["tokens"] * c["context"] > 32 * 1024 * 16000 or c["batch"] * c["context"] * kv > 32 * 8192 * 8:
            c["batch" if c["batch"] > 1 else "tokens"] = (c["batch"] if c["batch"] > 1 else c["tokens"]) // 2
        return c
    if op == "evict":
        c = dict(op=op, batch=_log_int(rng, 1, 32), context=_log_int(rng, 64, 100000), **common)
        c["keep"] = max(16, int(c["context"] * rng.uniform(0.05, 0.9)))
        c["recent"] = int(c["keep"] * rng.uniform(0.0, 0.5))
        while c["batch"] * c["context"] * kv > 16 * 8192 * 8:
            c["batch"] = max(1, c["batch"] // 2)
            if c["batch"] == 1:
                break
        return c
    c = dict(op=op, rows=1 if rng.random() < 0.3 else _log_int(rng, 2, 8192), n=_log_int(rng, 200, 16384), k=16 * _log_int(rng, 16, 512),
             bias=rng.random() < 0.5, silu=rng.random() < 0.5, out=rng.choice(("bf16", "bf16", "fp32")))
    while c["rows"] * c["n"] * c["k"] > 8192 ** 3:
        c["rows"] //= 2
    return c


def _new(tokens, lens, ragged):
    """How many of each sequence's last tokens are new."""
    if not ragged:
        return [min(n, tokens) for n in lens]
    new = [min(n, max(1, tokens - (i * 37) % (tokens // 2 + 1))) for i, n in enumerate(lens)]
    if len(lens) >= 4 and tokens > 1:
        new[-1] = 0  # a sequence of the batch that has nothing new in this call
    return new


def _lengths(c):
    """Each sequence's (own) length and new tokens; for a shared prefix also the groups' sizes and prefixes."""
    if c["op"] == "shared":
        sizes = [max(1, c["each"] - (2 * i) % c["each"]) if c["ragged"] else c["each"] for i in range(c["groups"])]
        prefixes = [max(1, c["prefix"] - (i * 577) % (c["prefix"] // 2 + 1)) if c["ragged"] else c["prefix"] for i in range(c["groups"])]
        b = sum(sizes)
    else:
        sizes = prefixes = None
        b = c["batch"]
    step = max(1, 977 * c["context"] // 8192)
    lens = [max(1, c["context"] - (i * step) % (c["context"] // 2 + 1)) if c["ragged"] else c["context"] for i in range(b)]
    new = _new(c["tokens"], lens, c["ragged"]) if "tokens" in c else None
    return lens, new, sizes, prefixes


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


def _tables(lists, page, g):
    """Page tables over one pool, for lists of lengths, the pages in an order of their own; and the pool's size."""
    counts = [[-(-n // page) for n in lens] for lens in lists]
    pool = sum(map(sum, counts)) + 3
    order = torch.randperm(pool, device="cuda", generator=g).to(torch.int32)
    tables, used = [], 0
    for count in counts:
        first = torch.tensor([used + sum(count[:i]) for i in range(len(count))], device="cuda")
        slot = torch.arange(max(count), device="cuda")
        held = slot[None] < torch.tensor(count, device="cuda")[:, None]
        table = torch.full((len(count), max(count)), -1, dtype=torch.int32, device="cuda")
        table[held] = order[(first[:, None] + slot[None])[held]]
        tables.append(table)
        used += sum(count)
    return tables, pool


def _pool(c, pool, g, s):
    shape = (pool, c["kv_heads"], c["page"], c["head_dim"])
    if c["cache"] == "int8":
        s["k"], s["k_scale"] = _rows_of_8_bits(shape, g)
        s["v"], s["v_scale"] = _rows_of_8_bits(shape, g)
    else:
        s["k"] = torch.randn(shape, device="cuda", generator=g, dtype=torch.bfloat16)
        s["v"] = torch.randn(shape, device="cuda", generator=g, dtype=torch.bfloat16)
        s["k_scale"] = s["v_scale"] = None


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g, c = _generator(seed), case
    s = {"case": case}
    if c["op"] == "linear":
        s["x"], s["x_scale"] = _rows_of_8_bits((c["rows"], c["k"]), g)
        s["w"], s["w_scale"] = _rows_of_8_bits((c["n"], c["k"]), g)
        s["w_scale"] /= math.sqrt(c["k"])
        s["bias"] = torch.randn(c["n"], device="cuda", generator=g) if c["bias"] else None
    else:
        lens, new, sizes, prefixes = _lengths(c)
        s["lens"], s["max_len"] = _int32(lens), max(lens)
        if c["op"] == "shared":
            (s["table"], s["prefix_table"]), pool = _tables([lens, prefixes], c["page"], g)
            s["prefix_lens"], s["max_prefix"] = _int32(prefixes), max(prefixes)
            first = [sum(sizes[:i]) for i in range(len(sizes) + 1)]
            s["group_start"] = _int32(first)
            s["group_of"] = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), torch.tensor(sizes, device="cuda"))
            s["max_group_new"] = max(sum(new[a:b]) for a, b in zip(first, first[1:]))
        elif c["op"] == "weighed":
            (s["table"],), pool = _tables([lens], c["page"], g)
            # what earlier steps left: sums of softmax weights, of the size of this call's own
            s["mass_before"] = torch.rand((pool, c["kv_heads"], c["page"]), device="cuda", generator=g)
            s["mass_before"] *= 2 * max(new) * (c["heads"] // c["kv_heads"]) / max(lens)
            s["mass"] = s["mass_before"].clone()
        else:
            (s["table"], s["new_table"]), pool = _tables([lens, [min(n, c["keep"]) for n in lens]], c["page"], g)
            # a few positions hold most of the weight, and many hold the same
            mass = torch.randn((pool, c["kv_heads"], c["page"]), device="cuda", generator=g)
            s["mass"] = (mass * 2 - 4).exp_().to(torch.bfloat16).float()
        _pool(c, pool, g, s)
        if new is not None:
            starts = [sum(new[:i]) for i in range(len(lens) + 1)]
            s["starts"], s["max_new"] = _int32(starts), max(new)
            s["seq_of"] = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), torch.tensor(new, device="cuda"))
            s["index"] = torch.arange(starts[-1], device="cuda") - s["starts"].long()[s["seq_of"]]
            s["q"] = torch.randn((starts[-1], c["heads"], c["head_dim"]), device="cuda", generator=g, dtype=torch.bfloat16)
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program keeps between calls: the cache, the attention's plan and workspace, the layer."""
    from conv_bn_silu_gb300 import _binding as B
    from conv_bn_silu_gb300 import tokens
    c = s["case"]
    if c["op"] == "linear":
        s["layer"] = tokens.LinearW8(s["w"], s["w_scale"], bias=s["bias"],
                                     activation=B.CBS_ACT_SILU if c["silu"] else B.CBS_ACT_IDENTITY)
        return
    s["cache"] = tokens.PagedCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    if c["op"] == "shared":
        s["attention"] = tokens.SharedPrefixAttention(
            s["cache"], batch=s["lens"].shape[0], groups=c["groups"], max_new=s["max_new"], max_group_new=s["max_group_new"],
            max_len=s["max_len"], max_prefix=s["max_prefix"], heads=c["heads"])
    elif c["op"] == "weighed":
        s["attention"] = tokens.WeighedAttention(s["cache"], batch=c["batch"], max_new=s["max_new"], max_len=s["max_len"],
                                                 heads=c["heads"], causal=c["causal"], window=c["window"])


# ------------------------------------------------------------- the plain forms
def _values(pool, scale, table, length):
    """A paged pool's rows in the sequences' order, in float: [batch, kv_heads, length, head_dim]."""
    at = table.clamp(min=0).long()
    x = pool[at].float()
    if scale is not None:
        x = x * scale[at][..., None]
    b, p, kv, page, d = x.shape
    return x.transpose(1, 2).reshape(b, kv, p * page, d)[:, :, :length]


def _side(s, side):
    """Every sequence's keys or values in order; zeros past its length.  With a shared prefix, that first."""
    own_held = torch.arange(s["max_len"], device="cuda")[None] < s["lens"][:, None]
    x = _values(s[side], s[side + "_scale"], s["table"], s["max_len"]).masked_fill(~own_held[:, None, :, None], 0.0)
    if s["case"]["op"] != "shared":
        return x
    held = torch.arange(s["max_prefix"], device="cuda")[None] < s["prefix_lens"][:, None]
    p = _values(s[side], s[side + "_scale"], s["prefix_table"], s["max_prefix"]).masked_fill(~held[:, None, :, None], 0.0)
    return torch.cat([p[s["group_of"]], x], 2)


def _seen(s):
    """Which keys each new token sees: [batch, new tokens, keys]."""
    c, t = s["case"], s["max_new"]
    lens, key = s["lens"].long(), torch.arange(s["max_len"], device="cuda")
    new = (s["starts"][1:] - s["starts"][:-1]).long()
    place = (lens - new)[:, None] + torch.arange(t, device="cuda")[None]
    seen = (key[None] < lens[:, None])[:, None, :].expand(-1, t, -1)
    if c.get("causal", True):
        seen = seen & (key[None, None] <= place[:, :, None])
    if c.get("window", 0):
        seen = seen & (key[None, None] > place[:, :, None] - c["window"])
    if c["op"] == "shared":
        before = torch.arange(s["max_prefix"], device="cuda")[None] < s["prefix_lens"][s["group_of"]][:, None]
        seen = torch.cat([before[:, None].expand(-1, t, -1), seen], 2)
    return seen


def _plain_softmax(s, k):
    """The new tokens' weights of the keys: [batch, kv_heads, heads of each, new tokens, keys]."""
    c = s["case"]
    b, t, h, kv, d = s["lens"].shape[0], s["max_new"], c["heads"], c["kv_heads"], c["head_dim"]
    q = torch.zeros((b, t, h, d), device="cuda")
    q[s["seq_of"], s["index"]] = s["q"].float()
    q = q.view(b, t, kv, h // kv, d).permute(0, 2, 3, 1, 4).reshape(b, kv, h // kv * t, d)
    scores = (q @ k.transpose(-1, -2)).view(b, kv, h // kv, t, -1).mul_(1.0 / math.sqrt(d))
    scores.masked_fill_(~_seen(s)[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    return p.div_(total.masked_fill(total == 0.0, 1.0))


def _plain_out(s, p, v):
    b, kv, g, t, n = p.shape
    out = (p.view(b, kv, g * t, n) @ v).view(b, kv, g, t, -1).permute(0, 3, 1, 2, 4).reshape(b, t, kv * g, -1)
    return out[s["seq_of"], s["index"]].to(torch.bfloat16)


def _plain_shared(s):
    return _plain_out(s, _plain_softmax(s, _side(s, "k")), _side(s, "v"))


def _plain_weighed(s):
    c = s["case"]
    mass = s["mass"].copy_(s["mass_before"]) if c["decay"] else s["mass"]
    p = _plain_softmax(s, _side(s, "k"))
    lens, new = s["lens"].long(), (s["starts"][1:] - s["starts"][:-1]).long()
    fresh = torch.arange(s["max_new"], device="cuda")[None] < new[:, None]
    received = (p * fresh[:, None, None, :, None]).sum((2, 3))
    key = torch.arange(s["max_len"], device="cuda")
    page, slot = s["table"][:, key // c["page"]].clamp(min=0).long(), key % c["page"]
    heads = torch.arange(c["kv_heads"], device="cuda")[None, :, None]
    before = mass[page[:, None], heads, slot] * c["decay"] if c["decay"] else torch.zeros_like(received)
    after = before.masked_fill((key[None] >= (lens - new)[:, None])[:, None], 0.0) + received
    at = ((key[None] < lens[:, None]) & (new > 0)[:, None])[:, None].expand_as(after)
    mass[page[:, None].expand_as(after)[at], heads.expand_as(after)[at], slot.expand_as(after)[at]] = after[at]
    return {"out": _plain_out(s, p, _side(s, "v")), "mass": mass}


def _plain_evict(s):
    c, lens, n = s["case"], s["lens"].long(), s["max_len"]
    b, kv, keep, page = lens.shape[0], c["kv_heads"], c["keep"], c["page"]
    key, heads = torch.arange(n, device="cuda"), torch.arange(kv, device="cuda")[None, :, None]
    at = s["table"][:, key // page].clamp(min=0).long()[:, None]
    mass = s["mass"][at, heads, key % page]
    mass = mass.masked_fill((key[None] >= lens[:, None] - c["recent"])[:, None], math.inf)
    mass = mass.masked_fill((key[None] >= lens[:, None])[:, None], -math.inf)
    order = mass.sort(dim=-1, descending=True, stable=True).indices[:, :, :keep]
    after = lens.clamp(max=keep)
    slot = torch.arange(order.shape[2], device="cuda")
    held = (slot[None] < after[:, None])[:, None].expand_as(order)
    kept = order.masked_fill(~held, n).sort(-1).values
    src, to = kept.clamp(max=n - 1), s["new_table"][:, slot // page].clamp(min=0).long()[:, None].expand_as(kept)[held]
    h = heads.expand_as(kept)
    from_page = s["table"].clamp(min=0).long()[torch.arange(b, device="cuda")[:, None, None], src // page]
    row, new_row = (from_page[held], h[held], (src % page)[held]), (to, h[held], (slot % page).expand_as(kept)[held])
    for x in (s["k"], s["v"], s["mass"], s["k_scale"], s["v_scale"]):
        if x is not None:
            x[new_row] = x[row]
    out = torch.full((b, kv, keep), -1, dtype=torch.int32, device="cuda")
    out[:, :, :kept.shape[2]] = kept.masked_fill(~held, -1)
    return _evicted(s, out, after.to(torch.int32), _values)


def _evicted(s, kept, lens, values):
    """What an eviction leaves; 8-bit pages as the values that they stand for, in order."""
    out = {"kept": kept, "lens": lens, "mass": s["mass"], "k": s["k"], "v": s["v"]}
    if s["case"]["cache"] == "int8":
        n = min(s["case"]["keep"], s["max_len"])
        held = (torch.arange(n, device="cuda")[None] < lens[:, None])[:, None, :, None]
        for side in ("k", "v"):
            x = values(s[side], s[side + "_scale"], s["new_table"], n).masked_fill(~held, 0.0)
            out[side] = x.transpose(1, 2).to(torch.bfloat16).contiguous()
    return out


def _plain_linear(s):
    c = s["case"]
    y = (s["x"].float() @ s["w"].float().t()) * s["x_scale"][:, None] * s["w_scale"]
    if c["bias"]:
        y = y + s["bias"]
    if c["silu"]:
        y = y / (1.0 + torch.exp(-y))
    return y.to(_TYPES[c["out"]])


def run(s):
    c = s["case"]
    if not own:
        return {"shared": _plain_shared, "weighed": _plain_weighed, "evict": _plain_evict, "linear": _plain_linear}[c["op"]](s)
    if c["op"] == "shared":
        return s["attention"](s["q"], s["starts"], s["lens"], s["table"], s["group_start"], s["prefix_lens"], s["prefix_table"])
    if c["op"] == "weighed":
        if c["decay"]:
            s["mass"].copy_(s["mass_before"])  # (so that every pass adds to the same)
        return {"out": s["attention"](s["q"], s["starts"], s["lens"], s["table"], s["mass"], decay=c["decay"]), "mass": s["mass"]}
    if c["op"] == "evict":
        kept, lens = s["cache"].evict(s["mass"], s["lens"], s["table"], s["new_table"], c["keep"], c["recent"])
        out = {"kept": kept, "lens": lens, "mass": s["mass"], "k": s["k"], "v": s["v"]}
        if c["cache"] == "int8":
            out["k"], out["v"] = s["cache"].read(lens, s["new_table"], min(c["keep"], s["max_len"]))
        return out
    return s["layer"](s["x"], s["x_scale"], dtype=_TYPES[c["out"]])


# ------------------------------------------------------------- bytes and flops
def work(case):
    c = case
    if c["op"] == "linear":
        n, k, m = c["n"], c["k"], c["rows"]
        return {"bytes": n * (k + 4) + m * (k + 4) + m * n * (2 if c["out"] == "bf16" else 4) + (4 * n if c["bias"] else 0),
                "flops": 2 * m * n * k}
    lens, new, sizes, prefixes = _lengths(c)
    kv, d = c["kv_heads"], c["head_dim"]
    row = d * (2 if c["cache"] == "bf16" else 1) + (4 if c["cache"] == "int8" else 0)
    if c["op"] == "evict":
        after = [min(n, c["keep"]) for n in lens]
        moved = 2 * sum(after) * kv * (2 * row + 4)  # keys, values and weights, read and written
        if c["cache"] == "int8":  # and the values that they stand for
            moved += 2 * sum(after) * kv * row + 2 * len(lens) * min(c["keep"], max(lens)) * kv * d * 2
        return {"bytes": sum(lens) * kv * 4 + moved + len(lens) * kv * c["keep"] * 4, "flops": 0}
    keys, scores = sum(prefixes) if prefixes else 0, 0
    for i, (n, t) in enumerate(zip(lens, new)):
        lo, hi = n - t + 1, n  # the keys up to the first and up to the last new token
        if not t:
            continue
        if not c.get("causal", True):
            keys, scores = keys + n, scores + n * t
            continue
        w = c.get("window", 0) or n
        full = max(0, min(t, hi - max(lo, w) + 1))  # new tokens that see a whole window
        part = t - full
        scores += full * w + (lo + lo + part - 1) * part // 2
        keys += n - max(0, lo - w)
    if prefixes:
        first = [sum(sizes[:i]) for i in range(len(sizes) + 1)]
        scores += sum(p * sum(new[a:b]) for p, a, b in zip(prefixes, first, first[1:]))
    moved = 2 * keys * kv * row + 2 * sum(new) * c["heads"] * d * 2
    if c["op"] == "weighed":
        moved += sum(n for n, t in zip(lens, new) if t) * kv * 4 * (2 if c["decay"] else 1)
    return {"bytes": moved, "flops": 4 * scores * c["heads"] * d}


# ------------------------------------------------------- definitions in 64 bits
def _rows(s, side, table, n):
    """The first n rows that one page list names, in 64 bits: [n, kv_heads, head_dim]."""
    pages = table[: -(-n // s["case"]["page"])].long()
    x = s[side][pages].double()
    if s[side + "_scale"] is not None:
        x *= s[side + "_scale"][pages].double().unsqueeze(-1)
    return x.permute(0, 2, 1, 3).flatten(0, 1)[:n]


def _history(s, i, side):
    x = _rows(s, side, s["table"][i], int(s["lens"][i]))
    if s["case"]["op"] == "shared":
        g = int(s["group_of"][i])
        x = torch.cat([_rows(s, side, s["prefix_table"][g], int(s["prefix_lens"][g])), x])
    return x


def _exact_attention(s):
    c = s["case"]
    group = c["heads"] // c["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    mass = s["mass_before"].double() if c["op"] == "weighed" else None
    for i in range(s["lens"].shape[0]):
        a, b = int(s["starts"][i]), int(s["starts"][i + 1])
        if a == b:
            continue
        keys, values = _history(s, i, "k"), _history(s, i, "v")
        n = keys.shape[0]
        place = torch.arange(n - (b - a), n, device="cuda").unsqueeze(1)
        key = torch.arange(n, device="cuda").unsqueeze(0)
        hidden = key > place if c.get("causal", True) else torch.zeros((b - a, n), dtype=torch.bool, device="cuda")
        if c.get("window", 0):
            hidden = hidden | (key <= place - c["window"])
        empty = hidden.all(1)
        received = torch.zeros((c["kv_heads"], n), dtype=torch.float64, device="cuda")
        for h in range(c["heads"]):
            x = torch.mm(s["q"][a:b, h].double(), keys[:, h // group].t()) / c["head_dim"] ** 0.5
            x[hidden] = -math.inf
            x[empty] = 0.0
            w = torch.softmax(x, 1)
            w[empty] = 0.0
            out[a:b, h] = torch.mm(w, values[:, h // group])
            received[h // group] += w.sum(0)
        if mass is not None:
            pages, slots = s["table"][i].long()[key[0] // c["page"]], key[0] % c["page"]
            old = mass[pages, :, slots] * c["decay"]
            old[n - (b - a):] = 0.0
            mass[pages, :, slots] = old + received.t()
    return out if mass is None else {"out": out, "mass": mass}


def _exact_evict(s):
    c = s["case"]
    keep, page, b = c["keep"], c["page"], s["lens"].shape[0]
    kept = torch.full((b, c["kv_heads"], keep), -1, dtype=torch.int32, device="cuda")
    pools = {x: s[x].double() for x in ("k", "v", "mass")}
    if c["cache"] == "int8":
        whole = (b, min(keep, s["max_len"]), c["kv_heads"], c["head_dim"])
        read = {x: torch.zeros(whole, dtype=torch.float64, device="cuda") for x in ("k", "v")}
    lens = []
    for i in range(b):
        n = int(s["lens"][i])
        m, key = min(n, keep), torch.arange(n, device="cuda")
        lens.append(m)
        for h in range(c["kv_heads"]):
            weight = pools["mass"][s["table"][i].long()[key // page], h, key % page].clone()
            weight[max(0, n - c["recent"]):] = math.inf
            # rank by weight, of equal ones the earlier first
            rank = torch.argsort(-weight, stable=True)
            stay = torch.sort(rank[:m])[0]
            kept[i, h, :m] = stay.int()
            old = s["table"][i].long()[stay // page], torch.full_like(stay, h), stay % page
            slot = torch.arange(m, device="cuda")
            new = s["new_table"][i].long()[slot // page], torch.full_like(slot, h), slot % page
            for x in pools:
                pools[x][new] = s[x][old].double()
            if c["cache"] == "int8":
                for x in read:
                    read[x][i, :m, h] = s[x][old].double() * s[x + "_scale"][old].double().unsqueeze(1)
    out = {"kept": kept, "lens": _int32(lens), **pools}
    return {**out, **read} if c["cache"] == "int8" else out


def _exact_linear(s):
    c = s["case"]
    y = torch.mm(s["x"].double() * s["x_scale"].double().unsqueeze(1), (s["w"].double() * s["w_scale"].double().unsqueeze(1)).t())
    if c["bias"]:
        y += s["bias"].double()
    return y * torch.sigmoid(y) if c["silu"] else y


def exact(case, seed):
    s = prepare(case, seed)
    return {"shared": _exact_attention, "weighed": _exact_attention, "evict": _exact_evict, "linear": _exact_linear}[case["op"]](s)
