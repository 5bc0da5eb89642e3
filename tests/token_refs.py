"""Plain 64-bit forms of the token operators, and inputs for their tests."""
from __future__ import annotations

import math

import torch


def make_paged(lens, kv_heads, head_dim, page, int8, seed, spare=2, junk=True):
    """A pool whose slots past the sequences' lengths hold NaN (junk), the
    page table (-1 where unused) and each sequence's rows in order."""
    g = torch.Generator().manual_seed(seed)
    count = [-(-n // page) for n in lens]
    pool = sum(count) + spare
    order = torch.randperm(pool, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(max(count), 1)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(count):
        table[b, :n] = order[at:at + n]
        at += n
    shape = (pool, kv_heads, page, head_dim)
    out = {"table": table}
    for side in ("k", "v"):
        if int8:
            out[side] = torch.randint(-127, 128, shape, generator=g, dtype=torch.int8)
            out[side + "_scale"] = torch.rand(shape[:3], generator=g) * 0.02 + 0.005
        else:
            out[side] = torch.randn(shape, generator=g).to(torch.bfloat16)
            out[side + "_scale"] = None
    if junk:
        used = torch.zeros((pool, page), dtype=torch.bool)
        for b, n in enumerate(lens):
            for pos in range(n):
                used[table[b, pos // page], pos % page] = True
        for side in ("k", "v"):
            hole = (~used)[:, None, :].expand(pool, kv_heads, page)
            if int8:
                out[side + "_scale"][hole] = float("nan")
            else:
                out[side][hole] = float("nan")
    return out


def rows_of(paged, side, b, n, page):
    """Sequence b's first n rows in 64 bits: [n, kv_heads, head_dim]."""
    pages = paged["table"][b, : -(-n // page)].long()
    x = paged[side].cpu()[pages].double()
    if paged[side + "_scale"] is not None:
        x = x * paged[side + "_scale"].cpu()[pages].double()[..., None]
    return x.permute(0, 2, 1, 3).reshape(-1, x.shape[1], x.shape[3])[:n]


def attention(q, paged, starts, lens, page, causal, window, scale):
    """(out, A): the attention in 64 bits, and sum p |v| / sum p, the size that
    a relative error of the probabilities is weighed with."""
    q = q.double()
    out, mag = torch.zeros_like(q), torch.zeros_like(q)
    kv = paged["k"].shape[1]
    group = q.shape[1] // kv
    for b, n in enumerate(lens):
        a, e = starts[b], starts[b + 1]
        if e == a or n == 0:
            continue
        k, v = rows_of(paged, "k", b, n, page), rows_of(paged, "v", b, n, page)
        place = torch.arange(n - (e - a), n)[:, None]
        key = torch.arange(n)[None]
        seen = torch.ones((e - a, n), dtype=torch.bool)
        if causal:
            seen &= key <= place
        if window:
            seen &= key > place - window
        for h in range(q.shape[1]):
            s = (q[a:e, h] @ k[:, h // group].nan_to_num(0.0, 0.0, 0.0).T) * scale
            s = torch.where(seen, s, -math.inf)
            top = s.amax(1, keepdim=True)
            p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
            p = torch.where(seen, p, torch.zeros_like(p))
            total = p.sum(1, keepdim=True)
            p = p / torch.where(total == 0, torch.ones_like(total), total)
            # a value that is not finite reaches only the tokens that see it
            vh = v[:, h // group]
            fine = vh.isfinite()
            clean = torch.where(fine, vh, torch.zeros_like(vh))
            o = p @ clean
            bad = (seen.double() @ (~fine).double()) > 0
            out[a:e, h] = torch.where(bad, torch.full_like(o, math.nan), o)
            mag[a:e, h] = p @ clean.abs()
    return out, mag


def attention_bound(ref, mag):
    """How far a bf16 output may be: its own rounding and each probability's
    rounding to bf16 (eight significant bits: at most 2^-8 of the value each),
    and 2^-11 for the scores' 32-bit sums and the exponential (each score is
    off by at most 2^-23 * D * |q||k|, below 2^-12 for the inputs here)."""
    return 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -11) * mag + 1e-30


def quantise_rows(x):
    """The library's 8-bit rows, in IEEE float32 steps: (codes, scale)."""
    x = x.float()
    top = x.abs().amax(-1)
    s = top / torch.full_like(top, 127.0)
    bad = ~x.isfinite().all(-1)
    codes = (x / torch.where(s > 0, s, torch.ones_like(s))[..., None]).round().clamp(-127, 127)
    codes = torch.where(bad[..., None] | (s == 0)[..., None], torch.zeros_like(codes), codes)
    return codes.to(torch.int8), torch.where(bad, torch.full_like(s, math.nan), s)


def pack_w4(codes):
    """[n, k] codes in 0..15 -> the packed bytes [n, k / 2]."""
    n, k = codes.shape
    c = codes.view(n, k // 8, 8).to(torch.uint8)
    nib = torch.stack([c[..., 0], c[..., 2], c[..., 4], c[..., 6], c[..., 1], c[..., 3], c[..., 5], c[..., 7]], -1)
    return (nib[..., 0::2] | (nib[..., 1::2] << 4)).reshape(n, k // 2).contiguous()
