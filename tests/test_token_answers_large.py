"""Shared prefixes, weighed attention and eviction over pools whose offsets pass 32 bits:
what they give at the pool's end is what they give in a small pool, to the bit."""
import pytest
import torch

from conv_bn_silu_gb300 import _binding as B
from tests import token_refs as refs

pytestmark = pytest.mark.gpu

I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def token_calls(cuda_lib):
    from conv_bn_silu_gb300 import build
    build.build_tokens()


@pytest.mark.parametrize("int8", [False, True])
def test_at_the_end_of_a_large_pool(int8):
    from conv_bn_silu_gb300 import tokens
    lens, heads, kv, d, page, keep = [700, 90, 300], 16, 8, 128, 64, 64
    paged = refs.make_paged(lens + [keep] * 3, kv, d, page, int8, 3, junk=False)
    small = paged["k"].shape[0]
    row = kv * page * d * (1 if int8 else 2)
    count = (1 << 32) // row + 2 * small   # pages: over 2^32 bytes, and 2^31 elements
    first = count - small
    big = {}
    for n in ("k", "v", "k_scale", "v_scale"):
        if paged[n] is not None:
            big[n] = torch.empty((count, *paged[n].shape[1:]), dtype=paged[n].dtype, device="cuda")
            big[n][first:].copy_(paged[n])
    compact = {n: paged[n].cuda() for n in big}
    caches = [tokens.PagedCache(p["k"], p["v"], p.get("k_scale"), p.get("v_scale")) for p in (compact, big)]
    masses = [torch.zeros((n, kv, page), device="cuda") for n in (small, count)]
    table = paged["table"].cuda()
    tables = [table, torch.where(table < 0, table, table + first)]
    i32 = lambda v: torch.tensor(v, dtype=I32, device="cuda")
    for new in (1, 60):   # few rows, chunks
        starts = i32([0, new, 2 * new, 3 * new])
        q = torch.randn((3 * new, heads, d), generator=torch.Generator().manual_seed(new)).to(torch.bfloat16).cuda()
        got = []
        for cache, mass, t in zip(caches, masses, tables):
            own = t[:3].contiguous()
            a = tokens.WeighedAttention(cache, 3, new, 700, heads)(q, starts, i32(lens), own, mass, decay=0.5)
            # the first sequence's pages as the prefix of the others
            group = i32([0, 3])
            b = tokens.SharedPrefixAttention(cache, 3, 1, new, 300, 700, heads)(
                q, starts, i32([90, 90, 300]), own[[1, 1, 2]].contiguous(), group, i32([700]), own[:1].contiguous())
            got.append((a, b))
        for x, y in zip(*got):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16)), new
    kept = [c.evict(m, i32(lens), t[:3].contiguous(), t[3:].contiguous(), keep, 5) for c, m, t in zip(caches, masses, tables)]
    assert torch.equal(kept[0][0], kept[1][0]) and torch.equal(kept[0][1], kept[1][1])
    assert B.cbs_read_device_status(True, torch.cuda.current_stream().cuda_stream) == B.CBS_OK
    assert torch.equal(masses[0], masses[1][first:]) and not masses[1][:first].any()
    for n in big:
        raw = lambda t: t.view(torch.int8) if t.dtype == torch.int8 else t.view(torch.int16 if t.dtype == torch.bfloat16 else I32)
        assert torch.equal(raw(compact[n]), raw(big[n][first:])), n
