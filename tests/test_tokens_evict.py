"""Eviction from a paged cache by weight: which positions stay, and that all that
belongs to them moves, against a plain choice position by position."""
import math

import pytest
import torch

from conv_bn_silu_gb300 import _binding as B
from tests import token_refs as refs
from tests.test_tokens_refusals import I, M, OK, U, cache as c_cache, refused, seqs

I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def token_calls(cuda_lib):
    from conv_bn_silu_gb300 import build
    build.build_tokens()


def stays(weights, keep, recent):
    """The positions of one head that stay, in order."""
    n = len(weights)
    recent, take = min(recent, n), min(keep, n)
    rank = lambda i: (-math.inf if math.isnan(weights[i]) else -weights[i], not math.isnan(weights[i]), i)
    heaviest = sorted(range(n - recent), key=rank)[:take - recent]
    return sorted(heaviest) + list(range(n - recent, n))


def setup(lens, keep, kv, d, page, int8, seed, mass=None, spare=0):
    """A pool with the sequences' pages and room for what stays, on the CPU."""
    after = [min(n, keep) for n in lens]
    paged = refs.make_paged(lens + after, kv, d, page, int8, seed, junk=False)
    table, new = paged["table"][:len(lens)], paged["table"][len(lens):]
    table = table[:, :max(1, -(-max(lens) // page) + spare)].contiguous()
    g = torch.Generator().manual_seed(seed + 7)
    pool = paged["k"].shape[0]
    weights = torch.rand((pool, kv, page), generator=g) if mass is None else mass(torch.rand((pool, kv, page), generator=g))
    return paged, table, new.contiguous(), weights


def run_case(lens, keep, recent, kv=2, d=64, page=16, int8=True, seed=0, mass=None):
    from conv_bn_silu_gb300 import tokens
    paged, table, new, weights = setup(lens, keep, kv, d, page, int8, seed, mass)
    pools = {n: paged[n] for n in ("k", "v", "k_scale", "v_scale") if paged[n] is not None}
    pools["mass"] = weights
    want = {n: t.clone() for n, t in pools.items()}
    dev = {n: t.cuda() for n, t in pools.items()}
    cache = tokens.PagedCache(dev["k"], dev["v"], dev.get("k_scale"), dev.get("v_scale"))
    kept, after = cache.evict(dev["mass"], torch.tensor(lens, dtype=I32, device="cuda"), table.cuda(), new.cuda(), keep, recent)
    assert B.cbs_read_device_status(True, torch.cuda.current_stream().cuda_stream) == B.CBS_OK
    assert after.tolist() == [min(n, keep) for n in lens]
    kept = kept.cpu()
    for b, n in enumerate(lens):
        for h in range(kv):
            pos = torch.arange(n)
            w = weights[table[b].long()[pos // page], h, pos % page].tolist()
            rows = stays(w, keep, recent)
            assert kept[b, h].tolist() == rows + [-1] * (keep - len(rows)), (b, h)
            old, to = torch.tensor(rows, dtype=torch.long), torch.arange(len(rows))
            for name, pool in want.items():
                pool[new[b].long()[to // page], h, to % page] = pools[name][table[b].long()[old // page], h, old % page]
    for name, pool in want.items():
        raw = pool.view({8: torch.int8, 16: torch.int16, 32: torch.int32}[8 * pool.element_size()])
        assert torch.equal(dev[name].cpu().view(raw.dtype), raw), name   # bit for bit, the other pages as they were


@pytest.mark.gpu
@pytest.mark.parametrize("int8,d,page", [(True, 64, 16), (True, 128, 64), (False, 64, 32), (False, 128, 16), (True, 64, 256)])
@pytest.mark.parametrize("lens,keep,recent", [
    ([1], 1, 0), ([1], 1, 1), ([1], 5, 2), ([2, 0, 3], 2, 1), ([17], 16, 0), ([40], 16, 16), ([300, 33, 0, 1000], 100, 7),
    ([1000, 999], 999, 500), ([2500], 1, 0), ([130], 129, 128),
])
def test_sizes(lens, keep, recent, int8, d, page):
    run_case(lens, keep, recent, d=d, page=page, int8=int8)


@pytest.mark.gpu
@pytest.mark.parametrize("name,mass", [
    ("equal", lambda r: torch.zeros_like(r)),
    ("two values", lambda r: (r > 0.5).float() * 3),
    ("signs and zeros", lambda r: torch.where(r < 0.2, -r, torch.where(r < 0.4, torch.where(r < 0.3, 0.0, -0.0), r))),
    ("tiny", lambda r: r * 1e-42),
    ("infinities", lambda r: torch.where(r < 0.1, -math.inf, torch.where(r > 0.9, math.inf, r))),
    ("NaN", lambda r: torch.where(r < 0.1, math.nan, torch.where(r > 0.9, math.inf, r))),
    ("negative NaN", lambda r: torch.where(r < 0.1, -torch.tensor(math.nan), r)),
    ("one bit", lambda r: (torch.full_like(r, 1.0).view(I32) + (r * 7).to(I32)).view(torch.float32)),
])
def test_weights(name, mass):
    run_case([700, 90], 300, 20, mass=mass)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,keep,recent", [([50000, 3], 20000, 100), ([120001], 7, 2), ([120001], 119999, 0), ([49153], 40000, 39999)])
def test_long_sequences(lens, keep, recent):
    """Past one CTA's share of the positions: clusters, ties across their edges."""
    run_case(lens, keep, recent, kv=1, page=64, mass=lambda r: (r * 50).floor())


@pytest.mark.gpu
def test_bad_pages():
    """An old page outside the pool is reported and moves nothing; so is a new one."""
    from conv_bn_silu_gb300 import tokens
    paged, table, new, weights = setup([40, 40], 20, 2, 64, 16, True, 1)
    dev = {n: paged[n].cuda() for n in ("k", "v", "k_scale", "v_scale")}
    cache = tokens.PagedCache(*dev.values())
    lens = torch.tensor([40, 40], dtype=I32, device="cuda")
    for which, row in (("old", 0), ("new", 1)):
        for bad in (-1, 10 ** 6):
            t, n = table.clone(), new.clone()
            (t if which == "old" else n)[row, 1] = bad
            kept, after = cache.evict(weights.cuda(), lens, t.cuda(), n.cuda(), 20, 5)
            assert B.cbs_read_device_status(True, torch.cuda.current_stream().cuda_stream) == B.CBS_ERR_INVALID_ARG
            assert after.tolist() == [20, 20] and kept.max() < 40
    # a length past the table's end is cut to it, and reported
    kept, after = cache.evict(weights.cuda(), lens + 1000, table.cuda(), new.cuda(), 20, 5)
    assert B.cbs_read_device_status(True, torch.cuda.current_stream().cuda_stream) == B.CBS_ERR_INVALID_ARG
    assert after.tolist() == [20, 20] and kept.max() < 48


@pytest.mark.gpu
def test_captured_and_other_streams():
    from conv_bn_silu_gb300 import tokens
    paged, table, new, weights = setup([500, 77], 64, 2, 64, 16, True, 2)
    dev = {n: paged[n].cuda() for n in ("k", "v", "k_scale", "v_scale")}
    cache = tokens.PagedCache(*dev.values())
    args = (weights.cuda(), torch.tensor([500, 77], dtype=I32, device="cuda"), table.cuda(), new.cuda(), 64, 8)
    first = [t.clone() for t in cache.evict(*args)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = cache.evict(*args)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            third = cache.evict(*args)
        for t in third:
            t.zero_()
        graph.replay()
        graph.replay()
    side.synchronize()
    for got in (second, third):
        assert all(torch.equal(a, b) for a, b in zip(first, got))


@pytest.mark.gpu
def test_nothing_held():
    """Tables without pages: no position stays, and none is looked for."""
    from conv_bn_silu_gb300 import tokens
    cache = tokens.PagedCache.empty(3, 2, 16, 64)
    mass = torch.zeros((3, 2, 16), device="cuda")
    i32 = lambda *shape: torch.zeros(shape, dtype=I32, device="cuda")
    kept, after = cache.evict(mass, i32(2), i32(2, 0), i32(2, 0), 5, 1)
    assert (kept == -1).all() and not after.any()
    kept, after = cache.evict(mass, i32(0), i32(0, 4), i32(0, 4), 5, 1)
    assert kept.shape == (0, 2, 5) and after.shape == (0,)
    assert B.cbs_read_device_status(True, torch.cuda.current_stream().cuda_stream) == B.CBS_OK


def test_refusals(cuda_lib):
    K = 1 << 30   # addresses that are checked for alignment and overlap only
    def call(c=None, s=None, mass=2 * K, table=3 * K, pages=4, keep=8, recent=2, kept=4 * K, lens=5 * K):
        B.cbs_cache_evict(c or c_cache(k=6 * K, v=7 * K, k_scale=8 * K, v_scale=9 * K), s or seqs(new_start=None, seq_lens=10 * K, page_table=11 * K),
                          mass, table, pages, keep, recent, kept, lens, None)
    refused(I, lambda: call(keep=0))
    refused(U, lambda: call(keep=(1 << 30) + 1, pages=64))
    refused(I, lambda: call(recent=-1))
    refused(I, lambda: call(recent=9))
    refused(I, lambda: call(pages=0))
    refused(I, lambda: call(keep=65, pages=3))
    refused(I, lambda: call(pages=-1))
    refused(U, lambda: call(s=seqs(max_pages=1 << 15), pages=1 << 15, keep=100))
    refused(I, lambda: call(mass=None))
    refused(M, lambda: call(mass=2 * K + 4))
    refused(I, lambda: call(table=None))
    refused(M, lambda: call(table=3 * K + 2))
    refused(I, lambda: call(kept=None))
    refused(I, lambda: call(lens=None))
    refused(U, lambda: call(c=c_cache(head_dim=96)))
    refused(I, lambda: call(lens=10 * K))        # on the lengths that are read
    refused(I, lambda: call(kept=2 * K + 16))    # on the weights
    refused(I, lambda: call(mass=6 * K))         # on the keys
    refused(I, lambda: call(kept=3 * K))         # on the new table
    call(s=seqs(batch=0), mass=None, kept=None, lens=None)


def test_python_refusals():
    from tests.test_tokens_devices import fake, calls  # noqa: F401
    import ctypes
    from conv_bn_silu_gb300 import tokens
    desc = B.cbs_cache(None, None, None, None, B.CBS_INT8, 4, 16, 2, 64)
    at = ctypes.addressof(desc), 0
    kinds = [((4, 2, 16), torch.float32), ((1,), I32), ((1, 4), I32), ((1, 2), I32)]
    for wrong in range(4):   # each on another device in turn
        with pytest.raises(ValueError, match="device"):
            tokens._calls().cache_evict(*at, *(fake(s, t, int(i == wrong)) for i, (s, t) in enumerate(kinds)), 8, 2)
    for i, other in ((0, ((4, 2, 8), torch.float32)), (0, ((4, 2, 16), torch.bfloat16)), (3, ((2, 2), I32)), (3, ((1, 2), torch.int64))):
        some = list(kinds)
        some[i] = other
        with pytest.raises(ValueError):
            tokens._calls().cache_evict(*at, *(fake(s, t) for s, t in some), 8, 2)
    with pytest.raises(ValueError, match="recent"):
        tokens._calls().cache_evict(*at, *(fake(s, t) for s, t in kinds), 8, 9)
