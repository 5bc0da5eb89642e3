"""Attention that weighs the cache's positions, against a plain 64-bit form."""
import ctypes
import math

import pytest
import torch

from conv_bn_silu_gb300 import _binding as B
from tests import token_refs as refs
from tests.test_tokens_refusals import I, M, OK, P, W, cache as c_cache, desc, refused, seqs

I32 = torch.int32
CHUNK = B.CBS_ATTN_CHUNK


@pytest.fixture(scope="module", autouse=True)
def token_calls(cuda_lib):
    from conv_bn_silu_gb300 import build
    build.build_tokens()


def received(q, paged, starts, lens, page, causal, window, scale):
    """What each sequence's positions receive, per key head ([kv, length]), and how
    far 32-bit arithmetic may be from it.

    A score's sum of D products, each addition rounded or cut (2^-23 of the sum of
    magnitudes at most), moves it by D 2^-23 sum |q k| scale, and so its weight by as
    much of itself; the row's sum by its largest such move.  The exponentials (2 ulp)
    and the product with 1 / sum add 2^-20, the n additions of the row's sum n 2^-23,
    and the R additions of a position's R 2^-23."""
    q = q.double()
    kv = paged["k"].shape[1]
    group = q.shape[1] // kv
    out = []
    for b, n in enumerate(lens):
        a, e = starts[b], starts[b + 1]
        got, far = torch.zeros((kv, n), dtype=torch.float64), torch.zeros((kv, n), dtype=torch.float64)
        out.append((got, far))
        if e == a or n == 0:
            continue
        k = refs.rows_of(paged, "k", b, n, page)
        place, key = torch.arange(n - (e - a), n)[:, None], torch.arange(n)[None]
        seen = torch.ones((e - a, n), dtype=torch.bool)
        if causal:
            seen &= key <= place
        if window:
            seen &= key > place - window
        for h in range(q.shape[1]):
            kh = k[:, h // group]
            s = torch.where(seen, (q[a:e, h] @ kh.T) * scale, -math.inf)
            top = s.amax(1, keepdim=True)
            p = torch.where(seen, torch.exp(s - torch.where(top == -math.inf, 0.0, top)), 0.0)
            total = p.sum(1, keepdim=True)
            p = p / torch.where(total == 0, 1.0, total)
            move = kh.shape[1] * 2.0 ** -23 * (q[a:e, h].abs() @ kh.abs().T) * abs(scale)
            move = torch.where(seen, move, 0.0)
            got[h // group] += p.sum(0)
            far[h // group] += (p * (move + move.amax(1, keepdim=True) + 2.0 ** -20 + n * 2.0 ** -23)).sum(0)
        far += got * ((e - a) * group * 2.0 ** -23)
    return out


def run_case(lens, new, heads, kv, d, page, int8, causal=True, window=0, scale=None, seed=0, kernel=-1, split=0, decay=1.0, padding=0,
             q=None, paged=None):
    from conv_bn_silu_gb300 import tokens
    paged = paged or refs.make_paged(lens, kv, d, page, int8, seed)
    starts = [sum(new[:i]) for i in range(len(new) + 1)]
    if q is None:
        q = torch.randn((starts[-1] + padding, heads, d), generator=torch.Generator().manual_seed(seed + 1)).to(torch.bfloat16)
    dev = {n: None if t is None else t.cuda() for n, t in paged.items()}
    cache = tokens.PagedCache(dev["k"], dev["v"], dev["k_scale"], dev["v_scale"])
    kinds = (cache, len(lens), max(max(new), 1), max(max(lens), 1), heads)
    attn = tokens.WeighedAttention(*kinds, causal=causal, window=window, scale=scale, force_kernel=kernel, force_split=split)
    plain = tokens.PagedAttention(*kinds, causal=causal, window=window, scale=scale, force_kernel=kernel, force_split=split)
    if q.shape[0] > len(lens) * max(max(new), 1):
        q = q[:starts[-1]]
    i32 = lambda v: torch.tensor(v, dtype=I32, device="cuda")
    args = (q.cuda(), i32(starts), i32(lens), dev["table"])
    pool = paged["k"].shape[0]
    before = torch.rand((pool, kv, page), generator=torch.Generator().manual_seed(seed + 2))
    # (what it was says nothing where the positions are new, or where it is forgotten)
    for b, n in enumerate(lens):
        for pos in range(0 if decay == 0.0 and new[b] else n - new[b], n):
            before[paged["table"][b, pos // page], :, pos % page] = math.nan
    mass = before.cuda()
    out = attn(*args, mass, decay=decay)
    if attn.plan.attention.kernel == plain.plan.kernel:
        assert torch.equal(out.view(torch.int16), plain(*args).view(torch.int16))   # the same attention, to the bit
    ref, mag = refs.attention(q, paged, starts, lens, page, causal, window, scale or d ** -0.5)
    assert ((out.double().cpu() - ref).abs() <= refs.attention_bound(ref, mag)).all()
    again = before.cuda()
    attn(*args, again, decay=decay, out=torch.empty_like(out))
    assert torch.equal(mass.view(I32), again.view(I32))
    assert B.cbs_read_device_status(True, torch.cuda.current_stream().cuda_stream) == B.CBS_OK
    got = mass.cpu().double()
    untouched = torch.ones((pool, page), dtype=torch.bool)
    for b, (rec, far) in enumerate(received(q, paged, starts, lens, page, causal, window, scale or d ** -0.5)):
        n = lens[b]
        if new[b] == 0:
            continue
        pos = torch.arange(n)
        pages, slots = paged["table"][b].long()[pos // page], pos % page
        untouched[pages, slots] = False
        old = before[pages, :, slots].T.double() * decay if decay else torch.zeros_like(rec)
        old[:, n - new[b]:] = 0.0
        want = old + rec
        bound = far + 2.0 ** -23 * (old + rec) + 1e-30
        here = got[pages, :, slots].T
        nan = want.isnan()
        assert torch.equal(here.isnan(), nan)
        err = (here - want).abs()
        assert (err <= bound)[~nan].all(), (b, float((err / bound)[~nan].max()))
    keep = untouched[:, None].expand(-1, kv, -1)
    assert torch.equal(mass.cpu()[keep].view(I32), before[keep].view(I32))   # other places as they were
    return attn


@pytest.mark.gpu
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[1], [2], [15], [16], [17], [63, 1, 300], [1000], [513, 0, 16, 31]])
def test_single_tokens(lens, d, int8):
    run_case(lens, [min(1, n) for n in lens], 8, 2, d, 16, int8, decay=0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("split", [1, 2, 7, 8, 20])
def test_ranges(split, int8):
    for kernel in (B.CBS_ATTN_ROWS, B.CBS_ATTN_CLUSTER, CHUNK):
        run_case([700, 90, 0], [1, 1, 0], 8, 2, 64, 16, int8, kernel=kernel, split=split)


@pytest.mark.gpu
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("heads,kv,d,page", [(8, 8, 64, 16), (6, 1, 128, 64), (24, 4, 64, 32), (4, 2, 128, 256), (5, 5, 128, 16), (9, 3, 64, 128)])
@pytest.mark.parametrize("decay", [0.0, 1.0, -0.25])
def test_chunks(heads, kv, d, page, int8, decay):
    run_case([300, 77, 5, 260], [100, 77, 1, 0], heads, kv, d, page, int8, decay=decay, padding=4)


@pytest.mark.gpu
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("kernel", [B.CBS_ATTN_ROWS, B.CBS_ATTN_CLUSTER, CHUNK])
@pytest.mark.parametrize("heads,kv,new", [(8, 2, [5, 1, 0]), (6, 1, [40, 33, 7]), (64, 1, [3, 2, 1]), (40, 8, [9, 1, 1])])
def test_every_kernel(heads, kv, new, kernel, int8):
    """More rows than a few-row tile, by either kernel: their scores are summed up by
    warps side by side."""
    run_case([90, 33, 400], new, heads, kv, 64, 16, int8, kernel=kernel, decay=0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 1), (True, 50), (True, 128), (False, 40), (True, 1 << 30), (True, 2 ** 31 - 1)])
@pytest.mark.parametrize("new", [[1, 1, 1], [3, 2, 1], [150, 33, 400]])
def test_masks(new, causal, window, int8):
    run_case([400, 33, 900], new, 8, 2, 64, 16, int8, causal=causal, window=window)


@pytest.mark.gpu
def test_many_rows():
    """Rows' buffers gone round many times, few keys; and keys beyond one tile of many."""
    run_case([130], [130], 64, 1, 64, 16, False)
    run_case([64], [64], 96, 1, 128, 64, True, causal=False)
    run_case([3000], [260], 8, 1, 128, 64, False, window=700)
    for heads in (129, 131, 160, 256):   # more query heads of a key head than a tile has rows
        run_case([140, 20], [3, 2], heads, 1, 64, 16, heads % 2 == 0, kernel=CHUNK)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1e-3, 1.5, -0.5])
@pytest.mark.parametrize("new", [[1, 1], [40, 90]])
def test_scales(new, scale):
    run_case([200, 140], new, 8, 2, 64, 16, False, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("new", [[1, 1], [3, 60]])
@pytest.mark.parametrize("size", [30.0, 1e18])
def test_one_key_takes_all(new, size, int8):
    """Rows so long that a score's last place is more than any difference that
    counts: a position then has a row's whole weight or none of it."""
    from conv_bn_silu_gb300 import tokens
    lens, heads, kv, d, page = [70, 130], 4, 2, 64, 16
    paged = refs.make_paged(lens, kv, d, page, int8, 9, junk=False)
    starts = [0, new[0], sum(new)]
    q = torch.randn((starts[-1], heads, d), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16) * size
    dev = {n: None if t is None else t.cuda() for n, t in paged.items()}
    cache = tokens.PagedCache(dev["k"], dev["v"], dev["k_scale"], dev["v_scale"])
    i32 = lambda v: torch.tensor(v, dtype=I32, device="cuda")
    mass = torch.zeros((paged["k"].shape[0], kv, page), device="cuda")
    attn = tokens.WeighedAttention(cache, 2, max(new), 130, heads, scale=100.0)
    attn(q.cuda(), i32(starts), i32(lens), dev["table"], mass)
    assert B.cbs_read_device_status(True, torch.cuda.current_stream().cuda_stream) == B.CBS_OK
    got = mass.cpu().double()
    for b, (rec, _) in enumerate(received(q, paged, starts, lens, page, True, 0, 100.0)):
        pos = torch.arange(lens[b])
        here = got[paged["table"][b].long()[pos // page], :, pos % page].T
        # whole numbers: no two of these keys' scores are within 2^-20 of one another
        assert torch.equal(rec.round(), here.round()), b
        assert (here - here.round()).abs().max() <= 1e-3


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 40])
def test_values_that_are_not_finite(new):
    """A NaN among the values is the output's business alone; a key's NaN makes the
    weights of every position that its row sees NaN, and of no other."""
    lens, news = [100, 90], [new, new]
    paged = refs.make_paged(lens, 2, 64, 16, False, 11)
    paged["v"][paged["table"][0, 1], 0, 2] = math.nan
    from conv_bn_silu_gb300 import tokens
    def weights(paged):
        dev = {n: None if t is None else t.cuda() for n, t in paged.items()}
        cache = tokens.PagedCache(dev["k"], dev["v"])
        q = torch.randn((2 * new, 4, 64), generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
        mass = torch.zeros((paged["k"].shape[0], 2, 16), device="cuda")
        i32 = lambda v: torch.tensor(v, dtype=I32, device="cuda")
        tokens.WeighedAttention(cache, 2, new, 100, 4)(q, i32([0, new, 2 * new]), i32(lens), dev["table"], mass)
        pos = torch.arange(100)
        first = mass.cpu()[paged["table"][0].long()[pos // 16], :, pos % 16]
        pos = pos[:90]
        return first, mass.cpu()[paged["table"][1].long()[pos // 16], :, pos % 16]
    first, second = weights(paged)
    assert first.isfinite().all() and second.isfinite().all()
    assert abs(first.sum().item() - 4 * new) < 1e-3 * new and abs(second.sum().item() - 4 * new) < 1e-3 * new
    paged["k"][paged["table"][0, 99 // 16], 1, 99 % 16] = math.nan   # seen by the last token alone
    third, fourth = weights(paged)
    assert torch.equal(third[:, 0], first[:, 0]) and torch.equal(fourth, second)
    assert third[:, 1].isnan().all()


@pytest.mark.gpu
def test_longer_than_planned():
    from conv_bn_silu_gb300 import tokens
    for new in (1, 40):
        paged = refs.make_paged([100, 60], 2, 64, 16, True, 1)
        cache = tokens.PagedCache(*(paged[n].cuda() for n in ("k", "v", "k_scale", "v_scale")))
        attn = tokens.WeighedAttention(cache, 2, new, 64, 4)
        i32 = lambda v: torch.tensor(v, dtype=I32, device="cuda")
        mass = torch.full((paged["k"].shape[0], 2, 16), -1.0, device="cuda")
        q = torch.ones((2 * new, 4, 64), dtype=torch.bfloat16, device="cuda")
        attn(q, i32([0, new, 2 * new]), i32([100, 60]), paged["table"].cuda(), mass, decay=0.0)
        assert B.cbs_read_device_status(True, torch.cuda.current_stream().cuda_stream) == B.CBS_ERR_INVALID_ARG
        at = lambda b, pos: mass[paged["table"][b].long()[pos // 16].cuda(), :, (pos % 16).cuda()]
        assert (at(0, torch.arange(64, 100)) == -1).all() and (at(0, torch.arange(64)) >= 0).all()
        assert abs(at(1, torch.arange(60)).sum().item() - 4 * new) < 1e-3 * new


@pytest.mark.gpu
def test_streams_forks_and_graphs():
    from conv_bn_silu_gb300 import tokens
    lens = [3000, 50, 60]
    paged = refs.make_paged(lens, 2, 64, 16, True, 5)
    cache = tokens.PagedCache(*(paged[n].cuda() for n in ("k", "v", "k_scale", "v_scale")))
    i32 = lambda v: torch.tensor(v, dtype=I32, device="cuda")
    table = paged["table"].cuda()
    for new in (1, 30):
        q = torch.randn((3, 3 * new, 8, 64), device="cuda", generator=torch.Generator("cuda").manual_seed(6)).to(torch.bfloat16)
        rest = (i32([0, new, 2 * new, 3 * new]), i32(lens), table)
        attn = tokens.WeighedAttention(cache, 3, new, 3000, 8)
        blank = lambda: torch.zeros((paged["k"].shape[0], 2, 16), device="cuda")
        masses = [blank() for _ in q]
        want = [attn(x, *rest, m, decay=0.5) for x, m in zip(q, masses)]
        streams, forks, got = [torch.cuda.Stream() for _ in q], [attn.fork() for _ in q], [[] for _ in q]
        torch.cuda.synchronize()
        for _ in range(10):
            for i, (s, f) in enumerate(zip(streams, forks)):
                with torch.cuda.stream(s):
                    m = blank()
                    got[i].append((f(q[i], *rest, m, decay=0.5), m))
        torch.cuda.synchronize()
        assert all(torch.equal(want[i], o) and torch.equal(masses[i], m) for i in range(3) for o, m in got[i])
        graph, held, mass = torch.cuda.CUDAGraph(), q[0].clone(), blank()
        with torch.cuda.graph(graph):
            out = attn(held, *rest, mass, decay=0.5)
        for i in (2, 1, 0):
            held.copy_(q[i])
            mass.zero_()
            graph.replay()
            assert torch.equal(out, want[i]) and torch.equal(mass, masses[i])


def test_refusals(cuda_lib):
    plan = B.cbs_weighed_plan(desc(force_split=2, force_kernel=B.CBS_ATTN_ROWS))
    assert plan.size == ctypes.sizeof(plan) and plan.workspace_bytes > plan.attention.workspace_bytes > 0
    K = 1 << 30
    def call(p=plan, c=None, s=None, q=K, scale=0.1, out=2 * K, mass=3 * K, decay=1.0, ws=4 * K, wb=None):
        B.cbs_weighed_attention(p, c or c_cache(k=5 * K, v=6 * K, k_scale=7 * K, v_scale=8 * K), s or seqs(), q, 256, scale, out, 256, mass,
                                decay, ws, plan.workspace_bytes if wb is None else wb, None)
    refused(I, lambda: call(mass=None))
    refused(M, lambda: call(mass=3 * K + 4))
    refused(I, lambda: call(decay=float("nan")))
    refused(I, lambda: call(decay=float("inf")))
    refused(I, lambda: call(scale=float("nan")))
    refused(I, lambda: call(q=None))
    refused(I, lambda: call(out=K))
    refused(W, lambda: call(ws=None))
    refused(W, lambda: call(wb=plan.attention.workspace_bytes))
    refused(P, lambda: call(c=c_cache(kv_heads=4)))
    refused(I, lambda: call(s=seqs(total=9)))
    for other in (K, 2 * K, 4 * K, 5 * K, 6 * K, 7 * K, 8 * K):   # on what the call reads or writes
        refused(I, lambda: call(mass=other))
    bad = B.cbs_weighed_plan_t.from_buffer_copy(plan)
    bad.abi_version = 1
    refused(P, lambda: call(p=bad))
    call(s=seqs(total=0), mass=None)
    refused(I, B.cbs_weighed_plan, desc(heads=3))


def test_python_refusals():
    from tests.test_tokens_devices import fake
    from conv_bn_silu_gb300 import tokens
    plan = B.cbs_weighed_plan(desc(batch=1))
    cache = B.cbs_cache(None, None, None, None, B.CBS_INT8, 4, 16, 2, 64)
    bf = torch.bfloat16
    kinds = [((3, 4, 64), bf), ((3, 4, 64), bf), ((2,), I32), ((1,), I32), ((1, 4), I32), ((4, 2, 16), torch.float32)]
    def call(made):
        q, out, starts, lens, table, mass = made
        tokens._calls().weighed_attention(ctypes.addressof(plan), ctypes.addressof(cache), 0, q, starts, lens, table, 0.1, out, None, 0, mass, 1.0)
    for wrong in range(6):
        with pytest.raises(ValueError, match="device"):
            call([fake(s, t, int(i == wrong)) for i, (s, t) in enumerate(kinds)])
    for i, other in ((5, ((4, 2, 8), torch.float32)), (5, ((4, 2, 16), bf)), (5, ((4, 2), torch.float32)), (0, ((3, 8, 64), bf))):
        some = list(kinds)
        some[i] = other
        with pytest.raises(ValueError):
            call([fake(s, t) for s, t in some])
