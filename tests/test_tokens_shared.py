"""Attention of sequences that go on from shared prefixes, against a plain 64-bit
form over each sequence's whole history."""
import ctypes
import math

import pytest
import torch

from conv_bn_silu_gb300 import _binding as B
from tests import token_refs as refs
from tests.test_tokens_refusals import I, M, OK, P, U, W, cache as c_cache, refused, seqs

I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def token_calls(cuda_lib):
    from conv_bn_silu_gb300 import build
    build.build_tokens()


def starts_of(counts):
    return [sum(counts[:i]) for i in range(len(counts) + 1)]


def reference(q, paged, own_rows, prefix_rows, group_of, starts, lens, prefixes, page, scale):
    """(out, sum p |v|) in 64 bits; a value that is not finite reaches those that see it."""
    q = q.double()
    out, mag = torch.zeros_like(q), torch.zeros_like(q)
    kv = paged["k"].shape[1]
    group = q.shape[1] // kv
    for b, n in enumerate(lens):
        a, e = starts[b], starts[b + 1]
        if a == e:
            continue
        g = group_of[b]
        both = [torch.cat([refs.rows_of(dict(paged, table=prefix_rows), side, g, prefixes[g], page),
                           refs.rows_of(dict(paged, table=own_rows), side, b, n, page)]) for side in ("k", "v")]
        k, v = both
        pre, total = prefixes[g], prefixes[g] + n
        place = torch.arange(total - (e - a), total)[:, None]
        key = torch.arange(total)[None]
        seen = (key < pre) | (key <= place)
        for h in range(q.shape[1]):
            s = torch.where(seen, (q[a:e, h] @ k[:, h // group].T) * scale, -math.inf)
            top = s.amax(1, keepdim=True)
            p = torch.where(seen, torch.exp(s - torch.where(top == -math.inf, 0.0, top)), 0.0)
            total_p = p.sum(1, keepdim=True)
            p = p / torch.where(total_p == 0, 1.0, total_p)
            vh = v[:, h // group]
            fine = vh.isfinite()
            clean = torch.where(fine, vh, 0.0)
            bad = (seen.double() @ (~fine).double()) > 0
            out[a:e, h] = torch.where(bad, math.nan, p @ clean)
            mag[a:e, h] = p @ clean.abs()
    return out, mag


def run_case(sizes, prefixes, lens, new, heads, kv, d, page, int8, seed=0, scale=None, padding=0, change=None, max_len=None, max_prefix=None):
    from conv_bn_silu_gb300 import tokens
    paged = refs.make_paged(list(lens) + list(prefixes), kv, d, page, int8, seed)
    if change is not None:
        change(paged, lens)
    table = paged["table"]
    own = table[:len(lens)].contiguous()
    pre = table[len(lens):].contiguous()
    starts, groups = starts_of(new), starts_of(sizes)
    group_of = [g for g, n in enumerate(sizes) for _ in range(n)]
    q = torch.randn((starts[-1] + padding, heads, d), generator=torch.Generator().manual_seed(seed + 1)).to(torch.bfloat16)
    dev = {n: None if t is None else t.cuda() for n, t in paged.items()}
    cache = tokens.PagedCache(dev["k"], dev["v"], dev["k_scale"], dev["v_scale"])
    attn = tokens.SharedPrefixAttention(cache, len(lens), len(sizes), max(max(new), 1), max_len or max(max(lens), 1),
                                        max(prefixes) if max_prefix is None else max_prefix, heads, scale=scale)
    if padding and starts[-1] + padding > attn.plan.max_total:
        padding = 0
        q = q[:starts[-1]]
    i32 = lambda v: torch.tensor(v, dtype=I32, device="cuda")
    args = (q.cuda(), i32(starts), i32(lens), own.cuda(), i32(groups), i32(prefixes), pre.cuda())
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    assert attn(*args, out=out) is out
    again = attn(*args)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    assert B.cbs_read_device_status(True, torch.cuda.current_stream().cuda_stream) == B.CBS_OK
    ref, mag = reference(q, paged, own, pre, group_of, starts, lens, prefixes, page, scale or d ** -0.5)
    got = out.double().cpu()
    nan = ref.isnan()
    assert torch.equal(~got.isfinite(), nan)
    bound = refs.attention_bound(ref, mag)
    err = (got - ref).abs()
    assert (err[~nan] <= bound[~nan]).all(), float((err / bound)[~nan].max())
    assert not got[starts[-1]:].any()   # padding is zeros
    return attn


@pytest.mark.gpu
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sizes,prefixes,lens", [
    ([1], [1], [1]), ([2], [16], [1, 2]), ([3], [400], [17, 1, 30]), ([1, 2, 1], [15, 33, 0], [5, 16, 31, 7]),
    ([8], [1000], [40] * 8), ([0, 2, 0, 3], [10, 200, 5, 100], [3, 300, 64, 1, 129]),
])
def test_single_tokens(sizes, prefixes, lens, d, int8):
    run_case(sizes, prefixes, lens, [1] * len(lens), 8, 2, d, 16, int8)


@pytest.mark.gpu
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("heads,kv,d,page", [(8, 8, 64, 16), (6, 1, 128, 64), (24, 4, 64, 32), (4, 2, 128, 256), (5, 5, 128, 16)])
def test_heads_and_pages(heads, kv, d, page, int8):
    run_case([3, 2], [300, 77], [60, 5, 100, 33, 260], [1] * 5, heads, kv, d, page, int8, padding=2)
    run_case([3, 2], [300, 77], [60, 5, 100, 33, 260], [20, 5, 0, 33, 100], heads, kv, d, page, int8, padding=3, seed=4)


@pytest.mark.gpu
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("new", [[2, 1, 3, 2], [40, 0, 1, 90], [0, 0, 0, 1], [128, 128, 128, 128]])
@pytest.mark.parametrize("prefixes", [[700, 129], [0, 2049]])
def test_chunks(new, prefixes, int8):
    run_case([1, 3], prefixes, [200, 150, 130, 400], new, 8, 2, 64, 16, int8)


@pytest.mark.gpu
@pytest.mark.parametrize("int8", [False, True])
def test_long_prefix_of_few(int8):
    """Ranges of a long prefix joined through the workspace, and in clusters."""
    attn = run_case([2], [20001], [9, 40], [1, 1], 4, 2, 64, 64, int8)
    assert attn.plan.prefix.split > 8 and attn.workspace_bytes > attn.plan.zeroed_bytes > 0
    run_case([30], [5003], [9 + i for i in range(30)], [1] * 30, 8, 1, 128, 64, int8)
    run_case([3], [40], [5001, 700, 12], [1, 1, 1], 4, 2, 64, 64, int8)


@pytest.mark.gpu
def test_longer_than_planned():
    run_case([2, 1], [900, 40], [300, 77, 500], [1, 1, 1], 8, 2, 64, 16, True, max_len=16, max_prefix=20)
    run_case([2, 1], [900, 40], [300, 77, 500], [30, 40, 5], 8, 2, 64, 16, False, max_len=16, max_prefix=20)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1e-4, 3.0, -0.2])
def test_scales(scale):
    """One part far above the other, and the reverse."""
    run_case([2, 2], [300, 200], [150, 3, 40, 90], [1, 3, 40, 1], 8, 2, 64, 16, False, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [[1, 1, 1], [50, 60, 70]])
def test_values_that_are_not_finite(new):
    """A NaN among one sequence's own values reaches it alone, and only tokens from it on."""
    def change(paged, lens):
        paged["v"][paged["table"][1, 0], 0, 3] = math.inf     # seen by all of sequence 1's tokens
        last = lens[2] - 1
        paged["v"][paged["table"][2, last // 16], 1, last % 16] = math.nan   # by its last token alone
    run_case([3], [100], [70, 80, 90], new, 4, 2, 64, 16, False, change=change)


@pytest.mark.gpu
def test_nothing_to_see():
    """No prefix and no own position that a token sees: zeros (a token past the sequence's length is reported)."""
    from conv_bn_silu_gb300 import tokens
    cache = tokens.PagedCache.empty(4, 2, 16, 64)
    for t in (cache.k, cache.v):
        t.zero_()
    for t in (cache.k_scale, cache.v_scale):
        t.fill_(float("nan"))
    i32 = lambda v: torch.tensor(v, dtype=I32, device="cuda")
    for new in (1, 70):
        attn = tokens.SharedPrefixAttention(cache, 1, 1, new, 16, 16, 4)
        out = attn(torch.ones((new, 4, 64), dtype=torch.bfloat16, device="cuda"), i32([0, new]), i32([0]), i32([[0]]), i32([0, 1]), i32([0]), i32([[1]]))
        assert not out.any()
        B.cbs_read_device_status(True, torch.cuda.current_stream().cuda_stream)


@pytest.mark.gpu
def test_bad_groups_and_pages():
    from conv_bn_silu_gb300 import tokens
    paged = refs.make_paged([20, 30, 40, 50], 2, 64, 16, True, 3)
    cache = tokens.PagedCache(*(paged[n].cuda() for n in ("k", "v", "k_scale", "v_scale")))
    i32 = lambda v: torch.tensor(v, dtype=I32, device="cuda")
    table = paged["table"].cuda()
    status = lambda: B.cbs_read_device_status(True, torch.cuda.current_stream().cuda_stream)
    for new in ([0, 1, 2, 3], [0, 20, 45, 60]):
        most = max(b - a for a, b in zip(new, new[1:]))
        attn = tokens.SharedPrefixAttention(cache, 3, 1, most, 50, 50, 8)
        q = torch.ones((new[-1], 8, 64), dtype=torch.bfloat16, device="cuda")
        call = lambda groups, lens, pre: attn(q, i32(new), i32([20, 30, 40]), table[:3].contiguous(), i32(groups), i32(lens), pre)
        call([0, 3], [50], table[3:].contiguous())
        assert status() == B.CBS_OK
        for groups in ([1, 3], [0, 2], [0, 4], [-1, 3], [3, 0], [0, 1 << 30]):
            call(groups, [50], table[3:].contiguous())
            assert status() == B.CBS_ERR_INVALID_ARG, groups
        for bad in (-1, 1 << 20):
            pre = table[3:].clone()
            pre[0, 1] = bad
            call([0, 3], [50], pre)
            assert status() == B.CBS_ERR_INVALID_ARG
        for length in (-1, 1 << 20):
            call([0, 3], [length], table[3:].contiguous())
            assert status() == B.CBS_ERR_INVALID_ARG
        with pytest.raises(B.CbsError):
            tokens.SharedPrefixAttention(cache, 3, 1, most, 50, 50, 8, max_group_new=most)(
                q, i32(new), i32([20, 30, 40]), table[:3].contiguous(), i32([0, 3]), i32([50]), table[3:].contiguous())


@pytest.mark.gpu
def test_streams_forks_and_graphs():
    from conv_bn_silu_gb300 import tokens
    lens, prefixes, new = [40, 50, 60], [3000], [1, 1, 1]
    paged = refs.make_paged(lens + prefixes, 2, 64, 16, True, 5)
    cache = tokens.PagedCache(*(paged[n].cuda() for n in ("k", "v", "k_scale", "v_scale")))
    i32 = lambda v: torch.tensor(v, dtype=I32, device="cuda")
    table = paged["table"].cuda()
    q = torch.randn((3, 3, 8, 64), device="cuda", generator=torch.Generator("cuda").manual_seed(6)).to(torch.bfloat16)
    rest = (i32([0, 1, 2, 3]), i32(lens), table[:3].contiguous(), i32([0, 3]), i32(prefixes), table[3:].contiguous())
    attn = tokens.SharedPrefixAttention(cache, 3, 1, 1, 60, 3000, 8)
    want = [attn(x, *rest) for x in q]
    streams, forks = [torch.cuda.Stream() for _ in q], [attn.fork() for _ in q]
    got = [[] for _ in q]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, (s, f) in enumerate(zip(streams, forks)):
            with torch.cuda.stream(s):
                got[i].append(f(q[i], *rest))
    torch.cuda.synchronize()
    assert all(torch.equal(want[i], o) for i in range(3) for o in got[i])
    graph = torch.cuda.CUDAGraph()
    held = q[0].clone()
    with torch.cuda.graph(graph):
        out = attn(held, *rest)
    for i in (2, 1, 0):
        held.copy_(q[i])
        graph.replay()
        assert torch.equal(out, want[i])
    # a slice of a fused product's rows, to a slice of another
    rows = torch.zeros((3, 14, 64), dtype=torch.bfloat16, device="cuda")
    rows[:, 4:12] = q[1]
    wide = torch.full((3, 20, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    attn(rows[:, 4:12], *rest, out=wide[:, 2:10])
    assert torch.equal(wide[:, 2:10], want[1]) and (wide[:, :2] == 9).all() and (wide[:, 10:] == 9).all()


def desc(**kw):
    d = dict(batch=4, groups=2, max_new=3, max_group_new=6, max_len=64, max_prefix=256, heads=4, kv_heads=2, head_dim=64,
             cache_prec=B.CBS_INT8, num_sms=0)
    d.update(kw)
    return B.cbs_shared_desc(*[d[n] for n, _ in B.cbs_shared_desc._fields_])


@pytest.mark.parametrize("status,kw", [
    (I, dict(batch=-1)), (I, dict(groups=-1)), (I, dict(max_new=-1)), (I, dict(max_group_new=-1)), (I, dict(max_len=-1)),
    (I, dict(max_prefix=-1)), (I, dict(heads=3)), (U, dict(head_dim=96)), (I, dict(cache_prec=B.CBS_FP32)), (U, dict(groups=70000)),
])
def test_plans_refused(cuda_lib, status, kw):
    refused(status, B.cbs_shared_plan, desc(**kw))


def test_calls_refused(cuda_lib):
    plan = B.cbs_shared_plan(desc())
    assert plan.max_total == 12 and plan.size == ctypes.sizeof(plan)
    assert plan.workspace_bytes >= plan.zeroed_bytes + 12 * 4 * (64 * 4 + 8)
    def pre(**kw):
        d = dict(group_start=OK, prefix_lens=OK, page_table=OK, groups=2, max_pages=4)
        d.update(kw)
        return B.cbs_prefixes(*[d[n] for n, _ in B.cbs_prefixes._fields_])
    def call(p=plan, c=None, s=None, x=None, q=OK, qs=256, scale=0.1, out=2 * OK, os=256, ws=4 * OK, wb=None):
        B.cbs_shared_attention(p, c or c_cache(), s or seqs(batch=4), x or pre(), q, qs, scale, out, os, ws,
                               plan.workspace_bytes if wb is None else wb, None)
    refused(I, lambda: call(q=None))
    refused(M, lambda: call(q=OK + 8))
    refused(I, lambda: call(out=OK + 16))
    refused(I, lambda: call(scale=float("inf")))
    refused(W, lambda: call(ws=None))
    refused(W, lambda: call(wb=plan.workspace_bytes - 1))
    refused(P, lambda: call(c=c_cache(kv_heads=4)))
    refused(P, lambda: call(s=seqs(batch=3)))
    refused(P, lambda: call(x=pre(groups=3)))
    refused(I, lambda: call(s=seqs(batch=4, total=13)))
    refused(I, lambda: call(x=pre(group_start=None)))
    refused(M, lambda: call(x=pre(group_start=OK + 2)))
    refused(I, lambda: call(x=pre(prefix_lens=None)))
    refused(I, lambda: call(x=pre(page_table=None)))
    refused(I, lambda: call(x=pre(max_pages=-1)))
    other = B.cbs_shared_plan_t.from_buffer_copy(plan)
    other.size = 8
    refused(P, lambda: call(p=other))
    call(s=seqs(batch=4, total=0))


def test_python_refusals():
    from tests.test_tokens_devices import fake
    from conv_bn_silu_gb300 import tokens
    plan = B.cbs_shared_plan(desc(batch=1, groups=1))
    cache = B.cbs_cache(None, None, None, None, B.CBS_INT8, 4, 16, 2, 64)
    bf = torch.bfloat16
    kinds = [((3, 4, 64), bf), ((3, 4, 64), bf), ((2,), I32), ((1,), I32), ((1, 4), I32), ((2,), I32), ((1,), I32), ((1, 4), I32)]
    def call(made):
        q, out, starts, lens, table, *groups = made
        tokens._calls().shared_attention(ctypes.addressof(plan), ctypes.addressof(cache), 0, q, starts, lens, table, 0.1, out, None, 0, *groups)
    for wrong in range(8):
        with pytest.raises(ValueError, match="device"):
            call([fake(s, t, int(i == wrong)) for i, (s, t) in enumerate(kinds)])
    for i, other in ((5, ((3,), I32)), (6, ((2,), I32)), (7, ((1, 4), torch.int64)), (7, ((4,), I32)), (0, ((3, 4, 32), bf))):
        some = list(kinds)
        some[i] = other
        with pytest.raises(ValueError):
            call([fake(s, t) for s, t in some])
