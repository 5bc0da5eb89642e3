"""GPU checks of attention over a paged cache against a plain 64-bit form."""
import math

import pytest
import torch

from conv_bn_silu_gb300 import _binding as B
from conv_bn_silu_gb300 import tokens
from tests import token_refs as refs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def token_calls(cuda_lib):
    from conv_bn_silu_gb300 import build
    build.build_tokens()



def starts_of(new):
    return [sum(new[:i]) for i in range(len(new) + 1)]


def run_case(lens, new, heads, kv, d, page, int8, causal=True, window=0, scale=None, seed=0, kernel=-1, split=0,
             q=None, paged=None, max_new=None, max_len=None):
    paged = paged or refs.make_paged(lens, kv, d, page, int8, seed)
    starts = starts_of(new)
    if q is None:
        g = torch.Generator().manual_seed(seed + 1)
        q = torch.randn((starts[-1], heads, d), generator=g).to(torch.bfloat16)
    dev = {n: None if t is None else t.cuda() for n, t in paged.items()}
    cache = tokens.PagedCache(dev["k"], dev["v"], dev["k_scale"], dev["v_scale"])
    attn = tokens.PagedAttention(cache, len(lens), max_new or max(max(new), 1), max_len or max(max(lens), 1), heads,
                                 causal=causal, window=window, scale=scale, force_kernel=kernel, force_split=split)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    args = (q.cuda(), i32(starts), i32(lens), dev["table"])
    out = torch.full((starts[-1], heads, d), 7.0, dtype=torch.bfloat16, device="cuda")
    attn(*args, out=out)
    again = attn(*args)   # the workspace is ready for the next call, and the answer is the same bits
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    assert B.cbs_read_device_status(True, torch.cuda.current_stream().cuda_stream) == B.CBS_OK
    ref, mag = refs.attention(q, paged, starts, lens, page, causal, window, scale or d ** -0.5)
    got = out.double().cpu()
    nan = ref.isnan()
    assert torch.equal(~got.isfinite(), nan), "a value that is not finite is not where it belongs"
    err = (got - ref).abs()[~nan]
    bound = refs.attention_bound(ref, mag)[~nan]
    assert (err <= bound).all(), (float((err / bound).max()), attn.plan.kernel, attn.plan.split)
    return got, attn


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[1], [2], [15], [16], [17], [63, 1, 300], [1000], [513, 0, 16, 31]])
def test_single_tokens(cuda_lib, lens, d, int8):
    run_case(lens, [min(1, n) for n in lens], 8, 2, d, 16, int8)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("heads,kv", [(1, 1), (6, 6), (8, 1), (12, 4), (24, 2), (35, 5)])
def test_head_layouts(cuda_lib, heads, kv, int8):
    run_case([129, 70], [1, 3], heads, kv, 64, 32, int8)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_page_sizes(cuda_lib, page, int8):
    run_case([300, 511, 257, 1], [5, 1, 40, 1], 8, 4, 128, page, int8)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens,new", [([40], [40]), ([130, 250], [130, 7]), ([700], [333]), ([64, 64, 64], [64, 0, 1]),
                                      ([1025], [129]), ([257], [256])])
def test_chunks(cuda_lib, lens, new, causal, int8):
    run_case(lens, new, 12, 4, 64, 16, int8, causal=causal)
    run_case(lens, new, 4, 4, 128, 64, int8, causal=causal)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("kernel", [B.CBS_ATTN_ROWS, B.CBS_ATTN_CHUNK])
@pytest.mark.parametrize("d,page", [(64, 16), (64, 256), (128, 32), (128, 128)])
def test_both_kernels(cuda_lib, d, page, kernel, int8):
    """The kernels hold over the same calls, whichever the plan would take."""
    kw = dict(d=d, page=page, int8=int8, kernel=kernel)
    run_case([1], [1], 2, 1, **kw)
    run_case([127, 128, 129, 0], [1, 128, 50, 0], 4, 2, **kw)
    run_case([640], [129], 6, 2, **kw)
    run_case([640], [129], 6, 2, causal=False, split=3, **kw)
    run_case([1300, 700], [70, 300], 8, 2, window=200, split=2, **kw)
    run_case([3, 0, 5], [6, 2, 1], 4, 2, **kw)
    run_case([900], [64], 35, 5, split=5, scale=0.3, **kw)


@pytest.mark.parametrize("kernel", [B.CBS_ATTN_ROWS, B.CBS_ATTN_CHUNK])
def test_scores_that_grow_along_the_keys(cuda_lib, kernel):
    """The running maximum moves at every tile, by much."""
    n, d, page, new = 700, 64, 16, 40
    paged = refs.make_paged([n], 1, d, page, False, 6)
    grow = torch.linspace(-8, 8, n)
    for pos in range(n):
        paged["k"][paged["table"][0, pos // page], 0, pos % page] = (grow[pos] * torch.ones(d)).to(torch.bfloat16)
    q = (torch.ones((new, 4, d)) * torch.linspace(-4, 4, new)[:, None, None]).to(torch.bfloat16)
    for split in (1, 3):
        run_case([n], [new], 4, 1, d, page, False, q=q, paged=paged, split=split, kernel=kernel)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("window", [1, 2, 16, 100, 5000])
def test_windows(cuda_lib, window, int8):
    run_case([400, 77], [150, 1], 8, 2, 64, 32, int8, window=window)
    run_case([400, 77], [3, 77], 8, 2, 128, 16, int8, window=window, causal=False)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("split", [1, 2, 3, 7, 40])
def test_splits(cuda_lib, split, int8):
    run_case([900, 33, 0, 500], [1, 1, 0, 2], 16, 2, 128, 16, int8, split=split)
    run_case([900, 260], [200, 260], 8, 2, 64, 64, int8, split=split)


@pytest.mark.parametrize("int8", [False, True])
def test_rows_that_see_nothing(cuda_lib, int8):
    """More new tokens than the sequence holds: those before its start see no
    key; an empty sequence's tokens neither.  Their outputs are zeros."""
    for causal in (True, False):
        got, _ = run_case([3, 0, 5], [6, 2, 1], 4, 2, 64, 16, int8, causal=causal)
        if causal:
            assert (got[:3] == 0).all()
        assert (got[6:8] == 0).all()


@pytest.mark.parametrize("kind", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("new", [2, 30, 200])
def test_hidden_keys_and_values_reach_nobody(cuda_lib, kind, new):
    """A key and a value that are not finite, at a place that only later
    tokens see: earlier tokens of the chunk are as if it were not there."""
    n, page = 260, 16
    for side in ("v", "k"):
        paged = refs.make_paged([n], 2, 64, page, False, 3)
        pos = n - new // 2 - 1          # in the middle of the chunk
        p, slot = paged["table"][0, pos // page], pos % page
        paged[side][p, 1, slot, 5] = kind
        q = torch.randn((new, 4, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
        place = torch.arange(n - new, n)
        dev = {k: None if t is None else t.cuda() for k, t in paged.items()}
        cache = tokens.PagedCache(dev["k"], dev["v"])
        attn = tokens.PagedAttention(cache, 1, new, n, 4)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
        out = attn(q.cuda(), i32([0, new]), i32([n]), dev["table"]).double().cpu()
        clean = {k: t for k, t in paged.items()}
        clean[side] = paged[side].clone()
        clean[side][p, 1, slot, 5] = 0.0
        ref, mag = refs.attention(q, clean, [0, new], [n], page, True, 0, 64 ** -0.5)
        blind = place < pos
        ok = (out - ref).abs() <= refs.attention_bound(ref, mag)
        assert ok[blind].all() and ok[:, :2].all()      # earlier tokens; the other key head
        if side == "v":
            assert not out[~blind][:, 2:, 5].isfinite().any()
            rest = torch.ones(64, dtype=torch.bool)
            rest[5] = False
            assert ok[:, :, rest].all()
        elif math.isnan(kind):
            assert out[~blind][:, 2:].isnan().all()


def test_large_scores_and_long_tails(cuda_lib):
    """Scores that grow along the keys (the running maximum moves often) and
    scores far apart (most probabilities vanish)."""
    n, d, page = 600, 64, 16
    paged = refs.make_paged([n], 1, d, page, False, 5)
    grow = torch.linspace(-6, 6, n)
    for pos in range(n):
        paged["k"][paged["table"][0, pos // page], 0, pos % page] = (grow[pos] * torch.ones(d)).to(torch.bfloat16)
    q = torch.ones((3, 2, d)).to(torch.bfloat16)
    q[1] *= -1
    q[2] *= 4
    for split in (1, 4):
        run_case([n], [3], 2, 1, d, page, False, q=q, paged=paged, split=split)


@pytest.mark.parametrize("int8", [False, True])
def test_slices_and_other_streams(cuda_lib, int8):
    """q as a slice of a fused product's rows, the output as a slice, on a
    stream of its own."""
    lens, new, kv, heads, d, page = [200, 90], [5, 20], 2, 6, 64, 16
    paged = refs.make_paged(lens, kv, d, page, int8, 9)
    dev = {k: None if t is None else t.cuda() for k, t in paged.items()}
    cache = tokens.PagedCache(dev["k"], dev["v"], dev["k_scale"], dev["v_scale"])
    attn = tokens.PagedAttention(cache, 2, 20, 200, heads)
    qkv = torch.randn((25, heads + 2 * kv, d), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    dq = qkv.cuda()
    wide = torch.zeros((25, heads + 3, d), dtype=torch.bfloat16, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    st, ln = i32([0, 5, 25]), i32(lens)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        attn.fork()(dq[:, :heads], st, ln, dev["table"], out=wide[:, 3:])
    side.synchronize()
    ref, mag = refs.attention(qkv[:, :heads], paged, [0, 5, 25], lens, page, True, 0, d ** -0.5)
    got = wide.double().cpu()
    assert ((got[:, 3:] - ref).abs() <= refs.attention_bound(ref, mag)).all()
    assert (got[:, :3] == 0).all()


def test_graph_replay_with_longer_sequences(cuda_lib):
    """A captured call serves other lengths: they are read on the device."""
    lens, d, page = [100, 900], 128, 16
    paged = refs.make_paged([1000, 1000], 2, d, page, False, 11, junk=False)
    dev = {k: None if t is None else t.cuda() for k, t in paged.items()}
    cache = tokens.PagedCache(dev["k"], dev["v"])
    attn = tokens.PagedAttention(cache, 2, 1, 1000, 8)
    q = torch.randn((2, 8, d), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    dq, st = q.cuda(), torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = attn(dq, st, ln, dev["table"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn(dq, st, ln, dev["table"], out=out)
    for lens in ([1, 1000], [777, 16]):
        ln.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        ref, mag = refs.attention(q, paged, [0, 1, 2], lens, page, True, 0, d ** -0.5)
        assert ((out.double().cpu() - ref).abs() <= refs.attention_bound(ref, mag)).all()


def test_places_out_of_range_are_reported(cuda_lib):
    """A page outside the pool is left out and reported; the other sequence's
    tokens are right; so is a length its table cannot hold."""
    lens, d, page = [80, 50], 64, 16
    paged = refs.make_paged(lens, 2, d, page, False, 13)
    dev = {k: None if t is None else t.cuda() for k, t in paged.items()}
    cache = tokens.PagedCache(dev["k"], dev["v"])
    attn = tokens.PagedAttention(cache, 2, 1, 80, 4)
    q = torch.randn((2, 4, d), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    table = dev["table"].clone()
    table[0, 1] = paged["k"].shape[0] + 5
    out = attn(q.cuda(), i32([0, 1, 2]), i32(lens), table).double().cpu()
    assert B.cbs_read_device_status(True, stream) == B.CBS_ERR_INVALID_ARG
    assert B.cbs_read_device_status(False, stream) == B.CBS_OK
    ref, mag = refs.attention(q, paged, [0, 1, 2], lens, page, True, 0, d ** -0.5)
    assert ((out[1] - ref[1]).abs() <= refs.attention_bound(ref, mag)[1]).all()
    attn(q.cuda(), i32([0, 1, 2]), i32([10 ** 6, 50]), dev["table"])
    assert B.cbs_read_device_status(True, stream) == B.CBS_ERR_INVALID_ARG
    attn(q.cuda(), i32([0, 1, 5]), i32(lens), dev["table"])
    assert B.cbs_read_device_status(True, stream) == B.CBS_ERR_INVALID_ARG
