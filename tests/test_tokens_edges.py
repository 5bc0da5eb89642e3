"""GPU checks of the token operators at the edges of their contracts: values
that are not finite or near the float range's ends, tokens of no sequence,
lengths a table cannot hold, pages behind a window."""
import math

import pytest
import torch

from conv_bn_silu_gb300 import _binding as B
from conv_bn_silu_gb300 import tokens
from tests import token_refs as refs

pytestmark = pytest.mark.gpu

U = 2.0 ** -24    # rounding to float moves a value by at most this share of it
UB = 2.0 ** -8    # to bfloat16 (eight significant bits)


@pytest.fixture(scope="module", autouse=True)
def token_calls(cuda_lib):
    from conv_bn_silu_gb300 import build
    build.build_tokens()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def status(reset=True):
    return B.cbs_read_device_status(reset, torch.cuda.current_stream().cuda_stream)


def on_gpu(paged):
    return {n: None if t is None else t.cuda() for n, t in paged.items()}


# ------------------------------------------------------------------ RMS norm
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("cols", [5, 64, 333, 4096, 6001, 16384])
def test_rmsnorm_8_bits_shows_what_is_not_finite(cuda_lib, cols, residual, dtype):
    """A row whose sum or whose product with the weights holds a NaN or an
    infinity reads back as NaN, whatever stands beside it; the others do not."""
    g = gen(cols)
    x = torch.randn((5, cols), generator=g).to(dtype)
    r = torch.zeros_like(x).cuda() if residual else None
    w = torch.rand(cols, generator=g) + 0.5
    at = cols - 3
    w[at] = 0
    x[1, at], x[2, at], x[3, 0] = math.inf, math.nan, -math.inf
    q = tokens.rmsnorm(x.cuda(), w.cuda(), 1e-5, residual=r, int8=True)
    assert q.scale.isnan().tolist() == [False, True, True, True, False]
    back = tokens.dequantize_rows(q.y, q.scale, torch.float32)
    assert back[1:4].isnan().all() and back[0].isfinite().all() and back[4].isfinite().all()
    for kind in (math.nan, math.inf):
        w[at] = kind
        q = tokens.rmsnorm(x[:1].cuda(), w.cuda(), 1e-5, residual=None if r is None else r[:1], int8=True)
        assert q.scale.isnan().all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", [7, 64, 1000, 4096, 6001, 8192, 32768])
def test_rmsnorm_rows_whose_squares_pass_the_float_range(cuda_lib, cols, dtype):
    """Finite rows of any size have finite answers.  The bound is that of rows
    of ordinary size: moving a value by a power of two is exact."""
    g = gen(cols + 1)
    x = torch.randn((7, cols), generator=g)
    x[0] *= 1e20
    x[1, cols // 2] = 3e38
    x[2] = 3e38
    x[3, : cols // 2 + 1] *= 1e18    # squares within the range, their sum perhaps not
    x[4, -1] = -1e25
    x[5] *= 2.0 ** 62
    x = x.to(dtype)
    w = torch.rand(cols, generator=g) * 0.5 + 0.5
    h = x.float()
    root = (h.double().square().mean(1, keepdim=True) + 1e-5).sqrt()
    ref = h.double() * w.double() / root
    y = tokens.rmsnorm(x.cuda(), w.cuda(), 1e-5).y.double().cpu()
    bound = ref.abs() * (40 * U + (UB if dtype == torch.bfloat16 else 0)) + 1e-37
    assert ((y - ref).abs() <= bound).all()
    q = tokens.rmsnorm(x.cuda(), w.cuda(), 1e-5, int8=True)
    codes, s = refs.quantise_rows(h * w)
    assert torch.equal(q.y.cpu(), codes)
    want = s.double() / root[:, 0]
    assert ((q.scale.double().cpu() - want).abs() <= want * 40 * U).all()


@pytest.mark.parametrize("kind", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantised_weights_show_what_is_not_finite(cuda_lib, group, kind):
    """An output that such a weight is part of is NaN; the others are as without it."""
    w = torch.randn((40, 4 * group), generator=gen(10))
    x = torch.randn((12, 4 * group), generator=gen(11)).to(torch.bfloat16).cuda()
    clean = tokens.LinearW4.quantize(w.cuda(), group)(x, dtype=torch.float32)
    w[7, group + 3] = kind
    layer = tokens.LinearW4.quantize(w.cuda(), group)
    codes, scale = torch.randint(-127, 128, x.shape, generator=gen(12), dtype=torch.int8).cuda(), torch.ones(12, device="cuda")
    for out in (layer(x, dtype=torch.float32), layer(x[:3], dtype=torch.float32), layer(codes, scale), layer(codes[:3], scale[:3])):
        assert out[:, 7].isnan().all() and int(out.isnan().sum()) == out.shape[0]
    keep = torch.arange(40) != 7
    assert torch.equal(layer(x, dtype=torch.float32)[:, keep], clean[:, keep])


# ------------------------------------------------- tokens of no sequence
KERNELS = [B.CBS_ATTN_ROWS, B.CBS_ATTN_CHUNK, B.CBS_ATTN_CLUSTER]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("d,new,split", [(64, [1, 0, 1], 1), (128, [3, 20, 0], 3), (64, [70, 5, 0], 2)])
def test_tokens_behind_the_last_sequence_are_padding(cuda_lib, d, new, split, kernel, int8):
    """A call of a fixed number of tokens with fewer real ones: the rest are
    zeros from attention and left out by the cache, and nothing is reported."""
    lens, heads, kv, page, pad = [100, 33, 300], 6, 2, 16, 37
    paged = refs.make_paged(lens, kv, d, page, int8, 31)
    dev = on_gpu(paged)
    starts = [sum(new[:i]) for i in range(4)]
    q = torch.randn((starts[-1] + pad, heads, d), generator=gen(3)).to(torch.bfloat16)
    cache = tokens.PagedCache(dev["k"], dev["v"], dev["k_scale"], dev["v_scale"])
    attn = tokens.PagedAttention(cache, 3, max(new), 300, heads, force_kernel=kernel, force_split=split)
    wide = torch.full((starts[-1] + pad, heads + 1, d), 7.0, dtype=torch.bfloat16, device="cuda")
    attn(q.cuda(), i32(starts), i32(lens), dev["table"], out=wide[:, 1:])
    assert status() == B.CBS_OK
    got = wide.double().cpu()
    ref, mag = refs.attention(q[:starts[-1]], paged, starts, lens, page, True, 0, d ** -0.5)
    assert ((got[:starts[-1], 1:] - ref).abs() <= refs.attention_bound(ref, mag)).all()
    assert (got[starts[-1]:, 1:] == 0).all() and (got[:, 0] == 7).all()

    before = {n: None if t is None else t.clone() for n, t in dev.items()}
    rows = torch.randn((starts[-1] + pad, kv, d), generator=gen(4)).to(torch.bfloat16).cuda()
    cache.write(rows, rows, i32(starts), i32(lens), dev["table"])
    assert status() == B.CBS_OK
    changed = (dev["k"].view(torch.uint8) != before["k"].view(torch.uint8)).flatten(3).any(-1).cpu()
    may = torch.zeros_like(changed)
    for b, n in enumerate(lens):
        for pos in range(n - new[b], n):
            may[paged["table"][b, pos // page], :, pos % page] = True
    assert torch.equal(changed, may)


@pytest.mark.parametrize("int8", [False, True])
def test_a_call_of_padding_alone(cuda_lib, int8):
    cache = tokens.PagedCache.empty(4, 2, 16, 64, dtype=torch.int8 if int8 else torch.bfloat16)
    q = torch.randn((5, 4, 64), device="cuda").to(torch.bfloat16)
    for lens, table in (([3, 0], [[1], [0]]), ([], torch.zeros((0, 1), dtype=torch.int32))):
        starts, table = i32([0] * (len(lens) + 1)), torch.as_tensor(table, dtype=torch.int32, device="cuda")
        out = torch.full((5, 5, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        tokens.PagedAttention(cache, len(lens), 1, 16, 4)(q, starts, i32(lens), table, out=out[:, :4])
        assert (out[:, :4] == 0).all() and (out[:, 4] == 7).all()
        cache.write(q[:, :2], q[:, 2:], starts, i32(lens), table)
        assert status() == B.CBS_OK


@pytest.mark.parametrize("new", [1, 40])
def test_tokens_before_the_first_sequence_are_reported(cuda_lib, new):
    cache = tokens.PagedCache.empty(8, 2, 16, 64)
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        t.fill_(1)
    q = torch.randn((new + 1, 4, 64), device="cuda").to(torch.bfloat16)
    args = i32([1, new + 1]), i32([100]), torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8)
    tokens.PagedAttention(cache, 1, new, 100, 4)(q, *args)
    assert status() == B.CBS_ERR_INVALID_ARG
    cache.write(q[:, :2], q[:, 2:], *args)
    assert status() == B.CBS_ERR_INVALID_ARG


# ----------------------------------------------- what a table does not hold
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_writes_past_the_table_change_nothing_else(cuda_lib, d, int8):
    """A length its table cannot hold: the tokens that have a page are written
    to it, the others are left out and reported."""
    cache = tokens.PagedCache.empty(3, 2, 16, d, dtype=torch.int8 if int8 else torch.bfloat16)
    table = i32([[2, 0]])
    x = torch.randn((5, 2, d), device="cuda")
    for new, length, slots in ((1, 33, []), (5, 34, [29, 30, 31]), (2, 1000, []), (3, -2, [])):
        for t in (cache.k, cache.v) + ((cache.k_scale, cache.v_scale) if int8 else ()):
            t.fill_(1)
        cache.write(x[:new], x[:new], i32([0, new]), i32([length]), table)
        assert status() == B.CBS_ERR_INVALID_ARG
        for t in (cache.k, cache.v):
            changed = (t != 1).any(-1).cpu()
            may = torch.zeros_like(changed)
            for pos in slots:
                may[(2, 0)[pos // 16], :, pos % 16] = True
            assert torch.equal(changed, may), (new, length)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("page,window,new,split", [(16, 20, 1, 1), (16, 100, 5, 2), (32, 200, 130, 1), (64, 64, 40, 3), (256, 1, 2, 1)])
def test_pages_behind_the_window_may_be_gone(cuda_lib, page, window, new, split, kernel, int8):
    """Table entries of pages wholly before every new token's window are not
    looked at: a program may have released them."""
    lens, heads, kv, d = [700, 333], 4, 2, 64
    paged = refs.make_paged(lens, kv, d, page, int8, 33)
    starts = [0, new, 2 * new]
    q = torch.randn((2 * new, heads, d), generator=gen(5)).to(torch.bfloat16)
    ref, mag = refs.attention(q, paged, starts, lens, page, True, window, d ** -0.5)
    table = paged["table"].clone()
    for b, n in enumerate(lens):
        first = max(n - new - window + 1, 0)
        table[b, : first // page] = -1
    dev = on_gpu(paged)
    attn = tokens.PagedAttention(tokens.PagedCache(dev["k"], dev["v"], dev["k_scale"], dev["v_scale"]), 2, new, 700, heads,
                                 window=window, force_kernel=kernel, force_split=split)
    got = attn(q.cuda(), i32(starts), i32(lens), table.cuda()).double().cpu()
    assert status() == B.CBS_OK
    assert ((got - ref).abs() <= refs.attention_bound(ref, mag)).all()


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("kernel", KERNELS)
def test_a_window_as_large_as_an_int(cuda_lib, kernel, int8):
    """It hides nothing, from tokens before a sequence's start either."""
    from tests.test_tokens_attention import run_case
    for causal in (True, False):
        run_case([3, 100], [6, 2], 4, 2, 64, 16, int8, causal=causal, window=2 ** 31 - 1, kernel=kernel)


# -------------------------------------------------- attention's number range
@pytest.mark.parametrize("kernel,size", [(k, 1e-36) for k in KERNELS] + [(k, 1e33) for k in KERNELS] +
                         [(B.CBS_ATTN_ROWS, 1e36), (B.CBS_ATTN_CLUSTER, 1e36)])
@pytest.mark.parametrize("d", [64, 128])
def test_queries_of_any_size_over_an_8_bit_cache(cuda_lib, d, kernel, size):
    """Queries near the float range's ends with keys that bring the scores back
    to ordinary size: the same bound as at ordinary sizes.  (Up to 2^112, beyond
    which sums of queries times codes may pass the range; the kernel of few rows
    moves the queries by a power of two first.)"""
    from tests.test_tokens_attention import run_case
    paged = refs.make_paged([200, 77], 2, d, 16, True, 35)
    paged["k_scale"] = paged["k_scale"] / size
    q = (torch.randn((3, 4, d), generator=gen(6)) * size).to(torch.bfloat16)
    run_case([200, 77], [2, 1], 4, 2, d, 16, True, q=q, paged=paged, kernel=kernel)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("split", [1, 3])
@pytest.mark.parametrize("size", [1e3, 1e5, 1e8])
def test_scores_far_from_zero(cuda_lib, size, split, kernel, int8):
    """Scores so large that a float's last place is worth many powers of two:
    the largest takes all (equal ones share).  Keys are whole multiples of one
    vector, so scores are either equal or apart by 1/127 of the largest."""
    from tests.test_tokens_attention import run_case
    n, d, page, new = 500, 64, 16, 40
    paged = refs.make_paged([n], 1, d, page, int8, 36)
    g = torch.randint(-127, 128, (n,), generator=gen(7))
    for pos in range(n):
        p, slot = paged["table"][0, pos // page], pos % page
        if int8:
            paged["k"][p, 0, slot], paged["k_scale"][p, 0, slot] = g[pos].to(torch.int8), size
        else:
            paged["k"][p, 0, slot] = (g[pos] * torch.ones(d)).to(torch.bfloat16) * size
    q = torch.ones((new, 4, d)) * size
    q[:, 1] *= -1
    q[::2, 2] *= -0.25
    q[:, 3] = 0
    run_case([n], [new], 4, 1, d, page, int8, q=q.to(torch.bfloat16), paged=paged, kernel=kernel, split=split)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("split", [1, 3])
def test_equal_values_come_back(cuda_lib, split, d, kernel):
    """An average of equal values is that value, however the probabilities were
    rounded: the sum that divides is of the rounded ones.  Sixty keys carry 93% to
    99% of the weight, at probabilities of 2^4 to 2^7.9 (the running maximum is not
    raised for them).  Sums of 900 products in float are within 2^-13 of
    themselves, far less than half a place of bfloat16."""
    n, page, heads, new = 900, 16, 4, 60
    paged = refs.make_paged([n], 1, d, page, False, 37)
    value = torch.tensor(255 / 128, dtype=torch.bfloat16)
    for side, x in (("k", 0.0), ("v", value)):
        paged[side][~paged[side].isnan()] = x
    for pos in range(n - 60, n):
        paged["k"][paged["table"][0, pos // page], 0, pos % page] = 1.0
    rows = torch.linspace(4, 7.9, new * heads) * math.log(2)
    q = rows.view(new, heads, 1).expand(new, heads, d).to(torch.bfloat16)
    dev = on_gpu(paged)
    attn = tokens.PagedAttention(tokens.PagedCache(dev["k"], dev["v"]), 1, new, n, heads, causal=False, scale=1 / d,
                                 force_kernel=kernel, force_split=split)
    out = attn(q.cuda().contiguous(), i32([0, new]), i32([n]), dev["table"])
    assert (out == value.cuda()).all()


# ------------------------------------------------------- calls from Python
def test_errors_of_the_calls(cuda_lib):
    """An output that does not fit memory raises what an allocation raises;
    a flag that has no truth value raises its own error."""
    cache = tokens.PagedCache.empty(4, 2, 16, 64)
    with pytest.raises(torch.OutOfMemoryError):
        cache.read(i32([3]), i32([[0]]), 2 ** 31 - 1)
    x = torch.zeros((2, 8), device="cuda")
    with pytest.raises(RuntimeError, match="ambiguous"):
        tokens.rmsnorm(x, torch.ones(8, device="cuda"), 1e-5, int8=torch.ones(2))
    k, _ = cache.read(i32([0]), i32([[0]]), 3)
    assert (k == 0).all() and status() == B.CBS_OK


def test_a_workspace_is_ready_for_any_stream(cuda_lib):
    """Made while its stream is busy, used at once on another one, and dropped
    while that one is: the counters are zero, and the memory is not given away
    before the call has ended."""
    paged = refs.make_paged([1000], 2, 64, 16, False, 41)
    dev = on_gpu(paged)
    cache = tokens.PagedCache(dev["k"], dev["v"])
    q = torch.randn((1, 4, 64), generator=gen(9)).to(torch.bfloat16)
    args = q.cuda(), i32([0, 1]), i32([1000]), dev["table"]
    ref, mag = refs.attention(q, paged, [0, 1], [1000], 16, True, 0, 64 ** -0.5)
    make = lambda: tokens.PagedAttention(cache, 1, 1, 1000, 4, force_kernel=B.CBS_ATTN_ROWS, force_split=7)
    size = make().workspace_bytes
    side, outs = torch.cuda.Stream(), []
    for _ in range(3):
        junk = torch.full((size,), 255, dtype=torch.uint8, device="cuda")   # what the allocator hands out next
        del junk
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)   # ten milliseconds or so
        attn = make()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
            outs.append(attn(*args))
        del attn
        again = torch.full((size,), 255, dtype=torch.uint8, device="cuda")   # on the first stream, at once
        del again
    torch.cuda.synchronize()
    for out in outs:
        assert ((out.double().cpu() - ref).abs() <= refs.attention_bound(ref, mag)).all()
    assert status() == B.CBS_OK


def test_outputs_beside_their_inputs(cuda_lib):
    """Slices of one tensor that share its rows but no element, and what may be
    written in place."""
    paged = refs.make_paged([90, 33], 2, 64, 16, False, 43)
    dev = on_gpu(paged)
    cache = tokens.PagedCache(dev["k"], dev["v"])
    rows = torch.randn((12, 10, 64), generator=gen(13)).to(torch.bfloat16)
    d = rows.cuda()
    for new in ([10, 2], [1, 1]):
        n = sum(new)
        starts = [0, new[0], n]
        attn = tokens.PagedAttention(cache, 2, new[0], 90, 4)
        out = attn(d[:n, :4], i32(starts), i32([90, 33]), dev["table"], out=d[:n, 4:8])
        ref, mag = refs.attention(rows[:n, :4], paged, starts, [90, 33], 16, True, 0, 64 ** -0.5)
        assert ((out.double().cpu() - ref).abs() <= refs.attention_bound(ref, mag)).all()
        with pytest.raises(B.CbsError, match="lies on q"):
            attn(d[:n, :4], i32(starts), i32([90, 33]), dev["table"], out=d[:n, 2:6])
    layer = tokens.LinearW4.quantize(torch.randn((64, 64), device="cuda"), 64)
    x = torch.randn((5, 64), generator=gen(14)).to(torch.bfloat16).cuda()
    with pytest.raises(B.CbsError, match="lies on an input"):
        layer(x, out=x)
    assert status() == B.CBS_OK
