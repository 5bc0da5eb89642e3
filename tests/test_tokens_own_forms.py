"""Shared prefixes: the sequences' own part by each kernel and in each of its forms.  A part
of more CTAs than the GPU holds at once runs beside the prefixes' and leaves its shares for a
join; a smaller one waits for the prefixes' shares and joins them itself.  The sizes here are
far from the border between both, whatever the prefixes take."""
import pytest
import torch

from conv_bn_silu_gb300 import _binding as B
from tests import token_refs as refs
from tests.test_tokens_shared import run_case, starts_of

I32 = torch.int32
ROWS, CHUNK, CLUSTER = B.CBS_ATTN_ROWS, B.CBS_ATTN_CHUNK, B.CBS_ATTN_CLUSTER
MOST_A_SM = 5   # few-row CTAs an SM, at most; the chunk kernel's: one


@pytest.fixture(scope="module", autouse=True)
def token_calls(cuda_lib):
    from conv_bn_silu_gb300 import build
    build.build_tokens()


def form(attn, tokens):
    """The own part's form where the sizes leave no doubt of it: at most eight CTAs of the
    prefixes' part for each of its tiles of 256 rows keep their SMs from the own part."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    own, prefix = attn.plan.own, attn.plan.prefix
    per_sm = 1 if own.kernel == CHUNK else MOST_A_SM
    if own.grid_ctas > sms * per_sm:
        return "beside"
    tiles = tokens * prefix.desc.heads // prefix.desc.kv_heads // 256 + (prefix.desc.batch + 1) // 2
    taken = 8 * tiles * prefix.desc.kv_heads if prefix.kernel == CHUNK else 0
    assert own.grid_ctas <= (sms - taken) * (1 if own.kernel == CHUNK else 2)
    return "waits"


def check(want_form, own_kernels, sizes, prefixes, lens, new, heads, kv, d, int8, padding, **kw):
    assert sum(new) + padding <= len(lens) * max(new)   # (else run_case would leave the padding out)
    attn = run_case(sizes, prefixes, lens, new, heads, kv, d, 16, int8, padding=padding, **kw)
    assert form(attn, sum(new) + padding) == want_form and attn.plan.own.kernel in own_kernels
    return attn


@pytest.mark.gpu
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("prefixes", [[0, 3], [40, 0], [900, 333]])
def test_few_rows_that_wait(prefixes, d, int8):
    """Single tokens, padding behind them (a sequence may bring two tokens and most bring one or none)."""
    for seed, lens in enumerate(([9, 1, 30], [300, 17, 1000])):
        check("waits", (ROWS, CLUSTER), [1, 2], prefixes, lens, [1, 1, 2] if lens[1] > 1 else [2, 1, 0], 4, 2, d, int8, 2, seed=seed)


@pytest.mark.gpu
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("prefixes", [[0, 7, 0], [50, 0, 200], [3000, 0, 1500]])
def test_few_rows_beside(prefixes, d, int8):
    """Single tokens of many sequences, some with none; a short prefix (few-row
    kernel), a long one (chunks) and none at all."""
    n = 120
    lens = [2 + (i * 29) % 70 for i in range(n)]
    new = [(i % 3 > 0) + (i % 40 == 5) for i in range(n)]
    attn = check("beside", (ROWS, CLUSTER), [60, 20, 40], prefixes, lens, new, 16, 8, d, int8, 9)
    if max(prefixes) in (7, 3000):
        assert (attn.plan.prefix.kernel == CHUNK) == (max(prefixes) == 3000)


@pytest.mark.gpu
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("prefixes,lens,new,padding", [([0], [4000, 50], [200, 30], 5), ([16000], [16000], [250], 0)])
def test_chunks_that_wait(prefixes, lens, new, padding, d, int8):
    """Behind a few-row kernel's prefix, with padding, and behind a chunk kernel's."""
    attn = check("waits", (CHUNK,), [len(lens)], prefixes, lens, new, 8, 1, d, int8, padding)
    assert (attn.plan.prefix.kernel == CHUNK) == (prefixes[0] > 0)


@pytest.mark.gpu
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("prefixes", [[0, 0], [2, 90], [1300, 400]])
def test_chunks_beside(prefixes, d, int8):
    n = 50
    lens = [140 + (i * 53) % 400 for i in range(n)]
    new = [40 + (i * 11) % 50 if i % 7 else i % 2 for i in range(n)]
    check("beside", (CHUNK,), [20, 30], prefixes, lens, new, 16, 4, d, int8, 11)


@pytest.mark.gpu
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("prefix", [60, 2500])
def test_steps_one_after_another(prefix, new, int8):
    """Steps that write keys and values and then attend, the prefix's last page anew as well,
    launched without a pause, with programmatic launches and without, and captured: the own
    part, which begins beside the prefixes' part, sees what was written before both."""
    from conv_bn_silu_gb300 import tokens
    batch, heads, kv, d, page, steps = 120 if new == 1 else 40, 16, 8, 64, 16, 6
    lens = [5 + (i * 29) % 70 for i in range(batch)]
    most = max(lens) + steps * new
    per, pre = -(-most // page), -(-prefix // page)
    cache = tokens.PagedCache.empty(batch * per + pre, kv, page, d, dtype=torch.int8 if int8 else torch.bfloat16)
    i32 = lambda v: torch.tensor(v, dtype=I32, device="cuda")
    order = torch.randperm(batch * per + pre, generator=torch.Generator().manual_seed(1)).to(I32).cuda()
    table, prefix_table = order[:batch * per].view(batch, per).contiguous(), order[batch * per:].view(1, pre).contiguous()
    attn = tokens.SharedPrefixAttention(cache, batch, 1, new, most, prefix, heads)
    assert form(attn, batch * new) == "beside"
    g = torch.Generator("cuda").manual_seed(2)
    draw = lambda *shape: torch.randn(shape, device="cuda", generator=g).to(torch.bfloat16)
    total = batch * new
    q, k, v = draw(steps, total, heads, d), draw(steps, total, kv, d), draw(steps, total, kv, d)
    tail = min(prefix, 10)
    pk, pv = draw(steps, tail, kv, d), draw(steps, tail, kv, d)
    first_k, first_v, first_p = draw(sum(lens), kv, d), draw(sum(lens), kv, d), draw(prefix, kv, d)
    starts, groups, one, length = i32(starts_of([new] * batch)), i32([0, batch]), i32([0, tail]), i32([prefix])
    outs = torch.empty((steps, total, heads, d), dtype=torch.bfloat16, device="cuda")
    now = i32(lens)

    def run(wait=False):
        now.copy_(first_lens)
        cache.write(first_k, first_v, first_starts, now, table)
        cache.write(first_p, first_p, whole, length, prefix_table)
        for i in range(steps):
            now.add_(new)
            cache.write(pk[i], pv[i], one, length, prefix_table)
            cache.write(k[i], v[i], starts, now, table)
            if wait:
                torch.cuda.synchronize()
            attn(q[i], starts, now, table, groups, length, prefix_table, out=outs[i])
            if wait:
                torch.cuda.synchronize()
    first_lens, first_starts, whole = i32(lens), i32(starts_of(lens)), i32([0, prefix])
    options = B.cbs_launch_options()
    try:
        B.cbs_set_launch_options(0)
        run(wait=True)
        want = outs.clone()
    finally:
        B.cbs_set_launch_options(options)
    for _ in range(5):
        outs.zero_()
        run()
        assert torch.equal(outs.view(torch.int16), want.view(torch.int16))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        outs.zero_()
        graph.replay()
        graph.replay()
        assert torch.equal(outs.view(torch.int16), want.view(torch.int16))
    assert want.float().abs().amax() > 0 and B.cbs_read_device_status(True, torch.cuda.current_stream().cuda_stream) == B.CBS_OK
