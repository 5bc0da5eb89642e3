"""GPU checks of attention over caches larger than L2: tiles arrive late, and
not in the order they were asked for."""
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


@pytest.mark.parametrize("split", [1, 3])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d,kv", [(128, 8), (64, 16)])
def test_chunks_over_a_cache_in_memory(cuda_lib, d, kv, int8, split):
    batch, length, new, page, heads = 16, 4001, 2, 64, 2 * kv
    g = torch.Generator("cuda").manual_seed(d + split)
    count = -(-length // page)
    shape = (batch * count, kv, page, d)
    table = torch.randperm(batch * count, device="cuda", generator=g).to(torch.int32).view(batch, count)
    if int8:
        k, v = (torch.randint(-127, 128, shape, dtype=torch.int8, device="cuda", generator=g) for _ in range(2))
        ks, vs = (torch.rand(shape[:3], device="cuda", generator=g) * 0.02 + 0.005 for _ in range(2))
    else:
        k, v = (torch.randn(shape, dtype=torch.bfloat16, device="cuda", generator=g) for _ in range(2))
        ks = vs = None
    q = torch.randn((batch * new, heads, d), dtype=torch.bfloat16, device="cuda", generator=g)
    starts = torch.arange(0, batch * new + 1, new, dtype=torch.int32, device="cuda")
    lens = torch.full((batch,), length, dtype=torch.int32, device="cuda")
    attn = tokens.PagedAttention(tokens.PagedCache(k, v, ks, vs), batch, new, length, heads,
                                 force_kernel=B.CBS_ATTN_CHUNK, force_split=split)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    outs = []
    for _ in range(3):   # from memory each time
        flush.zero_()
        torch.cuda.synchronize()
        outs.append(attn(q, starts, lens, table))
    assert B.cbs_read_device_status(True, torch.cuda.current_stream().cuda_stream) == B.CBS_OK
    assert all(torch.equal(o.view(torch.int16), outs[0].view(torch.int16)) for o in outs)
    for b in range(batch):
        at = table[b].long()
        rows = [x[at].double() * (1 if s is None else s[at].double()[..., None]) for x, s in ((k, ks), (v, vs))]
        kk, vv = (x.permute(1, 0, 2, 3).reshape(kv, count * page, d)[:, :length] for x in rows)
        qq = q[b * new:(b + 1) * new].double().view(new, kv, 2, d).permute(1, 0, 2, 3).reshape(kv, new * 2, d)
        scores = qq @ kk.transpose(1, 2) * d ** -0.5
        token = torch.arange(new, device="cuda").repeat_interleave(2)
        seen = torch.arange(length, device="cuda")[None] <= (length - new + token)[:, None]
        p = scores.masked_fill(~seen, float("-inf")).softmax(-1)
        back = lambda x: x.view(kv, new, 2, d).permute(1, 0, 2, 3).reshape(new, heads, d)
        ref, mag = back(p @ vv), back(p @ vv.abs())
        err = (outs[0][b * new:(b + 1) * new].double() - ref).abs()
        assert (err <= refs.attention_bound(ref, mag)).all(), (b, float((err / refs.attention_bound(ref, mag)).max()))


@pytest.mark.parametrize("split", [1, 3, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_values_only_later_tokens_see_over_ranges(cuda_lib, d, split):
    """A NaN among the keys or values of a chunk's own tokens: those before it
    keep their answers, in whichever range of keys it lies and however the
    ranges are joined; after a value's only its dimension is NaN."""
    n, new, page, lens = 1200, 140, 32, [1200, 40]
    starts, i32 = [0, new, new + 3], lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    q = torch.randn((new + 3, 8, d), generator=torch.Generator().manual_seed(22)).to(torch.bfloat16)
    for side, at in (("v", 1100), ("v", 1199), ("k", 1150)):
        paged = refs.make_paged(lens, 2, d, page, False, 21)
        place = paged[side][paged["table"][0, at // page], 1, at % page]
        place[3 if side == "v" else slice(None)] = float("nan")
        cache = tokens.PagedCache(paged["k"].cuda(), paged["v"].cuda())
        attn = tokens.PagedAttention(cache, 2, new, n, 8, force_kernel=B.CBS_ATTN_CHUNK, force_split=split)
        assert attn.plan.split == split
        got = attn(q.cuda(), i32(starts), i32(lens), paged["table"].cuda()).double().cpu()
        ref, mag = refs.attention(q, paged, starts, lens, page, True, 0, d ** -0.5)
        nan = torch.zeros(got.shape, dtype=torch.bool)
        nan[at - (n - new):new, 4:, 3 if side == "v" else slice(None)] = True   # the tokens that see it
        assert torch.equal(got.isnan(), nan) and torch.equal(got.isfinite(), ~nan)
        assert ((got - ref).abs() <= refs.attention_bound(ref, mag))[~nan].all()


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("split", [1, 2, 3, 7, 8, 40])
@pytest.mark.parametrize("d,new", [(64, 1), (128, 1), (64, 4), (128, 3)])
def test_ranges_of_few_rows_joined_in_a_cluster(cuda_lib, d, new, split, int8):
    """Sequences shorter than the ranges leave CTAs of a cluster without keys."""
    from tests.test_tokens_attention import run_case
    got, attn = run_case([1000, 33, 0, 500, 17], [new, min(new, 2), 0, 1, new], 16, 4, d, 16, int8, split=split,
                         kernel=B.CBS_ATTN_CLUSTER)
    assert attn.plan.split == min(split, 8) and attn.plan.workspace_bytes == 0
    run_case([1200, 700], [new, new], 8, 2, d, 32, int8, window=300, split=split, kernel=B.CBS_ATTN_CLUSTER)
    run_case([900], [new], 6, 2, d, 64, int8, causal=False, split=split, kernel=B.CBS_ATTN_CLUSTER)


def test_plans_choose_the_cluster(cuda_lib):
    """Where the planner itself takes up to eight ranges, no workspace is needed."""
    from tests.test_tokens_attention import run_case
    got, attn = run_case([1000], [1], 32, 8, 128, 16, False)
    assert attn.plan.kernel == B.CBS_ATTN_CLUSTER and attn.plan.split == 8 and attn.workspace is None


@pytest.mark.parametrize("split", [2, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_values_only_later_tokens_see_in_a_cluster(cuda_lib, d, split):
    n, new, page, lens = 600, 4, 32, [600, 40]
    paged = refs.make_paged(lens, 2, d, page, False, 23)
    paged["v"][paged["table"][0, 598 // page], 1, 598 % page][3] = float("nan")
    from tests.test_tokens_attention import run_case
    got, attn = run_case(lens, [new, 3], 4, 2, d, page, False, paged=paged, split=split, kernel=B.CBS_ATTN_CLUSTER)
    assert got[:2].isfinite().all() and got[2:4, 2:, 3].isnan().all()
