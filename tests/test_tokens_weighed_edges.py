"""Weighed attention at the edges of its contract: keys and values that are not
finite, rows far from zero, plans of a given split."""
import math

import pytest
import torch

from conv_bn_silu_gb300 import _binding as B
from tests import token_refs as refs
from tests.test_tokens_refusals import I, cache as c_cache, desc, refused, seqs
from tests.test_tokens_weighed import received

I32 = torch.int32
KERNELS = [B.CBS_ATTN_ROWS, B.CBS_ATTN_CLUSTER, B.CBS_ATTN_CHUNK]


@pytest.fixture(scope="module", autouse=True)
def token_calls(cuda_lib):
    from conv_bn_silu_gb300 import build
    build.build_tokens()


def weights(paged, q, lens, new, heads, scale, **plan):
    """(out, what each sequence's positions received: [kv, length])."""
    from conv_bn_silu_gb300 import tokens
    page = paged["k"].shape[2]
    starts = [sum(new[:i]) for i in range(len(new) + 1)]
    dev = {n: None if t is None else t.cuda() for n, t in paged.items()}
    cache = tokens.PagedCache(dev["k"], dev["v"], dev["k_scale"], dev["v_scale"])
    mass = torch.zeros(paged["k"].shape[:3], device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=I32, device="cuda")
    attn = tokens.WeighedAttention(cache, len(lens), max(new), max(lens), heads, scale=scale, **plan)
    out = attn(q.cuda(), i32(starts), i32(lens), dev["table"], mass)
    assert B.cbs_read_device_status(True, torch.cuda.current_stream().cuda_stream) == B.CBS_OK
    mass, got = mass.cpu().double(), []
    for b, n in enumerate(lens):
        pos = torch.arange(n)
        got.append(mass[paged["table"][b].long()[pos // page], :, pos % page].T)
    return out, got


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,kv", [(3, 1), (5, 1), (7, 1), (8, 2), (130, 1)])
def test_a_key_that_nobody_can_reach(heads, kv, d, kernel):
    """A key of minus infinity where every query is positive: scores of minus infinity, and
    no weight, for its position; the others as if it were not there."""
    lens, new, at = [400], [130], 20   # (every new token sees the first 270 positions)
    paged = refs.make_paged(lens, kv, d, 16, False, 3, junk=False)
    page, slot = paged["table"][0, at // 16], at % 16
    paged["k"][page, :, slot, 5] = -math.inf
    q = torch.randn((130, heads, d), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    q[..., 5] = q[..., 5].abs() + 0.5
    out, (got,) = weights(paged, q, lens, new, heads, None, force_kernel=kernel)
    assert got.isfinite().all() and (got[:, at] == 0).all() and out.isfinite().all()
    # what the others receive: the same with a key so far below that nothing reaches it
    paged["k"][page, :, slot] = 0
    paged["k"][page, :, slot, 5] = -3e4
    rec, far = received(q, paged, [0, 130], lens, 16, True, 0, d ** -0.5)[0]
    assert (rec[:, at] < 1e-30).all()
    others = torch.arange(400) != at
    # (that key's own error counts for nothing in the rows' sums, however large its products)
    far = torch.minimum(far, rec * 2.0 ** -8 + 1e-6)
    assert ((got - rec).abs() <= far + 2.0 ** -23 * rec + 1e-30)[:, others].all()


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("heads,kv", [(3, 1), (8, 2)])
def test_a_key_of_infinite_scale(heads, kv, kernel):
    """The same in 8 bits: a key whose scale is infinite, far below every query."""
    lens, new, at = [400], [130], 20
    paged = refs.make_paged(lens, kv, 64, 16, True, 3, junk=False)
    page, slot = paged["table"][0, at // 16], at % 16
    paged["k_scale"][page, :, slot], paged["k"][page, :, slot] = math.inf, 0
    paged["k"][page, :, slot, 5] = -100
    q = torch.randn((130, heads, 64), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    q[..., 5] = q[..., 5].abs() + 0.5
    out, (got,) = weights(paged, q, lens, new, heads, None, force_kernel=kernel)
    assert got.isfinite().all() and (got[:, at] == 0).all() and out.isfinite().all()
    # (what a row gives adds up to one, within n + R + 64 roundings of 2^-23 and the exponentials' 2^-20)
    assert ((got.sum(1) / (130 * heads // kv) - 1).abs() <= (400 + 130 * heads + 64) * 2.0 ** -23 + 2.0 ** -20).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("split", [0, 1, 3])
@pytest.mark.parametrize("size", [30.0, 1e18])
def test_far_rows_beside_values_that_are_not_finite(size, split, kernel):
    """As rows far from zero, with a NaN among the values of the last position: it sends
    the rows of a tile that may not see it on a way of their own, whose scores are summed
    up in another order.  A position still has a row's whole weight or none of it: what a row
    gives is taken from the same scores as what it is divided by."""
    lens, new, heads = [70, 130], [2, 2], 4
    paged = refs.make_paged(lens, 2, 64, 16, False, 9, junk=False)
    for b, n in enumerate(lens):
        paged["v"][paged["table"][b, (n - 1) // 16], :, (n - 1) % 16, 7] = math.nan
    q = torch.randn((4, heads, 64), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16) * size
    _, got = weights(paged, q, lens, new, heads, 100.0, force_kernel=kernel, force_split=split)
    for b, (rec, _) in enumerate(received(q, paged, [0, 2, 4], lens, 16, True, 0, 100.0)):
        assert got[b].isfinite().all(), b
        # whole numbers: no two of these keys' scores are within 2^-20 of one another
        assert torch.equal(rec.round(), got[b].round()), b
        assert (got[b] - got[b].round()).abs().max() <= 1e-3


def test_a_given_split_stays(cuda_lib):
    """force_split of the few-row kernel is its number of ranges, over eight too."""
    for kw in (dict(heads=8), dict(heads=8, cache_prec=B.CBS_BF16, force_kernel=B.CBS_ATTN_ROWS)):
        plan = B.cbs_weighed_plan(desc(batch=1, max_len=8000, force_split=20, **kw))
        assert (plan.attention.kernel, plan.attention.split) == (B.CBS_ATTN_ROWS, 20), kw
    plan = B.cbs_weighed_plan(desc(batch=1, max_len=8000, heads=8))
    assert (plan.attention.kernel, plan.attention.split) == (B.CBS_ATTN_CLUSTER, 8)


def test_weights_on_what_the_call_reads(cuda_lib):
    plan = B.cbs_weighed_plan(desc())
    K = 1 << 30
    c = c_cache(k=5 * K, v=6 * K, k_scale=7 * K, v_scale=8 * K)
    s = seqs(new_start=9 * K, seq_lens=10 * K, page_table=11 * K)
    for at in (9 * K, 10 * K, 11 * K, 9 * K - 16):   # new_start, seq_lens, page_table, and across one's start
        refused(I, B.cbs_weighed_attention, plan, c, s, K, 256, 0.1, 2 * K, 256, at, 1.0, 4 * K, plan.workspace_bytes, None)
