"""Attention of few rows by both forms of its kernel: how many CTAs a call has
decides between them (takes_second, csrc/k_attn_rows.cuh), and its results do not
depend on that."""
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


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("new,causal,window", [(1, True, 0), (2, True, 0), (2, False, 9), (7, True, 0)])
def test_many_sequences_as_few(d, int8, new, causal, window):
    """As many sequences as make from one to five and a half CTAs an SM (one row tile a head:
    of 8 rows, or of 16 in 8 bits), and the same ones a few at a time: to the bit; some of them
    against the 64-bit form."""
    from conv_bn_silu_gb300 import tokens
    kv, heads, page = 8, 16, 16
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    most = (11 * sms // 2 + kv - 1) // kv
    lens = [new + (i * 37) % (90 + 10 * (i % 7)) for i in range(most)]
    lens[5], lens[11] = 0, 15
    fresh = [min(new, n) for n in lens]
    paged = refs.make_paged(lens, kv, d, page, int8, 3)
    # A value that is not finite, seen by the last of two tokens alone.
    if not int8 and new == 2:
        paged["v"][paged["table"][20, (lens[20] - 1) // page], 1, (lens[20] - 1) % page, 3] = float("inf")
    dev = {n: None if t is None else t.cuda() for n, t in paged.items()}
    cache = tokens.PagedCache(dev["k"], dev["v"], dev["k_scale"], dev["v_scale"])
    q = torch.randn((sum(fresh), heads, d), generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    i32 = lambda v: torch.tensor(v, dtype=I32, device="cuda")

    def run(first, count):
        starts = [sum(fresh[first:first + i]) for i in range(count + 1)]
        attn = tokens.PagedAttention(cache, count, new, max(lens), heads, causal=causal, window=window,
                                     force_kernel=B.CBS_ATTN_ROWS, force_split=1)
        assert attn.plan.grid_ctas == count * kv * attn.plan.row_tiles
        a = sum(fresh[:first])
        return attn(q[a:a + starts[-1]].cuda(), i32(starts), i32(lens[first:first + count]), dev["table"][first:first + count].contiguous())
    few = [run(i, min(10, most - i)) for i in range(0, most, 10)]
    few = torch.cat(few)
    for count in sorted({(x * sms // 2 + kv - 1) // kv for x in range(2, 12)} | {2 * sms // kv + 1, 3 * sms // kv, 4 * sms // kv + 1, most}):
        got = run(0, count)
        assert torch.equal(got.view(torch.int16), few[:got.shape[0]].view(torch.int16)), count
    assert B.cbs_read_device_status(True, torch.cuda.current_stream().cuda_stream) == B.CBS_OK
    n, starts = 30, [sum(fresh[:i]) for i in range(31)]
    ref, mag = refs.attention(q[:starts[-1]], paged, starts, lens[:n], page, causal, window, d ** -0.5)
    got = few[:starts[-1]].double().cpu()
    nan = ref.isnan()
    assert torch.equal(~got.isfinite(), nan)
    assert ((got - ref).abs() <= refs.attention_bound(ref, mag))[~nan].all()
