"""8-bit products at the edges of their contract: scales whose product leaves the
float range, and the longest contraction."""
import pytest
import torch

from conv_bn_silu_gb300 import _binding as B
from tests.test_tokens_refusals import U, refused
from tests.test_tokens_w8 import inputs, run_case


@pytest.fixture(scope="module", autouse=True)
def token_calls(cuda_lib):
    from conv_bn_silu_gb300 import build
    build.build_tokens()


# A kernel each: few rows (one tile of eight, two), a tile of 16 and of 128 with shares
# of k and without, pairs of CTAs.
SHAPES = [(1, 200, 64), (12, 200, 64), (20, 200, 64), (20, 129, 1040), (1500, 777, 144), (700, 129, 8208), (3000, 777, 144)]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,n,k", SHAPES)
@pytest.mark.parametrize("x_size,w_size", [(1e-25, 1e-18), (1e-18, 1e-25), (1e33, 1e-30), (1e-30, 1e33)])
def test_scales_far_apart(rows, n, k, x_size, w_size):
    """x_scale w_scale is subnormal or one of the two near the range's end, y is an
    ordinary number: three roundings of 2^-24 (the sum, exact here, times each scale,
    and the bias's addition of none), 2^-22 with one to spare, and a subnormal's step."""
    from conv_bn_silu_gb300 import tokens
    x, xs, w, ws, _ = inputs(rows, n, k, 7)
    xs, ws = xs / 0.02 * x_size, ws * (60 * k ** 0.5) * w_size
    got = tokens.LinearW8(w.cuda(), ws.cuda())(x.cuda(), xs.cuda(), dtype=torch.float32)
    assert B.cbs_read_device_status(True, torch.cuda.current_stream().cuda_stream) == B.CBS_OK
    want = (x.cuda().double() @ w.cuda().double().t()) * xs.cuda().double()[:, None] * ws.cuda().double()
    assert got.isfinite().all()
    bound = 2.0 ** -22 * want.abs() + 2.0 ** -148
    assert ((got.double() - want).abs() <= bound).all(), float(((got.double() - want).abs() / bound).max())


@pytest.mark.gpu
@pytest.mark.parametrize("rows,n,k", SHAPES)
def test_rows_of_zeros_have_no_size(rows, n, k):
    """A sum of zero is zero (and the bias) whatever finite scales it has."""
    from conv_bn_silu_gb300 import tokens
    x, xs, w, ws, bias = inputs(rows, n, k, 8, bias=True)
    x[0] = 0
    got = tokens.LinearW8(w.cuda(), (ws * 0 + 1e30).cuda(), bias.cuda())(x.cuda(), (xs * 0 + 1e30).cuda(), dtype=torch.float32)
    assert torch.equal(got[0].cpu(), bias)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,n", [(1, 300), (12, 300), (20, 140), (100, 300), (300, 1000)])
def test_longest(rows, n):
    """Sums of one sign as far as they go: 65536 products of 2^14, each sixteen of
    them an addition that is off by 2^-23 of the sum so far at most."""
    k = 65536
    full = lambda x, w: (torch.full_like(x, -128), torch.full_like(w, -128))
    run_case(rows, n, k, codes=full, sums=(k / 16 + 16) * 2.0 ** -23)
    run_case(rows, n, k, seed=1, sums=(k / 16 + 16) * 2.0 ** -23)


def test_longer_is_refused(cuda_lib):
    """Past k = 65536 the bound of the sums' error, k / 16 additions of 2^-23, is more
    than 2^-11 of what they add up."""
    K = 1 << 30
    for k in (65536 + 16, 1 << 20, 1 << 30):
        refused(U, B.cbs_linear_w8, K, 2 * K, 3 * K, 4 * K, None, 5 * K, B.CBS_BF16, 2, 8, k, B.CBS_ACT_IDENTITY, None)
        refused(U, B.cbs_quantize_w8, K, 8, k, 2 * K, 3 * K, None)
