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
