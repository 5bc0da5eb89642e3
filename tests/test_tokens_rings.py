"""GPU checks of the 4-bit products over layers so deep that every ring of
stages in shared memory is gone round, each share of k having more stages than
its ring holds (the deepest holds four; k is shared by eight CTAs or warps at
most), against a 64-bit form."""
import pytest
import torch

from conv_bn_silu_gb300 import _binding as B
from conv_bn_silu_gb300 import tokens

pytestmark = pytest.mark.gpu

U, UB = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def token_calls(cuda_lib):
    from conv_bn_silu_gb300 import build
    build.build_tokens()


def check(rows, n, k, group, int8, zeros, bias, silu):
    g = torch.Generator("cuda").manual_seed(rows + n + k)
    kg = k // group
    codes = torch.randint(0, 16, (n, k), generator=g, device="cuda", dtype=torch.uint8)
    c = codes.view(n, k // 8, 8)
    packed = (c[..., [0, 4, 1, 5]] | c[..., [2, 6, 3, 7]] << 4).reshape(n, k // 2)   # (byte i: nibbles 2 i and 2 i + 1)
    scales = (torch.rand((kg, n), generator=g, device="cuda") * 0.02 + 0.01).to(torch.bfloat16)
    z = torch.randint(0, 16, (kg, n), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    b = torch.randn(n, generator=g, device="cuda") if bias else None
    if int8:
        x = torch.randint(-127, 128, (rows, k), generator=g, device="cuda", dtype=torch.int8)
        xs = torch.rand(rows, generator=g, device="cuda") * 0.02 + 0.001
    else:
        x, xs = torch.randn((rows, k), generator=g, device="cuda").to(torch.bfloat16), None
    layer = tokens.LinearW4(packed, scales, group, zeros=z, bias=b, activation=B.CBS_ACT_SILU if silu else B.CBS_ACT_IDENTITY)
    out = [layer(x, xs, dtype=torch.float32) for _ in range(2)]
    assert torch.equal(*out)
    w = codes.double().view(n, kg, group)
    w -= z.t().double().unsqueeze(2) if zeros else 8
    w *= scales.t().double().unsqueeze(2)
    w = w.view(n, k)
    xd = x.double() * (xs.double().unsqueeze(1) if int8 else 1.0)
    y = xd @ w.t()
    size = xd.abs() @ w.abs_().t()
    if bias:
        y, size = y + b.double(), size + b.double().abs()
    ref = y * torch.sigmoid(y) if silu else y
    # A tensor-core sum may drop up to a unit (2^-23) of its largest term at each
    # 16-deep step; then a float sum over groups and shares of k, and the
    # epilogue's few roundings.  SiLU's slope is at most 1.1.
    steps = (0 if int8 else group // 16) + kg + 16
    bound = size * steps * 2.0 ** -23 * 1.1 + ref.abs() * 8 * U + 1e-30
    err = (out[0].double() - ref).abs()
    assert (err <= bound).all(), float((err / bound).max())
    err = (layer(x, xs).double() - ref).abs()
    assert (err <= bound + ref.abs() * UB).all()
    assert B.cbs_read_device_status(True, torch.cuda.current_stream().cuda_stream) == B.CBS_OK


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,n", [(16, 260), (9, 515), (32, 132), (17, 257), (64, 388), (33, 131), (70, 1001)])
def test_products_on_tcgen05(cuda_lib, rows, n, group, int8):
    """41 stages of 256 and a part of one: at least five a share."""
    check(rows, n, 41 * 256 + group, group, int8, zeros=n % 4 != 0 or group == 64, bias=rows % 2 == 1, silu=group == 128)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("rows,n,group", [(16, 20000, 64), (13, 20001, 32), (32, 20002, 128), (40, 20000, 64)])
def test_products_of_one_or_two_shares(cuda_lib, rows, n, group, int8):
    """So many outputs that k is not shared, or by two."""
    check(rows, n, 42 * 256 + group, group, int8, zeros=True, bias=True, silu=False)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("rows,n,group", [(1, 5000, 128), (5, 5001, 64), (8, 5004, 32)])
def test_few_rows_of_a_large_layer(cuda_lib, rows, n, group, int8):
    """Over 48 M weights: too many for the kernel of few rows."""
    k = 41 * 256 + group
    assert n * k > 48 << 20
    check(rows, n, k, group, int8, zeros=rows > 1, bias=False, silu=False)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,n,k", [(1, 100, 8192), (8, 33, 8192), (3, 1001, 8192 + 1024), (4, 30001, 1280)])
def test_few_rows(cuda_lib, rows, n, k, group, int8):
    """A ring of four stages of 128: at least eight a warp's share (the last one
    only a part where the groups allow), and ten where no warp shares k."""
    check(rows, n, k + (group if group < 128 else 0), group, int8, zeros=rows != 3, bias=rows == 3, silu=rows == 8)
