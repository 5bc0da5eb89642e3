"""Products of 8-bit integers with a scale for each token and channel, against
the same in 64 bits."""
import pytest
import torch

from conv_bn_silu_gb300 import _binding as B
from tests.test_tokens_refusals import I, M, U, refused


@pytest.fixture(scope="module", autouse=True)
def token_calls(cuda_lib):
    from conv_bn_silu_gb300 import build
    build.build_tokens()


def inputs(rows, n, k, seed, bias=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-128, 128, (rows, k), generator=g, dtype=torch.int8)
    w = torch.randint(-128, 128, (n, k), generator=g, dtype=torch.int8)
    xs = torch.rand(rows, generator=g) * 0.02 + 0.01
    ws = (torch.rand(n, generator=g) + 0.5) / (60 * k ** 0.5)
    return x, xs, w, ws, torch.randn(n, generator=g) if bias else None


def reference(x, xs, w, ws, bias, silu):
    """y, and the size that 32-bit roundings of its parts are weighed with."""
    parts = (x.cuda().double() @ w.cuda().double().t()) * xs.cuda().double()[:, None] * ws.cuda().double()
    y, size = parts, parts.abs()
    if bias is not None:
        y, size = y + bias.cuda().double(), size + bias.cuda().double().abs()
    return (y * torch.sigmoid(y) if silu else y), size


def run_case(rows, n, k, bias=False, silu=False, dtype=torch.float32, seed=0, codes=None, sums=0.0):
    """The sums are whole numbers below 2^24 (128 * 128 * k at most, for k up to
    1023; sums of random codes are below 6 sqrt(k) 75^2, under 2^23 for k up to
    62000), so y has four roundings of 32 bits of its parts: the scales' product,
    that with the sum, the bias's addition, and one to spare.  SiLU stretches them
    by at most 1.1 and adds an exponential (2 ulp), a sum and a division, which
    move y by under 2^-21 of itself; the output's own rounding is half a step."""
    from conv_bn_silu_gb300 import tokens
    x, xs, w, ws, b = inputs(rows, n, k, seed, bias)
    if codes is not None:
        x, w = codes(x, w)
    layer = tokens.LinearW8(w.cuda(), ws.cuda(), None if b is None else b.cuda(), B.CBS_ACT_SILU if silu else B.CBS_ACT_IDENTITY)
    out = torch.full((rows, n), 7.0, dtype=dtype, device="cuda")
    assert layer(x.cuda(), xs.cuda(), out=out) is out
    again = layer(x.cuda(), xs.cuda(), dtype=dtype)
    assert torch.equal(out, again)
    assert B.cbs_read_device_status(True, torch.cuda.current_stream().cuda_stream) == B.CBS_OK
    y, size = reference(x, xs, w, ws, b, silu)
    bound = (2.0 ** -22 + sums) * size * (1.1 if silu else 1.0) + (2.0 ** -21 * y.abs() if silu else 0.0)
    bound += torch.finfo(dtype).eps / 2 * (y.abs() + bound) + 1e-30
    err = (out.double() - y).abs()
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.gpu
@pytest.mark.parametrize("n,k", [(1, 16), (127, 48), (128, 128), (129, 144), (300, 1040), (1001, 2064)])
@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 16, 17, 33, 64, 65, 128, 129, 200, 256, 257, 400, 513])
def test_sizes(rows, n, k):
    run_case(rows, n, k, bias=rows % 2 == 0, silu=n % 2 == 1, dtype=torch.float32 if (rows + n) % 3 else torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,n,k", [(1, 6144, 4096), (16, 4096, 14336), (40, 256, 16384), (100, 512, 8192), (1600, 1536, 512),
                                      (3000, 2048, 4096), (1, 70000, 256), (70000, 64, 32), (5000000, 3, 16)])
def test_larger(rows, n, k):
    """Shares of k, rings gone round many times, many tiles."""
    run_case(rows, n, k, dtype=torch.bfloat16)
    run_case(rows, n, k, bias=True, dtype=torch.float32, seed=1)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 20, 300])
@pytest.mark.parametrize("a,b", [(127, 127), (-128, 127), (-128, -128)])
def test_largest_codes(rows, a, b):
    """Sums up to 2^24 are exact (128 * 128 * 1008 < 2^24); past that every MMA's
    addition (sixteen products) rounds to 24 bits or cuts after 23."""
    full = lambda x, w: (torch.full_like(x, a), torch.full_like(w, b))
    run_case(rows, 140, 1008, codes=full)
    run_case(rows, 140, 8192, codes=full, sums=(8192 / 16 + 8) * 2.0 ** -23)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 20, 300])
def test_special_scales(rows):
    """A NaN or an infinity in a scale reaches its own row or channel, and zeros give zeros."""
    from conv_bn_silu_gb300 import tokens
    x, xs, w, ws, _ = inputs(rows, 200, 64, 3)
    xs[0], ws[7], ws[9] = float("nan"), float("inf"), 0.0
    y = tokens.LinearW8(w.cuda(), ws.cuda())(x.cuda(), xs.cuda(), dtype=torch.float32)
    assert y[0].isnan().all()
    assert not y[1:, 7].isfinite().any() and (y[1:, 9] == 0).all()
    fine = torch.ones(200, dtype=torch.bool)
    fine[7] = False
    assert y[1:, fine].isfinite().all()


@pytest.mark.gpu
def test_quantised_weights():
    from conv_bn_silu_gb300 import tokens
    from tests import token_refs as refs
    w = torch.randn((37, 96), generator=torch.Generator().manual_seed(4))
    w[1], w[2, 5], w[3, 6], w[4] = 0.0, float("nan"), float("-inf"), w[4] * 1e-30
    layer = tokens.LinearW8.quantize(w.cuda())
    codes, scale = refs.quantise_rows(w)
    fine = scale.isfinite()
    assert torch.equal(layer.codes.cpu()[fine], codes[fine])
    assert torch.equal(layer.scales.cpu()[fine], scale[fine]) and layer.scales.cpu()[~fine].isnan().all()


@pytest.mark.gpu
def test_captured_and_other_streams():
    from conv_bn_silu_gb300 import tokens
    for rows in (3, 50, 600):
        x, xs, w, ws, _ = inputs(rows, 520, 384, 5)
        layer, x, xs = tokens.LinearW8(w.cuda(), ws.cuda()), x.cuda(), xs.cuda()
        first = layer(x, xs)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            second = layer(x, xs)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                third = layer(x, xs)
            third.zero_()
            graph.replay()
        side.synchronize()
        assert torch.equal(first, second) and torch.equal(first, third)


@pytest.mark.gpu
def test_no_rows():
    from conv_bn_silu_gb300 import tokens
    _, _, w, ws, _ = inputs(1, 20, 32, 6)
    assert tokens.LinearW8(w.cuda(), ws.cuda())(torch.empty((0, 32), dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda")).shape == (0, 20)


def test_refusals(cuda_lib):
    K = 1 << 30   # addresses that are checked for alignment and overlap only
    def call(x=K, xs=2 * K, w=3 * K, ws=4 * K, b=None, y=5 * K, o=B.CBS_BF16, rows=2, n=8, k=64, act=B.CBS_ACT_IDENTITY):
        B.cbs_linear_w8(x, xs, w, ws, b, y, o, rows, n, k, act, None)
    refused(I, lambda: call(o=B.CBS_INT8))
    refused(U, lambda: call(k=40))
    refused(I, lambda: call(k=0))
    refused(I, lambda: call(n=0))
    refused(I, lambda: call(rows=-1))
    refused(U, lambda: call(rows=1 << 25))
    refused(U, lambda: call(n=(1 << 30) + 1))
    refused(U, lambda: call(k=(1 << 30) + 16))
    refused(I, lambda: call(act=5))
    refused(I, lambda: call(x=None))
    refused(I, lambda: call(xs=None))
    refused(I, lambda: call(ws=None))
    refused(M, lambda: call(w=3 * K + 8))
    refused(M, lambda: call(b=6 * K + 4))
    refused(I, lambda: call(y=K + 16))
    refused(I, lambda: call(y=4 * K))
    call(rows=0, x=None)
    refused(U, lambda: B.cbs_quantize_w8(K, 8, 100, 2 * K, 3 * K, None))
    refused(I, lambda: B.cbs_quantize_w8(None, 8, 128, 2 * K, 3 * K, None))
    refused(I, lambda: B.cbs_quantize_w8(K, 8, 128, K + 64, 3 * K, None))


def test_python_refusals():
    from tests.test_tokens_devices import fake
    from conv_bn_silu_gb300 import tokens
    i8, f32 = torch.int8, torch.float32
    layer = (0, 16, 64, B.CBS_ACT_IDENTITY, None, None, None)
    kinds = [((2, 64), i8), ((2,), f32), ((2, 16), torch.bfloat16)]
    call = lambda made: tokens._calls().linear_w8(*made, True, *layer)
    for wrong in range(3):
        with pytest.raises(ValueError, match="device"):
            call([fake(s, t, int(i == wrong)) for i, (s, t) in enumerate(kinds)])
    for i, other in ((0, ((2, 48), i8)), (0, ((2, 64), torch.uint8)), (1, ((3,), f32)), (1, ((2,), torch.bfloat16)),
                     (2, ((2, 16), i8)), (2, ((2, 15), torch.bfloat16))):
        some = list(kinds)
        some[i] = other
        with pytest.raises(ValueError):
            call([fake(s, t) for s, t in some])
    for made in ([((16, 40), i8), ((16,), f32)], [((16, 64), torch.uint8), ((16,), f32)], [((16, 64), i8), ((15,), f32)]):
        with pytest.raises(ValueError):
            tokens.LinearW8(*(fake(s, t) for s, t in made))
    with pytest.raises(ValueError, match="not on cuda:0"):
        tokens.LinearW8(fake((16, 64), i8), fake((16,), f32, 1))
