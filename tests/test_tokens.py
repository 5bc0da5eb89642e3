"""GPU checks of the RMS norm, the paged cache's write and read, and the 4-bit
products against plain forms (codes bit for bit, floats within bounds derived
beside each check)."""
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

U = 2.0 ** -24    # rounding to float moves a value by at most this share of it
UB = 2.0 ** -8    # to bfloat16 (eight significant bits)


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------ RMS norm
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 8), (2, 64), (7, 1000), (4, 1001), (300, 127), (2, 2051),
                                       (3, 4096), (2, 8191), (1, 16384), (2, 32767), (1, 32768)])
def test_rmsnorm(cuda_lib, rows, cols, residual, dtype):
    g = gen(rows * 31 + cols)
    x = torch.randn((rows, cols), generator=g).to(dtype)
    r = (torch.randn((rows, cols), generator=g) * 3).to(dtype) if residual else None
    w = torch.rand(cols, generator=g) + 0.5
    h = x.float() + r.float() if residual else x.float()
    dev = lambda t: None if t is None else t.cuda()
    out = tokens.rmsnorm(dev(x), dev(w), 1e-5, residual=dev(r))
    q = tokens.rmsnorm(dev(x), dev(w), 1e-5, residual=dev(r), int8=True)
    if residual:   # one addition, one rounding: the same bits
        assert torch.equal(out.h.cpu(), h.to(dtype)) and torch.equal(q.h.cpu(), h.to(dtype))
    root = (h.double().square().mean(1, keepdim=True) + 1e-5).sqrt()
    ref = h.double() * w.double() / root
    # A float sum of n squares in a tree of at most 8 VPT + 10 steps and the
    # root's and products' roundings: under 40 half units; then the output's own.
    bound = ref.abs() * (40 * U + (UB if dtype == torch.bfloat16 else 0)) + 1e-37
    assert ((out.y.double().cpu() - ref).abs() <= bound).all()
    # The codes do not depend on the sum's order: bit for bit.
    codes, s = refs.quantise_rows(h * w)
    assert torch.equal(q.y.cpu(), codes)
    want = s.double() / root[:, 0]
    assert ((q.scale.double().cpu() - want).abs() <= want * 40 * U).all()
    back = tokens.dequantize_rows(q.y, q.scale, torch.float32).cpu()
    assert torch.equal(back, q.y.cpu().float() * q.scale.cpu()[:, None])
    back = tokens.dequantize_rows(q.y, q.scale).cpu()
    assert torch.equal(back, (q.y.cpu().float() * q.scale.cpu()[:, None]).to(torch.bfloat16))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rmsnorm_in_place_and_special_rows(cuda_lib, dtype):
    g = gen(4)
    x = torch.randn((6, 333), generator=g).to(dtype)
    x[1] = 0
    x[2, 7] = math.nan
    x[3, 332] = math.inf
    x[4] = 1e-30
    r = torch.zeros_like(x)
    w = torch.ones(333)
    xd, rd = x.cuda(), r.cuda()
    q = tokens.rmsnorm(xd, w.cuda(), 1e-6, residual=rd, int8=True, h_out=rd)   # the sum over the residual
    assert q.h is rd and torch.equal(rd.isnan().cpu(), x.isnan())
    back = tokens.dequantize_rows(q.y, q.scale, torch.float32).cpu()
    assert back[2].isnan().all() and back[3].isnan().all() and (back[1] == 0).all()
    assert torch.equal(q.y.cpu()[0], refs.quantise_rows(x[:1])[0][0])
    assert (q.y.cpu()[4] == 127).all()
    y = tokens.rmsnorm(xd, w.cuda(), 1e-6, residual=torch.zeros_like(xd), h_out=xd)
    assert y.h is xd and (y.y.cpu()[1] == 0).all() and y.y.cpu()[2].isnan().all()


# ------------------------------------------------------------ the paged cache
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kv,d,page,lens,new", [(1, 64, 16, [1], [1]), (3, 64, 32, [33, 100, 7], [33, 1, 0]),
                                                (2, 128, 16, [50, 0, 17, 300], [20, 0, 17, 1]),
                                                (8, 128, 256, [700], [259])])
def test_cache_write_and_read(cuda_lib, kv, d, page, lens, new, dtype, int8):
    paged = refs.make_paged(lens, kv, d, page, int8, 21)
    starts = [sum(new[:i]) for i in range(len(new) + 1)]
    g = gen(5)
    rows = (torch.randn((starts[-1], 3, kv, d), generator=g) * 5).to(dtype)
    if starts[-1] > 3:
        rows[1, 1, 0] = 0
        rows[2, 2, kv - 1, 3] = math.inf
        rows[3, 1, 0, d - 1] = math.nan
    dev = {n: None if t is None else t.cuda() for n, t in paged.items()}
    before = {n: None if t is None else t.clone() for n, t in dev.items()}
    cache = tokens.PagedCache(dev["k"], dev["v"], dev["k_scale"], dev["v_scale"])
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    rd = rows.cuda()
    cache.write(rd[:, 1], rd[:, 2], i32(starts), i32(lens), dev["table"])
    want = {n: None if t is None else t.cpu().clone() for n, t in before.items()}
    for b in range(len(lens)):
        for i in range(new[b]):
            pos = lens[b] - new[b] + i
            p, slot = paged["table"][b, pos // page].long(), pos % page
            for side, at in (("k", 1), ("v", 2)):
                row = rows[starts[b] + i, at]
                if int8:
                    want[side][p, :, slot], want[side + "_scale"][p, :, slot] = refs.quantise_rows(row)
                else:
                    want[side][p, :, slot] = row.to(torch.bfloat16)
    for n in ("k", "v", "k_scale", "v_scale"):
        if want[n] is not None:
            assert torch.equal(torch.nan_to_num(dev[n].cpu().float(), 123.0), torch.nan_to_num(want[n].float(), 123.0)), n
    max_len = max(lens) + 3
    for out_dtype in (torch.bfloat16, torch.float32):
        k, v = cache.read(i32(lens), dev["table"], max_len, out_dtype)
        for side, got in (("k", k), ("v", v)):
            for b, n in enumerate(lens):
                ref = refs.rows_of({**want, "table": paged["table"]}, side, b, n, page).float().to(out_dtype)
                assert torch.equal(torch.nan_to_num(got[b, :n].cpu(), 9.0), torch.nan_to_num(ref, 9.0))
                assert (got[b, n:] == 0).all()
    k, _ = cache.read(i32(lens), dev["table"], 5)
    assert k.shape == (len(lens), 5, kv, d)
    assert B.cbs_read_device_status(True, torch.cuda.current_stream().cuda_stream) == B.CBS_OK


def test_cache_places_out_of_range_are_left_out(cuda_lib):
    cache = tokens.PagedCache.empty(4, 2, 16, 64)
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        t.fill_(1)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    x = torch.randn((3, 2, 64), device="cuda")
    table = i32([[9, 2]])                                    # positions 0..15 are in no page of the pool
    cache.write(x, x, i32([0, 3]), i32([17]), table)         # positions 14, 15, 16
    assert B.cbs_read_device_status(True, stream) == B.CBS_ERR_INVALID_ARG
    changed = (cache.k != 1).any(-1)
    assert changed[2, :, 0].all() and int(changed.sum()) == 2
    k, _ = cache.read(i32([17]), table, 20)
    assert B.cbs_read_device_status(True, stream) == B.CBS_ERR_INVALID_ARG
    assert (k[0, :16] == 0).all() and (k[0, 16] != 0).any() and (k[0, 17:] == 0).all()
    cache.write(x, x, i32([0, 2]), i32([1]), i32([[0]]))     # more new tokens than the length; one in no sequence
    assert B.cbs_read_device_status(True, stream) == B.CBS_ERR_INVALID_ARG


def test_offsets_past_32_bits(cuda_lib):
    """A cache whose last page lies over 2^32 bytes in: write, read and
    attention reach it."""
    pages, kv, page, d = 66000, 2, 256, 128                  # 8.65e9 bytes of keys in bf16
    cache = tokens.PagedCache.empty(pages, kv, page, d, dtype=torch.bfloat16)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    table, lens, starts = i32([[pages - 1], [3]]), i32([200, 130]), i32([0, 200, 330])
    g = gen(8)
    rows = torch.randn((330, 2, kv, d), generator=g).to(torch.bfloat16)
    rd = rows.cuda()
    cache.write(rd[:, 0], rd[:, 1], starts, lens, table)
    k, v = cache.read(lens, table, 200)
    assert torch.equal(k[0].cpu(), rows[:200, 0]) and torch.equal(v[0].cpu(), rows[:200, 1])
    assert torch.equal(k[1, :130].cpu(), rows[200:, 0])
    paged = {"k": torch.zeros((2, kv, page, d), dtype=torch.bfloat16), "v": torch.zeros((2, kv, page, d), dtype=torch.bfloat16),
             "k_scale": None, "v_scale": None, "table": torch.tensor([[0], [1]])}
    for b, (a, e) in enumerate(((0, 200), (200, 330))):
        paged["k"][b, :, :e - a], paged["v"][b, :, :e - a] = rows[a:e, 0].transpose(0, 1), rows[a:e, 1].transpose(0, 1)
    for new in (1, 130):
        q = torch.randn((2 * new, 4, d), generator=g).to(torch.bfloat16)
        attn = tokens.PagedAttention(cache, 2, new, 200, 4)
        out = attn(q.cuda(), i32([0, new, 2 * new]), lens, table).double().cpu()
        ref, mag = refs.attention(q, paged, [0, new, 2 * new], [200, 130], page, True, 0, d ** -0.5)
        assert ((out - ref).abs() <= refs.attention_bound(ref, mag)).all()


# ------------------------------------------------------------ 4-bit products
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("rows,n,kg", [(1, 16, 1), (1, 1, 3), (2, 17, 5), (8, 100, 8), (9, 33, 4), (16, 500, 16),
                                       (17, 31, 7), (32, 64, 33), (33, 129, 9), (70, 200, 12)])
def test_linear_w4(cuda_lib, rows, n, kg, group, int8):
    k = kg * group
    g = gen(rows + n * 3 + k)
    codes = torch.randint(0, 16, (n, k), generator=g)
    scales = (torch.rand((kg, n), generator=g) * 0.02 + 0.01).to(torch.bfloat16)
    with_zeros, with_bias, silu = rows % 2 == 1, n % 2 == 1, kg % 2 == 1
    zeros = torch.randint(0, 16, (kg, n), generator=g).to(torch.uint8) if with_zeros else None
    bias = torch.randn(n, generator=g) if with_bias else None
    if int8:
        x = torch.randint(-127, 128, (rows, k), generator=g, dtype=torch.int8)
        xs = torch.rand(rows, generator=g) * 0.02 + 0.001
    else:
        x, xs = torch.randn((rows, k), generator=g).to(torch.bfloat16), None
    dev = lambda t: None if t is None else t.cuda()
    layer = tokens.LinearW4(refs.pack_w4(codes).cuda(), scales.cuda(), group, zeros=dev(zeros), bias=dev(bias),
                            activation=B.CBS_ACT_SILU if silu else B.CBS_ACT_IDENTITY)
    w = codes.double().view(n, kg, group) - (zeros.double().t()[..., None] if with_zeros else 8.0)
    w = (w * scales.double().t()[..., None]).view(n, k)
    xd = x.double() * (xs.double()[:, None] if int8 else 1.0)
    z = xd @ w.t() + (bias.double() if with_bias else 0.0)
    size = xd.abs() @ w.abs().t() + (bias.double().abs() if with_bias else 0.0)
    ref = z / (1 + torch.exp(-z)) if silu else z
    # A tensor-core sum may drop up to a unit (2^-23) of its largest term at
    # each 16-deep step; then a float sum over groups and shares of k, and the
    # epilogue's few roundings.  SiLU's slope is at most 1.1.
    steps = (0 if int8 else group // 16) + kg + 16
    bound = size * steps * 2.0 ** -23 * 1.1 + ref.abs() * 8 * U + 1e-30
    out = layer(dev(x), dev(xs), dtype=torch.float32).double().cpu()
    assert ((out - ref).abs() <= bound).all(), float(((out - ref).abs() / bound).max())
    out = layer(dev(x), dev(xs)).double().cpu()
    assert ((out - ref).abs() <= bound + ref.abs() * UB).all()


@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantize_w4(cuda_lib, group):
    n, k = 37, 4 * group
    w = torch.randn((n, k), generator=gen(3))
    w[5, :group] = 0
    layer = tokens.LinearW4.quantize(w.cuda(), group)
    by = w.view(n, k // group, group)
    s = (by.abs().amax(-1) / torch.full((), 7.0)).to(torch.bfloat16)
    assert torch.equal(layer.scales.cpu(), s.t().contiguous())
    sf = s.float()[..., None]
    codes = torch.where(sf > 0, (by / torch.where(sf > 0, sf, torch.ones_like(sf))).round().clamp(-7, 7), torch.zeros_like(by)) + 8
    assert torch.equal(layer.packed.cpu(), refs.pack_w4(codes.view(n, k).to(torch.int64)))
    x = torch.randn((4, k), generator=gen(4)).to(torch.bfloat16)
    deq = ((codes - 8).double() * s.double()[..., None]).view(n, k)
    ref = x.double() @ deq.t()
    out = layer(x.cuda(), dtype=torch.float32).double().cpu()
    assert ((out - ref).abs() <= (x.double().abs() @ deq.abs().t()) * 40 * 2.0 ** -23).all()


def test_linear_w4_not_finite_inputs_stay_in_their_row(cuda_lib):
    x = torch.randn((3, 256), generator=gen(1)).to(torch.bfloat16)
    x[1, 100] = math.nan
    layer = tokens.LinearW4.quantize(torch.randn((40, 256), generator=gen(2)).cuda(), 64)
    out = layer(x.cuda()).cpu()
    assert out[1].isnan().all() and out[0].isfinite().all() and out[2].isfinite().all()


def test_calls_refuse_unfit_tensors(cuda_lib):
    """Types, shapes, layouts and devices are refused before anything runs;
    what only the C call can tell comes back as CbsError."""
    f32 = lambda *s: torch.zeros(s, device="cuda")
    bf = lambda *s: torch.zeros(s, device="cuda", dtype=torch.bfloat16)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    bad = lambda f: pytest.raises(ValueError, f)
    bad(lambda: tokens.rmsnorm(torch.zeros(2, 8), f32(8), 1e-5))
    bad(lambda: tokens.rmsnorm(f32(2, 8).half(), f32(8), 1e-5))
    bad(lambda: tokens.rmsnorm(f32(2, 8), f32(9), 1e-5))
    bad(lambda: tokens.rmsnorm(f32(8, 2).t(), f32(8), 1e-5))
    bad(lambda: tokens.rmsnorm(f32(2, 8), f32(8), 1e-5, residual=bf(2, 8)))
    bad(lambda: tokens.rmsnorm(f32(2, 8), f32(8), 1e-5, h_out=f32(2, 8)))
    bad(lambda: tokens.dequantize_rows(f32(2, 8), f32(2)))
    bad(lambda: tokens.dequantize_rows(f32(2, 8).to(torch.int8), f32(2), torch.float16))
    with pytest.raises(B.CbsError) as e:
        tokens.rmsnorm(f32(2, 8), f32(8), -1.0)
    assert e.value.status == B.CBS_ERR_INVALID_ARG
    with pytest.raises(B.CbsError) as e:
        tokens.rmsnorm(f32(3, 9).view(-1)[1:19].view(2, 9), f32(9), 1e-5)
    assert e.value.status == B.CBS_ERR_MISALIGNED
    layer = tokens.LinearW4.quantize(torch.randn((16, 128), device="cuda"), 64)
    bad(lambda: layer(f32(2, 128)))
    bad(lambda: layer(bf(2, 64)))
    bad(lambda: layer(bf(2, 128), f32(2)))
    bad(lambda: layer(bf(2, 128).to(torch.int8)))
    bad(lambda: layer(bf(2, 128), out=f32(2, 15)))
    bad(lambda: tokens.LinearW4.quantize(torch.randn((16, 100), device="cuda"), 64))
    cache = tokens.PagedCache.empty(4, 2, 16, 64)
    k = bf(3, 2, 64)
    ok = (i32([0, 3]), i32([3]), i32([[0]]))
    cache.write(k, k, *ok)
    bad(lambda: cache.write(bf(3, 2, 32), k, *ok))
    bad(lambda: cache.write(k, k[:2], *ok))
    bad(lambda: cache.write(k, k, ok[0].long(), ok[1], ok[2]))
    bad(lambda: cache.write(k, k, i32([0, 1, 3]), ok[1], ok[2]))
    bad(lambda: cache.read(ok[1], i32([0]), 4))
    bad(lambda: tokens.PagedCache(cache.k, cache.v))
    attn = tokens.PagedAttention(cache, 1, 3, 16, 4)
    bad(lambda: attn(f32(3, 4, 64), *ok))
    bad(lambda: attn(bf(3, 2, 64), *ok))
    bad(lambda: attn(bf(3, 4, 64), *ok, out=bf(2, 4, 64)))
    assert attn(bf(3, 4, 64), *ok).shape == (3, 4, 64)


@pytest.mark.parametrize("int8", [False, True])
def test_nothing_to_do(cuda_lib, int8):
    """Empty batches, rows and calls come back empty."""
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    cache = tokens.PagedCache.empty(4, 2, 16, 64, dtype=torch.int8 if int8 else torch.bfloat16)
    none = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    cache.write(none, none, i32([0, 0]), i32([0]), i32([[0]]))
    k, v = cache.read(i32([0]), i32([[0]]), 3)
    assert (k == 0).all() and (v == 0).all() and k.shape == (1, 3, 2, 64)
    assert tokens.PagedAttention(cache, 1, 4, 16, 4)(none.new_zeros((0, 4, 64)), i32([0, 0]), i32([0]), i32([[0]])).shape == (0, 4, 64)
    x = torch.zeros((0, 128), dtype=torch.bfloat16, device="cuda")
    assert tokens.rmsnorm(x, torch.ones(128, device="cuda"), 1e-5, int8=int8).y.shape == (0, 128)
    assert tokens.LinearW4.quantize(torch.randn((16, 128), device="cuda"), 64)(x).shape == (0, 16)
    assert B.cbs_read_device_status(True, torch.cuda.current_stream().cuda_stream) == B.CBS_OK
