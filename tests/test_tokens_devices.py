"""Tensors of another device are refused before anything is launched.  The
tensors here are fakes that name a device and hold no memory, so none of this
needs a GPU."""
import ctypes
from unittest import mock

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from conv_bn_silu_gb300 import _binding as B
from conv_bn_silu_gb300 import tokens


@pytest.fixture(scope="module", autouse=True)
def calls(cuda_lib):
    from conv_bn_silu_gb300 import build
    build.build_tokens()
    return tokens._calls()


def fake(shape, dtype, device=0):
    # (Where there is a GPU, making one would open the device it names, which need not exist.)
    with mock.patch("torch.cuda.is_available", return_value=False), FakeTensorMode(allow_non_fake_inputs=True):
        return torch.empty(shape, dtype=dtype, device=f"cuda:{device}")


BF, F32, I8, I32, U8 = torch.bfloat16, torch.float32, torch.int8, torch.int32, torch.uint8


def refused(call, kinds, at, where):
    """`call` on fakes of `kinds`, all on one device but number `at`."""
    args = [fake(shape, dtype, int(i == at)) for i, (shape, dtype) in enumerate(kinds)]
    with pytest.raises(ValueError, match=where):
        call(*args)


@pytest.mark.parametrize("at", [1, 2, 3])
def test_norm(at):
    kinds = [((2, 8), BF), ((8,), F32), ((2, 8), BF), ((2, 8), BF)]
    refused(lambda x, w, r, h: tokens.rmsnorm(x, w, 1e-5, residual=r, h_out=h), kinds, at, "on another device")


def test_rows():
    refused(tokens.dequantize_rows, [((2, 8), I8), ((2,), F32)], 1, "on another device")


@pytest.mark.parametrize("at", [0, 1, 2])
def test_product_calls(calls, at):
    layer = (0, 16, 64, 64, B.CBS_ACT_IDENTITY, None, None, None, None)   # device, sizes and no arrays
    refused(lambda x, s, out: calls.linear_w4(x, s, out, True, *layer), [((2, 64), I8), ((2,), F32), ((2, 16), BF)], at,
            "device")


@pytest.mark.parametrize("at", [1, 2, 3])
def test_layers(at):
    kinds = [((16, 32), U8), ((1, 16), BF), ((1, 16), U8), ((16,), F32)]
    refused(lambda w, s, z, b: tokens.LinearW4(w, s, 64, z, b), kinds, at, "not on cuda:0")


@pytest.mark.parametrize("at", [1, 2, 3])
def test_caches(at):
    pool = (4, 2, 16, 64)
    refused(tokens.PagedCache, [(pool, I8), (pool, I8), (pool[:3], F32), (pool[:3], F32)], at, "not on cuda:0")


SEQUENCES = [((2,), I32), ((1,), I32), ((1, 4), I32)]   # new_start, seq_lens, page_table


@pytest.fixture
def cache():
    desc = B.cbs_cache(None, None, None, None, B.CBS_INT8, 4, 16, 2, 64)
    yield ctypes.addressof(desc), 0
    del desc


@pytest.mark.parametrize("at", range(5))
def test_cache_writes(calls, cache, at):
    rows = ((3, 2, 64), BF)
    refused(lambda k, v, *s: calls.cache_write(*cache, k, v, *s), [rows, rows, *SEQUENCES], at, "device")


@pytest.mark.parametrize("at", range(2))
def test_cache_reads(calls, cache, at):
    refused(lambda *s: calls.cache_read(*cache, *s, 4, True), SEQUENCES[1:], at, "device")


@pytest.mark.parametrize("at", range(5))
def test_attention(calls, cache, at):
    plan = B.cbs_attn_plan(B.cbs_attn_desc(1, 3, 64, 4, 2, 64, B.CBS_INT8, 1, 0, 152, -1, 0))
    rows = ((3, 4, 64), BF)
    refused(lambda q, out, *s: calls.attention(ctypes.addressof(plan), *cache, q, *s, 0.1, out, None, 0), [rows, rows, *SEQUENCES],
            at, "device")
