"""8-bit products by every tile and number of shares of k: what cbs_linear_w8 takes
for a size goes by its costs (csrc/k_w8.cu), so the sizes here are such that it takes
each of them, with odd widths, tails of k, SiLU and last tiles of few rows."""
import pytest
import torch

from tests.test_tokens_w8 import run_case


@pytest.fixture(scope="module", autouse=True)
def token_calls(cuda_lib):
    from conv_bn_silu_gb300 import build
    build.build_tokens()


def both(rows, n, k):
    run_case(rows, n, k, bias=True, silu=True, dtype=torch.float32)
    run_case(rows, n, k, dtype=torch.bfloat16, seed=1)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,n,k", [(2561, 1001, 2064), (300, 9001, 144), (3000, 777, 144), (1025, 6001, 1040), (16385, 129, 144)])
def test_pairs(rows, n, k):
    """Tiles of 256 rows by pairs of CTAs, many a pair or one; of the last one 1, 44, 184, 1 and 1 rows."""
    both(rows, n, k)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,n,k", [
    (1500, 777, 144), (200, 6001, 144), (2049, 3001, 400), (2500, 129, 2064), (1500, 129, 2064), (700, 129, 8208), (500, 257, 8208),
    (65, 9001, 528), (33, 6001, 2064), (33, 4001, 4112), (257, 129, 4112), (17, 129, 528), (17, 9001, 2064), (300, 129, 1040),
    (17, 129, 4112), (17, 129, 144), (9, 12001, 2576), (20, 129, 1040), (17, 129, 2064), (3, 13001, 8208)])
def test_shares(rows, n, k):
    """Tiles of 128 (whole, and 2, 4 and 8 shares of k), 64, 32 and 16 rows (the same)."""
    both(rows, n, k)
