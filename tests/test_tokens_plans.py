"""Plans of the token operators (host only)."""
import pytest

from conv_bn_silu_gb300 import _binding as B


def plan(**kw):
    d = dict(batch=1, max_new=1, max_len=32768, heads=32, kv_heads=8, head_dim=128, cache_prec=B.CBS_BF16, causal=1,
             window=0, num_sms=152, force_kernel=-1, force_split=0)
    d.update(kw)
    return B.cbs_attn_plan(B.cbs_attn_desc(*[d[n] for n, _ in B.cbs_attn_desc._fields_]))


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 64, 1 << 30, 40000])
@pytest.mark.parametrize("new", [1, 64, 2048])
def test_a_window_that_hides_nothing_changes_no_plan(cuda_lib, new, window):
    """However large: the keys in sight are the whole sequence's."""
    for prec in (B.CBS_BF16, B.CBS_INT8):
        wide, none = plan(max_new=new, window=window, cache_prec=prec), plan(max_new=new, cache_prec=prec)
        assert (wide.kernel, wide.split, wide.workspace_bytes) == (none.kernel, none.split, none.workspace_bytes)
        assert new > 64 or none.split > 1


@pytest.mark.parametrize("kernel", [-1, B.CBS_ATTN_ROWS, B.CBS_ATTN_CLUSTER])
@pytest.mark.parametrize("new", [1, 2, 3, 8, 9, 40])
def test_row_tiles_hold_the_rows(cuda_lib, new, kernel):
    """Tiles of 8 rows, 16 over an 8-bit cache where there are more than 8."""
    for prec in (B.CBS_BF16, B.CBS_INT8):
        p = plan(max_new=new, cache_prec=prec, force_kernel=kernel)
        rows = 4 * new
        if p.kernel != B.CBS_ATTN_CHUNK:
            assert p.row_tile == (16 if rows > 8 and prec == B.CBS_INT8 else 8)
        assert p.row_tiles == -(-rows // p.row_tile)
