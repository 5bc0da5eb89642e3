"""Plans of the token operators, and outputs on their inputs (host only)."""
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


OK = 1 << 20   # an address that is checked, not read


def lies_on_an_input(call, *args):
    with pytest.raises(B.CbsError, match="lies") as e:
        call(*args)
    assert e.value.status == B.CBS_ERR_INVALID_ARG


def attend(out, out_stride, q=OK, q_stride=256, total=6):
    d = B.cbs_attn_desc(2, 4, 64, 4, 2, 64, B.CBS_INT8, 1, 0, 0, -1, 1)
    cache = B.cbs_cache(OK, OK, OK, OK, B.CBS_INT8, 8, 16, 2, 64)
    B.cbs_paged_attention(B.cbs_attn_plan(d), cache, B.cbs_sequences(OK, OK, OK, 2, 4, total), q, q_stride, 0.1, out, out_stride,
                          None, 0, None)


@pytest.mark.parametrize("at,out_stride,q_stride,total", [
    (0, 256, 256, 6),              # the same tokens
    (512, 256, 256, 6),            # a token later
    (-512, 256, 256, 6),
    (16, 1024, 1024, 6),           # in wider rows: half a head further
    (1024 * 2 - 16, 1024, 1024, 6),   # and across two rows
    (0, 512, 256, 6),              # in rows of another pitch
    (128, 256, 256, 1),            # one token
])
def test_attention_refuses_an_output_on_its_queries(cuda_lib, at, out_stride, q_stride, total):
    lies_on_an_input(attend, OK + at, out_stride, OK, q_stride, total)


def test_products_and_norms_refuse_outputs_on_their_inputs(cuda_lib):
    def product(x=OK, xp=B.CBS_BF16, xs=None, y=OK, o=B.CBS_BF16, rows=2, n=64, k=64):
        B.cbs_linear_w4(x, xp, xs, OK * 4, OK * 4, None, None, y, o, rows, n, k, 64, B.CBS_ACT_IDENTITY, None)
    lies_on_an_input(product)
    lies_on_an_input(lambda: product(y=OK + 2 * 64 * 2 - 16))
    lies_on_an_input(lambda: product(y=OK - 2 * 64 * 2 + 16))
    lies_on_an_input(lambda: product(x=OK * 2, xp=B.CBS_INT8, xs=OK + 16))

    def norm(x=OK, r=OK * 2, h=None, y=OK * 3, s=OK * 4, i=B.CBS_BF16, o=B.CBS_BF16):
        B.cbs_rmsnorm(x, r, OK * 5, h, y, s, 4, 64, 1e-5, i, o, None)
    lies_on_an_input(lambda: norm(h=OK + 16))
    lies_on_an_input(lambda: norm(h=OK * 2 - 16))
    lies_on_an_input(lambda: norm(h=OK * 3))            # y's own place
    lies_on_an_input(lambda: norm(h=OK, y=OK))
    lies_on_an_input(lambda: norm(y=OK + 16))
    lies_on_an_input(lambda: norm(y=OK, o=B.CBS_INT8))  # codes over the values
    lies_on_an_input(lambda: norm(y=OK * 2 + 32, o=B.CBS_INT8))
    lies_on_an_input(lambda: norm(s=OK, o=B.CBS_INT8))
    lies_on_an_input(lambda: B.cbs_dequantize_rows(OK, OK * 2, OK, 4, 64, B.CBS_BF16, None))
    lies_on_an_input(lambda: B.cbs_dequantize_rows(OK, OK * 2, OK * 2 - 16, 4, 64, B.CBS_BF16, None))
