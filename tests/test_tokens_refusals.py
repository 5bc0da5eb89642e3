"""Argument checks of the token operators' C calls (none reaches a GPU)."""
import ctypes

import pytest

from conv_bn_silu_gb300 import _binding as B

OK = 1 << 20   # an address that is checked for alignment only


def cache(**kw):
    d = dict(k=OK, v=OK, k_scale=OK, v_scale=OK, prec=B.CBS_INT8, num_pages=8, page_size=16, kv_heads=2, head_dim=64)
    d.update(kw)
    if d["prec"] == B.CBS_BF16 and "k_scale" not in kw:
        d["k_scale"] = d["v_scale"] = None
    return B.cbs_cache(*[d[n] for n, _ in B.cbs_cache._fields_])


def seqs(**kw):
    d = dict(new_start=OK, seq_lens=OK, page_table=OK, batch=2, max_pages=4, total=6)
    d.update(kw)
    return B.cbs_sequences(*[d[n] for n, _ in B.cbs_sequences._fields_])


def desc(**kw):
    d = dict(batch=2, max_new=4, max_len=64, heads=4, kv_heads=2, head_dim=64, cache_prec=B.CBS_INT8, causal=1,
             window=0, num_sms=0, force_kernel=-1, force_split=0)
    d.update(kw)
    return B.cbs_attn_desc(*[d[n] for n, _ in B.cbs_attn_desc._fields_])


def refused(status, call, *args):
    with pytest.raises(B.CbsError) as e:
        call(*args)
    assert e.value.status == status, e.value


I, U, M, W, P = (B.CBS_ERR_INVALID_ARG, B.CBS_ERR_UNSUPPORTED, B.CBS_ERR_MISALIGNED, B.CBS_ERR_WORKSPACE,
                 B.CBS_ERR_PLAN_MISMATCH)


@pytest.mark.parametrize("status,kw", [
    (I, dict(prec=B.CBS_FP32)), (U, dict(head_dim=96)), (I, dict(kv_heads=0)), (U, dict(page_size=48)),
    (U, dict(page_size=8)), (I, dict(num_pages=0)), (I, dict(k=None)), (M, dict(v=OK + 8)), (I, dict(k_scale=None)),
    (I, dict(prec=B.CBS_BF16, k_scale=OK)), (U, dict(num_pages=1 << 27, kv_heads=16)),
])
def test_caches(cuda_lib, status, kw):
    c = cache(**kw)
    refused(status, B.cbs_cache_write, c, seqs(), OK, 128, OK, 128, B.CBS_BF16, None)
    refused(status, B.cbs_cache_read, c, seqs(), 16, OK, OK, B.CBS_BF16, None)


@pytest.mark.parametrize("status,kw", [
    (I, dict(new_start=None)), (I, dict(seq_lens=None)), (I, dict(page_table=None)), (M, dict(seq_lens=OK + 2)),
    (I, dict(batch=-1)), (I, dict(total=-1)), (I, dict(max_pages=-1)),
])
def test_sequences(cuda_lib, status, kw):
    refused(status, B.cbs_cache_write, cache(), seqs(**kw), OK, 128, OK, 128, B.CBS_BF16, None)


def test_cache_calls(cuda_lib):
    w = lambda *a: B.cbs_cache_write(cache(), seqs(), *a, None)
    refused(I, w, OK, 128, OK, 128, B.CBS_INT8)
    refused(I, w, OK, 120, OK, 128, B.CBS_BF16)
    refused(M, w, OK, 132, OK, 128, B.CBS_BF16)
    refused(I, w, None, 128, OK, 128, B.CBS_BF16)
    refused(M, w, OK, 128, OK + 4, 128, B.CBS_FP32)
    refused(I, B.cbs_cache_write, None, seqs(), OK, 128, OK, 128, B.CBS_BF16, None)
    refused(I, B.cbs_cache_read, cache(), seqs(), -1, OK, OK, B.CBS_BF16, None)
    refused(I, B.cbs_cache_read, cache(), seqs(), 16, None, OK, B.CBS_BF16, None)
    # nothing to do is no error
    B.cbs_cache_write(cache(), seqs(total=0), None, 128, None, 128, B.CBS_BF16, None)
    B.cbs_cache_write(cache(), seqs(batch=0), None, 128, None, 128, B.CBS_BF16, None)
    B.cbs_cache_read(cache(), seqs(), 0, None, None, B.CBS_BF16, None)


@pytest.mark.parametrize("status,kw", [
    (I, dict(heads=3)), (U, dict(head_dim=80)), (I, dict(cache_prec=B.CBS_FP32)), (I, dict(batch=-1)),
    (I, dict(window=-1)), (I, dict(force_kernel=99)), (I, dict(force_split=-1)), (U, dict(batch=70000)),
])
def test_attention_plans(cuda_lib, status, kw):
    refused(status, B.cbs_attn_plan, desc(**kw))


def test_attention_plan_split(cuda_lib):
    """One stream's single token over a long history is split over the SMs;
    many streams are not."""
    one = B.cbs_attn_plan(desc(batch=1, max_new=1, max_len=32768, heads=32, kv_heads=8, head_dim=128))
    many = B.cbs_attn_plan(desc(batch=1024, max_new=1, max_len=256, heads=32, kv_heads=8, head_dim=128))
    assert one.split > 8 and one.workspace_bytes > 0 and one.row_tile == 8
    assert many.split == 1 and many.workspace_bytes == 0
    assert B.cbs_attn_plan(desc(force_split=5)).split == 5


def test_attention_calls(cuda_lib):
    plan = B.cbs_attn_plan(desc(force_split=2))
    def call(p=plan, c=None, s=None, q=OK, qs=256, scale=0.1, out=OK, os=256, ws=OK, wb=None):
        B.cbs_paged_attention(p, c or cache(), s or seqs(), q, qs, scale, out, os, ws,
                              plan.workspace_bytes if wb is None else wb, None)
    refused(I, lambda: call(q=None))
    refused(M, lambda: call(q=OK + 8))
    refused(I, lambda: call(qs=128))
    refused(M, lambda: call(os=260))
    refused(I, lambda: call(scale=float("nan")))
    refused(W, lambda: call(ws=None))
    refused(W, lambda: call(wb=plan.workspace_bytes - 1))
    refused(M, lambda: call(ws=OK + 4))
    refused(P, lambda: call(c=cache(kv_heads=4)))
    refused(P, lambda: call(s=seqs(batch=3)))
    bad = B.cbs_attn_plan_t.from_buffer_copy(plan)
    bad.size = 8
    refused(P, lambda: call(p=bad))
    call(s=seqs(total=0))
    refused(I, lambda: call(p=B.cbs_attn_plan(desc(max_new=0))))


def test_norm_and_rows(cuda_lib):
    def call(x=OK, r=None, w=OK, h=None, y=OK, s=OK, rows=2, cols=64, eps=1e-5, i=B.CBS_BF16, o=B.CBS_INT8):
        B.cbs_rmsnorm(x, r, w, h, y, s, rows, cols, eps, i, o, None)
    refused(I, lambda: call(i=B.CBS_INT8))
    refused(I, lambda: call(o=B.CBS_FP32))
    refused(I, lambda: call(cols=0))
    refused(U, lambda: call(cols=40000))
    refused(I, lambda: call(eps=-1.0))
    refused(I, lambda: call(h=OK))
    refused(I, lambda: call(s=None))
    refused(M, lambda: call(x=OK + 2))
    refused(M, lambda: call(r=OK + 2))
    refused(I, lambda: call(w=None))
    call(rows=0, x=None)
    refused(I, lambda: B.cbs_dequantize_rows(OK, OK, OK, 2, 64, B.CBS_INT8, None))
    refused(I, lambda: B.cbs_dequantize_rows(OK, None, OK, 2, 64, B.CBS_BF16, None))
    refused(M, lambda: B.cbs_dequantize_rows(OK + 1, OK, OK, 2, 64, B.CBS_BF16, None))


def test_w4(cuda_lib):
    def call(x=OK, xp=B.CBS_BF16, xs=None, w=OK, s=OK, z=None, b=None, y=OK, o=B.CBS_BF16, rows=2, n=8, k=128, g=64,
             act=B.CBS_ACT_IDENTITY):
        B.cbs_linear_w4(x, xp, xs, w, s, z, b, y, o, rows, n, k, g, act, None)
    refused(I, lambda: call(xp=B.CBS_FP32))
    refused(I, lambda: call(xs=OK))
    refused(I, lambda: call(xp=B.CBS_INT8))
    refused(I, lambda: call(o=B.CBS_INT8))
    refused(U, lambda: call(g=16))
    refused(U, lambda: call(k=96))
    refused(I, lambda: call(n=0))
    refused(I, lambda: call(rows=-1))
    refused(I, lambda: call(act=5))
    refused(M, lambda: call(w=OK + 4))
    refused(I, lambda: call(s=None))
    refused(M, lambda: call(z=OK + 1))
    call(rows=0, x=None)
    refused(U, lambda: B.cbs_quantize_w4(OK, 8, 100, 64, OK, OK, None))
    refused(I, lambda: B.cbs_quantize_w4(None, 8, 128, 64, OK, OK, None))
