"""Token operators over the C ABI: RMS norm to 8 bits, products with 4-bit
weights, a paged key/value cache in 8 bits or bfloat16, and attention of new
tokens over it.  One quantised step of a model that answers in tokens about
what the layers saw; `token_head` runs them together.

PyTorch supplies device memory and streams; every value is computed in
libcbs.so's kernels, on the current stream.  Tensors are contiguous unless an
argument says that it may be a slice; types and shapes are checked here, the
rest (alignment, limits) by the C calls, which raise CbsError.
"""
from __future__ import annotations

import ctypes
from collections import namedtuple

import torch

from . import _binding as B
from .layer import current_stream, device_sms

_PREC = {torch.float32: B.CBS_FP32, torch.bfloat16: B.CBS_BF16, torch.int8: B.CBS_INT8}
_FLOATS = (torch.float32, torch.bfloat16)

RmsNorm = namedtuple("RmsNorm", "y scale h")


def _want(ok: bool, message: str):
    if not ok:
        raise ValueError(message)


def _dense(t: torch.Tensor, name: str, dtypes, shape=None):
    _want(isinstance(t, torch.Tensor) and t.is_cuda, f"{name}: a CUDA tensor")
    _want(t.dtype in dtypes, f"{name}: {t.dtype}, expected one of {[str(d) for d in dtypes]}")
    _want(t.is_contiguous(), f"{name}: not contiguous")
    _want(shape is None or tuple(t.shape) == tuple(shape), f"{name}: shape {tuple(t.shape)}, expected {shape}")


def _token_stride(t: torch.Tensor, name: str, heads: int, head_dim: int) -> int:
    """Elements between the tokens of [tokens, heads, head_dim], which may be
    a slice of a fused product's rows."""
    _want(isinstance(t, torch.Tensor) and t.is_cuda, f"{name}: a CUDA tensor")
    _want(t.dim() == 3 and t.shape[1] == heads and t.shape[2] == head_dim,
          f"{name}: shape {tuple(t.shape)}, expected (tokens, {heads}, {head_dim})")
    _want(t.stride(2) == 1 and (heads == 1 or t.stride(1) == head_dim), f"{name}: a token's values are not contiguous")
    return t.stride(0) if t.shape[0] > 1 else heads * head_dim


def rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float, residual: torch.Tensor | None = None,
            int8: bool = False, h_out: torch.Tensor | None = None) -> RmsNorm:
    """h = x + residual; y = h weight / sqrt(mean(h^2) + eps), per row.

    Returns (y, scale, h): y in x's type, or int8 codes with a float scale per
    row; h is the sum rounded to x's type (written to h_out, which may be x or
    residual), or x itself without a residual."""
    _dense(x, "x", _FLOATS)
    _want(x.dim() == 2, "x: two dimensions")
    rows, cols = x.shape
    _dense(weight, "weight", (torch.float32,), (cols,))
    h = x
    if residual is not None:
        _dense(residual, "residual", (x.dtype,), x.shape)
        h = torch.empty_like(x) if h_out is None else h_out
        _dense(h, "h_out", (x.dtype,), x.shape)
    else:
        _want(h_out is None, "h_out without a residual is x itself")
    y = torch.empty(x.shape, dtype=torch.int8 if int8 else x.dtype, device=x.device)
    scale = torch.empty(rows, dtype=torch.float32, device=x.device) if int8 else None
    B.cbs_rmsnorm(x, residual, weight, None if residual is None else h, y, scale, rows, cols, eps, _PREC[x.dtype],
                  _PREC[y.dtype], current_stream())
    return RmsNorm(y, scale, h)


def dequantize_rows(q: torch.Tensor, scale: torch.Tensor, dtype=torch.bfloat16) -> torch.Tensor:
    """out[r, c] = q[r, c] scale[r]: rows in 8 bits back to float."""
    _dense(q, "q", (torch.int8,))
    _want(q.dim() == 2, "q: two dimensions")
    _dense(scale, "scale", (torch.float32,), (q.shape[0],))
    _want(dtype in _FLOATS, "dtype: float32 or bfloat16")
    out = torch.empty(q.shape, dtype=dtype, device=q.device)
    B.cbs_dequantize_rows(q, scale, out, q.shape[0], q.shape[1], _PREC[dtype], current_stream())
    return out


class LinearW4:
    """A layer of 4-bit weights: y = act(x W^T + bias), W = s (q - z) by groups
    along k (the packed layout is cbs_linear_w4's)."""

    def __init__(self, packed: torch.Tensor, scales: torch.Tensor, group: int, zeros: torch.Tensor | None = None,
                 bias: torch.Tensor | None = None, activation: int = B.CBS_ACT_IDENTITY):
        _dense(packed, "packed", (torch.uint8,))
        _want(packed.dim() == 2, "packed: [n, k / 2]")
        _want(group in (32, 64, 128), "group: 32, 64 or 128")
        self.n, self.k, self.group = packed.shape[0], packed.shape[1] * 2, group
        _want(self.k % group == 0, f"k = {self.k} is not a multiple of the group ({group})")
        shape = (self.k // group, self.n)
        _dense(scales, "scales", (torch.bfloat16,), shape)
        if zeros is not None:
            _dense(zeros, "zeros", (torch.uint8,), shape)
        if bias is not None:
            _dense(bias, "bias", (torch.float32,), (self.n,))
        self.packed, self.scales, self.zeros, self.bias, self.activation = packed, scales, zeros, bias, activation

    @classmethod
    def quantize(cls, w: torch.Tensor, group: int = 64, bias: torch.Tensor | None = None,
                 activation: int = B.CBS_ACT_IDENTITY) -> "LinearW4":
        """The layer of float weights w [n, k], quantised once on the GPU
        (symmetric, the largest weight of a group at 7)."""
        _dense(w, "w", (torch.float32,))
        _want(w.dim() == 2, "w: [n, k]")
        _want(group in (32, 64, 128) and w.shape[1] % group == 0, "group: 32, 64 or 128, dividing k")
        n, k = w.shape
        packed = torch.empty((n, k // 2), dtype=torch.uint8, device=w.device)
        scales = torch.empty((k // group, n), dtype=torch.bfloat16, device=w.device)
        B.cbs_quantize_w4(w, n, k, group, packed, scales, current_stream())
        return cls(packed, scales, group, bias=bias, activation=activation)

    def __call__(self, x: torch.Tensor, x_scale: torch.Tensor | None = None, dtype=torch.bfloat16,
                 out: torch.Tensor | None = None) -> torch.Tensor:
        """x: bfloat16 [rows, k], or int8 codes with x_scale float [rows]."""
        _dense(x, "x", (torch.bfloat16, torch.int8))
        _want(x.dim() == 2 and x.shape[1] == self.k, f"x: shape {tuple(x.shape)}, expected (rows, {self.k})")
        rows = x.shape[0]
        _want((x_scale is not None) == (x.dtype == torch.int8), "x_scale: with int8 inputs, and only with them")
        if x_scale is not None:
            _dense(x_scale, "x_scale", (torch.float32,), (rows,))
        if out is None:
            _want(dtype in _FLOATS, "dtype: float32 or bfloat16")
            out = torch.empty((rows, self.n), dtype=dtype, device=x.device)
        else:
            _dense(out, "out", _FLOATS, (rows, self.n))
        B.cbs_linear_w4(x, _PREC[x.dtype], x_scale, self.packed, self.scales, self.zeros, self.bias, out,
                        _PREC[out.dtype], rows, self.n, self.k, self.group, self.activation, current_stream())
        return out


class PagedCache:
    """Keys and values in pages [num_pages, kv_heads, page_size, head_dim]:
    bfloat16, or int8 with a float scale for each page, head and position."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor | None = None,
                 v_scale: torch.Tensor | None = None):
        _dense(k, "k", (torch.bfloat16, torch.int8))
        _want(k.dim() == 4, "k: [num_pages, kv_heads, page_size, head_dim]")
        _dense(v, "v", (k.dtype,), k.shape)
        int8 = k.dtype == torch.int8
        _want((k_scale is not None) == int8 and (v_scale is not None) == int8, "scales: with an int8 cache, and only there")
        if int8:
            _dense(k_scale, "k_scale", (torch.float32,), k.shape[:3])
            _dense(v_scale, "v_scale", (torch.float32,), k.shape[:3])
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = k.shape
        self.prec = _PREC[k.dtype]
        self.desc = B.cbs_cache(B._p(k), B._p(v), B._p(k_scale), B._p(v_scale), self.prec, *(
            self.num_pages, self.page_size, self.kv_heads, self.head_dim))
        self._ref = ctypes.byref(self.desc)

    @classmethod
    def empty(cls, num_pages: int, kv_heads: int, page_size: int, head_dim: int, dtype=torch.int8, device="cuda"):
        shape = (num_pages, kv_heads, page_size, head_dim)
        k, v = (torch.empty(shape, dtype=dtype, device=device) for _ in range(2))
        if dtype != torch.int8:
            return cls(k, v)
        return cls(k, v, *(torch.empty(shape[:3], dtype=torch.float32, device=device) for _ in range(2)))

    def sequences(self, new_start, seq_lens, page_table, total: int) -> B.cbs_sequences:
        """A call's sequences (see cbs_sequences), their arrays checked."""
        _dense(seq_lens, "seq_lens", (torch.int32,))
        _want(seq_lens.dim() == 1, "seq_lens: one dimension")
        batch = seq_lens.shape[0]
        _dense(page_table, "page_table", (torch.int32,))
        _want(page_table.dim() == 2 and page_table.shape[0] == batch, "page_table: [batch, max_pages]")
        if new_start is not None:
            _dense(new_start, "new_start", (torch.int32,), (batch + 1,))
        return B.cbs_sequences(B._p(new_start), B._p(seq_lens), B._p(page_table), batch, page_table.shape[1], total)

    def write(self, k: torch.Tensor, v: torch.Tensor, new_start: torch.Tensor, seq_lens: torch.Tensor,
              page_table: torch.Tensor):
        """The new tokens' keys and values ([tokens, kv_heads, head_dim],
        float32 or bfloat16; slices of a fused product's rows do) into their
        pages.  seq_lens counts the new tokens."""
        ks = _token_stride(k, "k", self.kv_heads, self.head_dim)
        vs = _token_stride(v, "v", self.kv_heads, self.head_dim)
        _want(k.dtype in _FLOATS and v.dtype == k.dtype and v.shape == k.shape, "k, v: one shape, float32 or bfloat16")
        seqs = self.sequences(new_start, seq_lens, page_table, k.shape[0])
        B.cbs_cache_write(self._ref, ctypes.byref(seqs), k, ks, v, vs, _PREC[k.dtype], current_stream())

    def read(self, seq_lens: torch.Tensor, page_table: torch.Tensor, max_len: int, dtype=torch.bfloat16):
        """The sequences' keys and values in order, each
        [batch, max_len, kv_heads, head_dim], zero past a sequence's length."""
        _want(dtype in _FLOATS, "dtype: float32 or bfloat16")
        seqs = self.sequences(None, seq_lens, page_table, 0)
        shape = (seqs.batch, max_len, self.kv_heads, self.head_dim)
        k, v = (torch.empty(shape, dtype=dtype, device=self.k.device) for _ in range(2))
        B.cbs_cache_read(self._ref, ctypes.byref(seqs), max_len, k, v, _PREC[dtype], current_stream())
        return k, v


class PagedAttention:
    """Attention of new tokens over a paged cache: the plan for one kind of
    call and the workspace it needs.  Calls that may run at the same time need
    an instance each (`fork`)."""

    def __init__(self, cache: PagedCache, batch: int, max_new: int, max_len: int, heads: int, causal: bool = True,
                 window: int = 0, scale: float | None = None, force_kernel: int = -1, force_split: int = 0):
        self.cache, self.heads = cache, heads
        self.scale = cache.head_dim ** -0.5 if scale is None else float(scale)
        desc = B.cbs_attn_desc(batch, max_new, max_len, heads, cache.kv_heads, cache.head_dim, cache.prec, int(causal),
                               window, device_sms(), force_kernel, force_split)
        self.plan = B.cbs_attn_plan(desc)
        self._plan_ref = ctypes.byref(self.plan)
        self._make_workspace()

    def _make_workspace(self):
        self.workspace_bytes = int(self.plan.workspace_bytes)
        self.workspace = None
        if self.workspace_bytes:
            self.workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=self.cache.k.device)
            B.cbs_workspace_init(self.workspace, self.workspace_bytes, current_stream())

    def fork(self) -> "PagedAttention":
        """The same plan and cache with a workspace of its own."""
        twin = object.__new__(PagedAttention)
        twin.__dict__.update(self.__dict__)
        twin._make_workspace()
        return twin

    def __call__(self, q: torch.Tensor, new_start: torch.Tensor, seq_lens: torch.Tensor, page_table: torch.Tensor,
                 out: torch.Tensor | None = None) -> torch.Tensor:
        """q: bfloat16 [tokens, heads, head_dim] (a slice of a fused product's
        rows does).  The cache already holds the new tokens."""
        d = self.cache.head_dim
        qs = _token_stride(q, "q", self.heads, d)
        _want(q.dtype == torch.bfloat16, "q: bfloat16")
        if out is None:
            out = torch.empty((q.shape[0], self.heads, d), dtype=torch.bfloat16, device=q.device)
        os_ = _token_stride(out, "out", self.heads, d)
        _want(out.dtype == torch.bfloat16 and out.shape == q.shape, "out: bfloat16, shaped like q")
        seqs = self.cache.sequences(new_start, seq_lens, page_table, q.shape[0])
        B.cbs_paged_attention(self._plan_ref, self.cache._ref, ctypes.byref(seqs), q, qs, self.scale, out, os_,
                              self.workspace, self.workspace_bytes, current_stream())
        return out
