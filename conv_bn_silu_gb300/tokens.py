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
from .layer import device_sms

_PREC = {torch.float32: B.CBS_FP32, torch.bfloat16: B.CBS_BF16, torch.int8: B.CBS_INT8}
_FLOATS = (torch.float32, torch.bfloat16)
_BF16, _F32, _I8, _I32 = torch.bfloat16, torch.float32, torch.int8, torch.int32

RmsNorm = namedtuple("RmsNorm", "y scale h")

# A single-token step is as long as its calls' host time, so the checks below
# cost a few attribute reads each and build their messages only on failure.


def _stream(t: torch.Tensor) -> int:
    """The current stream of the tensor's device (a raw handle)."""
    return torch._C._cuda_getCurrentRawStream(t.device.index)


def _refuse(message: str):
    raise ValueError(message)


def _dense(t: torch.Tensor, name: str, dtypes, shape=None):
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        _refuse(f"{name}: expected a CUDA tensor")
    if t.dtype not in dtypes:
        _refuse(f"{name}: {t.dtype}, expected one of {[str(d) for d in dtypes]}")
    if not t.is_contiguous():
        _refuse(f"{name}: not contiguous")
    if shape is not None and t.shape != shape:
        _refuse(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _tokens(t: torch.Tensor, name: str, dtype, heads: int, head_dim: int) -> int:
    """Elements between the tokens of [tokens, heads, head_dim], which may be
    a slice of a fused product's rows."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype):
        _refuse(f"{name}: expected a CUDA tensor of {dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != head_dim:
        _refuse(f"{name}: shape {tuple(shape)}, expected (tokens, {heads}, {head_dim})")
    step, head, one = t.stride()
    if one != 1 or (head != head_dim and heads != 1):
        _refuse(f"{name}: a token's values are not contiguous")
    return step if shape[0] > 1 else heads * head_dim


def rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float, residual: torch.Tensor | None = None,
            int8: bool = False, h_out: torch.Tensor | None = None) -> RmsNorm:
    """h = x + residual; y = h weight / sqrt(mean(h^2) + eps), per row.

    Returns (y, scale, h): y in x's type, or int8 codes with a float scale per
    row; h is the sum rounded to x's type (written to h_out, which may be x or
    residual), or x itself without a residual."""
    _dense(x, "x", _FLOATS)
    shape, dtype = x.shape, x.dtype
    if len(shape) != 2:
        _refuse("x: expected two dimensions")
    rows, cols = shape
    _dense(weight, "weight", (_F32,), (cols,))
    h, h_at, r_at = x, None, None
    if residual is not None:
        _dense(residual, "residual", (dtype,), shape)
        if h_out is None:
            h = torch.empty_like(x)
        else:
            _dense(h_out, "h_out", (dtype,), shape)
            h = h_out
        h_at, r_at = h.data_ptr(), residual.data_ptr()
    elif h_out is not None:
        _refuse("h_out without a residual is x itself")
    if int8:
        y = torch.empty(shape, dtype=_I8, device=x.device)
        scale = torch.empty(rows, dtype=_F32, device=x.device)
        s_at, out = scale.data_ptr(), B.CBS_INT8
    else:
        y, scale, s_at, out = torch.empty_like(x), None, None, _PREC[dtype]
    status = B.lib().cbs_rmsnorm(x.data_ptr(), r_at, weight.data_ptr(), h_at, y.data_ptr(), s_at, rows, cols, eps,
                                 _PREC[dtype], out, _stream(x))
    if status:
        B._check(status, "cbs_rmsnorm")
    return RmsNorm(y, scale, h)


def dequantize_rows(q: torch.Tensor, scale: torch.Tensor, dtype=torch.bfloat16) -> torch.Tensor:
    """out[r, c] = q[r, c] scale[r]: rows in 8 bits back to float."""
    _dense(q, "q", (_I8,))
    shape = q.shape
    if len(shape) != 2:
        _refuse("q: expected two dimensions")
    _dense(scale, "scale", (_F32,), (shape[0],))
    if dtype not in _FLOATS:
        _refuse("dtype: float32 or bfloat16")
    out = torch.empty(shape, dtype=dtype, device=q.device)
    status = B.lib().cbs_dequantize_rows(q.data_ptr(), scale.data_ptr(), out.data_ptr(), shape[0], shape[1],
                                         _PREC[dtype], _stream(q))
    if status:
        B._check(status, "cbs_dequantize_rows")
    return out


class LinearW4:
    """A layer of 4-bit weights: y = act(x W^T + bias), W = s (q - z) by groups
    along k (the packed layout is cbs_linear_w4's)."""

    def __init__(self, packed: torch.Tensor, scales: torch.Tensor, group: int, zeros: torch.Tensor | None = None,
                 bias: torch.Tensor | None = None, activation: int = B.CBS_ACT_IDENTITY):
        _dense(packed, "packed", (torch.uint8,))
        if packed.dim() != 2:
            _refuse("packed: expected [n, k / 2]")
        if group not in (32, 64, 128):
            _refuse("group: 32, 64 or 128")
        self.n, self.k, self.group = packed.shape[0], packed.shape[1] * 2, group
        if self.k % group:
            _refuse(f"k = {self.k} is not a multiple of the group ({group})")
        shape = (self.k // group, self.n)
        _dense(scales, "scales", (_BF16,), shape)
        if zeros is not None:
            _dense(zeros, "zeros", (torch.uint8,), shape)
        if bias is not None:
            _dense(bias, "bias", (_F32,), (self.n,))
        self.packed, self.scales, self.zeros, self.bias, self.activation = packed, scales, zeros, bias, activation
        self._at = tuple(map(B._p, (packed, scales, zeros, bias)))   # the layer's own tensors, held above

    @classmethod
    def quantize(cls, w: torch.Tensor, group: int = 64, bias: torch.Tensor | None = None,
                 activation: int = B.CBS_ACT_IDENTITY) -> "LinearW4":
        """The layer of float weights w [n, k], quantised once on the GPU
        (symmetric, the largest weight of a group at 7)."""
        _dense(w, "w", (_F32,))
        if w.dim() != 2 or group not in (32, 64, 128) or w.shape[1] % group:
            _refuse("w: expected [n, k], with k a multiple of the group (32, 64 or 128)")
        n, k = w.shape
        packed = torch.empty((n, k // 2), dtype=torch.uint8, device=w.device)
        scales = torch.empty((k // group, n), dtype=_BF16, device=w.device)
        B.cbs_quantize_w4(w, n, k, group, packed, scales, _stream(w))
        return cls(packed, scales, group, bias=bias, activation=activation)

    def __call__(self, x: torch.Tensor, x_scale: torch.Tensor | None = None, dtype=torch.bfloat16,
                 out: torch.Tensor | None = None) -> torch.Tensor:
        """x: bfloat16 [rows, k], or int8 codes with x_scale float [rows]."""
        _dense(x, "x", (_BF16, _I8))
        shape = x.shape
        if len(shape) != 2 or shape[1] != self.k:
            _refuse(f"x: shape {tuple(shape)}, expected (rows, {self.k})")
        rows, prec = shape[0], _PREC[x.dtype]
        if (x_scale is not None) != (prec == B.CBS_INT8):
            _refuse("x_scale: with int8 inputs, and only with them")
        if x_scale is not None:
            _dense(x_scale, "x_scale", (_F32,), (rows,))
            x_scale = x_scale.data_ptr()
        if out is None:
            if dtype not in _FLOATS:
                _refuse("dtype: float32 or bfloat16")
            out = torch.empty((rows, self.n), dtype=dtype, device=x.device)
        else:
            _dense(out, "out", _FLOATS, (rows, self.n))
        w, scales, zeros, bias = self._at
        status = B.lib().cbs_linear_w4(x.data_ptr(), prec, x_scale, w, scales, zeros, bias, out.data_ptr(),
                                       _PREC[out.dtype], rows, self.n, self.k, self.group, self.activation, _stream(x))
        if status:
            B._check(status, "cbs_linear_w4")
        return out


class PagedCache:
    """Keys and values in pages [num_pages, kv_heads, page_size, head_dim]:
    bfloat16, or int8 with a float scale for each page, head and position."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor | None = None,
                 v_scale: torch.Tensor | None = None):
        _dense(k, "k", (_BF16, _I8))
        if k.dim() != 4:
            _refuse("k: expected [num_pages, kv_heads, page_size, head_dim]")
        _dense(v, "v", (k.dtype,), k.shape)
        int8 = k.dtype == _I8
        if (k_scale is not None) != int8 or (v_scale is not None) != int8:
            _refuse("scales: with an int8 cache, and only there")
        if int8:
            _dense(k_scale, "k_scale", (_F32,), k.shape[:3])
            _dense(v_scale, "v_scale", (_F32,), k.shape[:3])
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
        _dense(seq_lens, "seq_lens", (_I32,))
        _dense(page_table, "page_table", (_I32,))
        shape = page_table.shape
        if seq_lens.dim() != 1 or len(shape) != 2 or shape[0] != seq_lens.shape[0]:
            _refuse("seq_lens, page_table: expected [batch], [batch, max_pages]")
        starts = None
        if new_start is not None:
            _dense(new_start, "new_start", (_I32,), (shape[0] + 1,))
            starts = new_start.data_ptr()
        return B.cbs_sequences(starts, seq_lens.data_ptr(), page_table.data_ptr(), shape[0], shape[1], total)

    def write(self, k: torch.Tensor, v: torch.Tensor, new_start: torch.Tensor, seq_lens: torch.Tensor,
              page_table: torch.Tensor):
        """The new tokens' keys and values ([tokens, kv_heads, head_dim],
        float32 or bfloat16; slices of a fused product's rows do) into their
        pages.  seq_lens counts the new tokens."""
        dtype = k.dtype
        if dtype not in _FLOATS:
            _refuse("k, v: float32 or bfloat16")
        ks = _tokens(k, "k", dtype, self.kv_heads, self.head_dim)
        vs = _tokens(v, "v", dtype, self.kv_heads, self.head_dim)
        total = k.shape[0]
        if v.shape[0] != total:
            _refuse("k, v: expected the same tokens")
        seqs = self.sequences(new_start, seq_lens, page_table, total)
        status = B.lib().cbs_cache_write(self._ref, ctypes.byref(seqs), k.data_ptr(), ks, v.data_ptr(), vs,
                                         _PREC[dtype], _stream(k))
        if status:
            B._check(status, "cbs_cache_write")

    def read(self, seq_lens: torch.Tensor, page_table: torch.Tensor, max_len: int, dtype=torch.bfloat16):
        """The sequences' keys and values in order, each
        [batch, max_len, kv_heads, head_dim], zero past a sequence's length."""
        if dtype not in _FLOATS:
            _refuse("dtype: float32 or bfloat16")
        seqs = self.sequences(None, seq_lens, page_table, 0)
        shape, device = (page_table.shape[0], max_len, self.kv_heads, self.head_dim), self.k.device
        k, v = torch.empty(shape, dtype=dtype, device=device), torch.empty(shape, dtype=dtype, device=device)
        status = B.lib().cbs_cache_read(self._ref, ctypes.byref(seqs), max_len, k.data_ptr(), v.data_ptr(),
                                        _PREC[dtype], _stream(k))
        if status:
            B._check(status, "cbs_cache_read")
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
        self.workspace = self._workspace_at = None
        if self.workspace_bytes:
            self.workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=self.cache.k.device)
            B.cbs_workspace_init(self.workspace, self.workspace_bytes, _stream(self.workspace))
            self._workspace_at = self.workspace.data_ptr()

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
        cache = self.cache
        d = cache.head_dim
        qs = _tokens(q, "q", _BF16, self.heads, d)
        total = q.shape[0]
        if out is None:
            out = torch.empty((total, self.heads, d), dtype=_BF16, device=q.device)
            os = self.heads * d
        else:
            os = _tokens(out, "out", _BF16, self.heads, d)
            if out.shape[0] != total:
                _refuse("out: expected the tokens of q")
        seqs = cache.sequences(new_start, seq_lens, page_table, total)
        status = B.lib().cbs_paged_attention(self._plan_ref, cache._ref, ctypes.byref(seqs), q.data_ptr(), qs,
                                             self.scale, out.data_ptr(), os, self._workspace_at, self.workspace_bytes,
                                             _stream(q))
        if status:
            B._check(status, "cbs_paged_attention")
        return out
