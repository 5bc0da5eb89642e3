"""Token operators over the C ABI: RMS norm to 8 bits, products with 4-bit
weights, a paged key/value cache in 8 bits or bfloat16, and attention of new
tokens over it.  One quantised step of a model that answers in tokens about
what the layers saw; `token_head` runs them together.

PyTorch supplies device memory and streams; every value is computed in
libcbs.so's kernels, on the current stream of the tensors' device (all of a call's
are on one).  Tensors are contiguous unless an argument says that it may be a slice.  Types and shapes are checked by the calls
of csrc/tokens_py.cpp (ValueError), the rest (alignment, limits, outputs on their
inputs) by the C calls behind them, which raise CbsError.

For inference only: a tensor that requires a gradient is taken as it is, and the
result carries none.  The calls are not traced: a tensor without memory (a fake
one) raises PyTorch's own error.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
from collections import namedtuple

import torch

from . import _binding as B
from .layer import current_stream, device_sms

_FLOATS = (torch.float32, torch.bfloat16)
_BF16, _F32, _I8 = torch.bfloat16, torch.float32, torch.int8

RmsNorm = namedtuple("RmsNorm", "y scale h")

_module = None


def _calls():
    """csrc/tokens_py.cpp, built beside libcbs.so; there is no other path."""
    global _module
    if _module is None:
        B.lib()
        path = os.path.join(os.path.dirname(B.LIB_PATH), "_tokens.so")
        if not os.path.exists(path):
            raise ImportError(f"the token operators' calls are not built ({path}); run conv_bn_silu_gb300/build.py")
        spec = importlib.util.spec_from_file_location("_tokens", path)
        _module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(_module)
    return _module


def _done(result, where: str):
    """A call's tensors, or CbsError for the status it came back with."""
    if type(result) is int:
        B._check(result, where)
    return result


def _refuse(message: str):
    raise ValueError(message)


def _dense(t: torch.Tensor, name: str, dtypes, shape=None, device=None):
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        _refuse(f"{name}: expected a CUDA tensor")
    if device is not None and t.device != device:
        _refuse(f"{name}: on {t.device}, not on {device}")
    if t.dtype not in dtypes:
        _refuse(f"{name}: {t.dtype}, expected one of {[str(d) for d in dtypes]}")
    if not t.is_contiguous():
        _refuse(f"{name}: not contiguous")
    if shape is not None and t.shape != shape:
        _refuse(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float, residual: torch.Tensor | None = None,
            int8: bool = False, h_out: torch.Tensor | None = None) -> RmsNorm:
    """h = x + residual; y = h weight / sqrt(mean(h^2) + eps), per row of x.

    Returns (y, scale, h): y in x's type, or int8 codes with a float scale per
    row; h is the sum rounded to x's type (written to h_out, which may be x or
    residual), or x itself without a residual."""
    return RmsNorm._make(_done(_calls().rmsnorm(x, weight, eps, residual, int8, h_out), "cbs_rmsnorm"))


def dequantize_rows(q: torch.Tensor, scale: torch.Tensor, dtype=torch.bfloat16) -> torch.Tensor:
    """out[r, c] = q[r, c] scale[r]: rows in 8 bits back to float."""
    if dtype not in _FLOATS:
        _refuse("dtype: float32 or bfloat16")
    return _done(_calls().dequantize_rows(q, scale, dtype is _BF16), "cbs_dequantize_rows")


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
        _dense(scales, "scales", (_BF16,), shape, packed.device)
        if zeros is not None:
            _dense(zeros, "zeros", (torch.uint8,), shape, packed.device)
        if bias is not None:
            _dense(bias, "bias", (_F32,), (self.n,), packed.device)
        self.packed, self.scales, self.zeros, self.bias, self.activation = packed, scales, zeros, bias, activation
        # what a call needs of the layer: its device and sizes, and its own tensors (held above)
        self._args = (packed.device.index, self.n, self.k, group, activation, *map(B._p, (packed, scales, zeros, bias)))

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
        with torch.cuda.device(w.device):
            B.cbs_quantize_w4(w, n, k, group, packed, scales, current_stream())
        return cls(packed, scales, group, bias=bias, activation=activation)

    def __call__(self, x: torch.Tensor, x_scale: torch.Tensor | None = None, dtype=torch.bfloat16,
                 out: torch.Tensor | None = None) -> torch.Tensor:
        """x: bfloat16 [rows, k], or int8 codes with x_scale float [rows].  The
        result is of `dtype`, or of out's type where out is given."""
        if dtype not in _FLOATS:
            _refuse("dtype: float32 or bfloat16")
        return _done(_calls().linear_w4(x, x_scale, out, dtype is _BF16, *self._args), "cbs_linear_w4")


class LinearW8:
    """A layer of 8-bit weights [n, k] (k at most 65536), a float scale for each output:
    y = act(x_scale w_scale (x W^T) + bias), for one row of codes as for thousands."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, bias: torch.Tensor | None = None,
                 activation: int = B.CBS_ACT_IDENTITY):
        _dense(codes, "codes", (_I8,))
        if codes.dim() != 2:
            _refuse("codes: expected [n, k]")
        self.n, self.k = codes.shape
        if self.k % 16:
            _refuse(f"k = {self.k} is not a multiple of 16")
        _dense(scales, "scales", (_F32,), (self.n,), codes.device)
        if bias is not None:
            _dense(bias, "bias", (_F32,), (self.n,), codes.device)
        self.codes, self.scales, self.bias, self.activation = codes, scales, bias, activation
        self._args = (codes.device.index, self.n, self.k, activation, *map(B._p, (codes, scales, bias)))

    @classmethod
    def quantize(cls, w: torch.Tensor, bias: torch.Tensor | None = None, activation: int = B.CBS_ACT_IDENTITY) -> "LinearW8":
        """The layer of float weights w [n, k], quantised once on the GPU (an
        output's largest weight at 127)."""
        _dense(w, "w", (_F32,))
        if w.dim() != 2 or w.shape[1] % 16:
            _refuse("w: expected [n, k], with k a multiple of 16")
        codes = torch.empty(w.shape, dtype=_I8, device=w.device)
        scales = torch.empty(w.shape[0], dtype=_F32, device=w.device)
        with torch.cuda.device(w.device):
            B.cbs_quantize_w8(w, *w.shape, codes, scales, current_stream())
        return cls(codes, scales, bias=bias, activation=activation)

    def __call__(self, x: torch.Tensor, x_scale: torch.Tensor, dtype=torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
        """x: int8 codes [rows, k] with x_scale float [rows].  The result is of
        `dtype`, or of out's type where out is given."""
        if dtype not in _FLOATS:
            _refuse("dtype: float32 or bfloat16")
        return _done(_calls().linear_w8(x, x_scale, out, dtype is _BF16, *self._args), "cbs_linear_w8")


class PagedCache:
    """Keys and values in pages [num_pages, kv_heads, page_size, head_dim]:
    bfloat16, or int8 with a float scale for each page, head and position."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor | None = None,
                 v_scale: torch.Tensor | None = None):
        _dense(k, "k", (_BF16, _I8))
        if k.dim() != 4:
            _refuse("k: expected [num_pages, kv_heads, page_size, head_dim]")
        _dense(v, "v", (k.dtype,), k.shape, k.device)
        int8 = k.dtype == _I8
        if (k_scale is not None) != int8 or (v_scale is not None) != int8:
            _refuse("scales: with an int8 cache, and only there")
        if int8:
            _dense(k_scale, "k_scale", (_F32,), k.shape[:3], k.device)
            _dense(v_scale, "v_scale", (_F32,), k.shape[:3], k.device)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = k.shape
        self.prec = B.CBS_INT8 if int8 else B.CBS_BF16
        self.desc = B.cbs_cache(B._p(k), B._p(v), B._p(k_scale), B._p(v_scale), self.prec, *(
            self.num_pages, self.page_size, self.kv_heads, self.head_dim))
        self._at = ctypes.addressof(self.desc), k.device.index

    @classmethod
    def empty(cls, num_pages: int, kv_heads: int, page_size: int, head_dim: int, dtype=torch.int8, device="cuda"):
        shape = (num_pages, kv_heads, page_size, head_dim)
        k, v = (torch.empty(shape, dtype=dtype, device=device) for _ in range(2))
        if dtype != torch.int8:
            return cls(k, v)
        return cls(k, v, *(torch.empty(shape[:3], dtype=torch.float32, device=device) for _ in range(2)))

    def write(self, k: torch.Tensor, v: torch.Tensor, new_start: torch.Tensor, seq_lens: torch.Tensor,
              page_table: torch.Tensor):
        """The new tokens' keys and values ([tokens, kv_heads, head_dim],
        float32 or bfloat16; slices of a fused product's rows do) into their
        pages.  seq_lens counts the new tokens."""
        _done(_calls().cache_write(*self._at, k, v, new_start, seq_lens, page_table), "cbs_cache_write")

    def read(self, seq_lens: torch.Tensor, page_table: torch.Tensor, max_len: int, dtype=torch.bfloat16):
        """The sequences' keys and values in order, each
        [batch, max_len, kv_heads, head_dim], zero past a sequence's length."""
        if dtype not in _FLOATS:
            _refuse("dtype: float32 or bfloat16")
        return _done(_calls().cache_read(*self._at, seq_lens, page_table, max_len, dtype is _BF16), "cbs_cache_read")[:2]

    def evict(self, mass: torch.Tensor, seq_lens: torch.Tensor, page_table: torch.Tensor, new_table: torch.Tensor, keep: int,
              recent: int = 0):
        """The last `recent` positions of each sequence and the heaviest others,
        `keep` in all, in order to the pages of new_table (int32 [batch, pages],
        none of them the sequences' own, none twice: not checked); each key head chooses by itself.  mass:
        float32 [num_pages, kv_heads, page_size] (WeighedAttention adds it up), which
        moves along.  Returns the old positions (int32 [batch, kv_heads, keep], -1
        past them) and the new lengths."""
        return _done(_calls().cache_evict(*self._at, mass, seq_lens, page_table, new_table, keep, recent), "cbs_cache_evict")[:2]


class PagedAttention:
    """Attention of new tokens over a paged cache: the plan for one kind of
    call and the workspace it needs, ready for any stream once the constructor
    has returned.  Calls that may run at the same time need an instance each
    (`fork`); a captured call needs its instance for as long as its graph."""

    def __init__(self, cache: PagedCache, batch: int, max_new: int, max_len: int, heads: int, causal: bool = True,
                 window: int = 0, scale: float | None = None, force_kernel: int = -1, force_split: int = 0):
        self.cache, self.heads = cache, heads
        self.scale = cache.head_dim ** -0.5 if scale is None else float(scale)
        with torch.cuda.device(cache.k.device):
            sms = device_sms()
        desc = B.cbs_attn_desc(batch, max_new, max_len, heads, cache.kv_heads, cache.head_dim, cache.prec, int(causal),
                               window, sms, force_kernel, force_split)
        self.plan = B.cbs_attn_plan(desc)
        self._plan_at = ctypes.addressof(self.plan)
        self._make_workspace()

    def _make_workspace(self):
        self.workspace_bytes, zeroed = int(self.plan.workspace_bytes), self._zeroed_bytes()
        self.workspace, self._stream = None, 0
        if self.workspace_bytes:
            with torch.cuda.device(self.cache.k.device):
                self.workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device="cuda")
                self._stream = current_stream()
                B.cbs_workspace_init(self.workspace, zeroed, self._stream)
                # Zeroed before anyone can use it on another stream.  (Within a capture
                # the zeroing is part of the graph, and what follows it is ordered.)
                if not torch.cuda.is_current_stream_capturing():
                    torch.cuda.current_stream().synchronize()

    def _zeroed_bytes(self) -> int:
        return int(self.plan.workspace_bytes)

    def fork(self):
        """The same plan and cache with a workspace of its own."""
        twin = object.__new__(type(self))
        twin.__dict__.update(self.__dict__)
        twin._make_workspace()
        return twin

    def __call__(self, q: torch.Tensor, new_start: torch.Tensor, seq_lens: torch.Tensor, page_table: torch.Tensor,
                 out: torch.Tensor | None = None) -> torch.Tensor:
        """q: bfloat16 [tokens, heads, head_dim] (a slice of a fused product's
        rows does).  The cache already holds the new tokens."""
        return _done(_calls().attention(self._plan_at, *self.cache._at, q, new_start, seq_lens, page_table, self.scale, out,
                                        self.workspace, self._stream), "cbs_paged_attention")


class WeighedAttention(PagedAttention):
    """PagedAttention that also adds up the weight each position of the cache
    receives, for PagedCache.evict.  Lengths are at most max_len."""

    def __init__(self, cache: PagedCache, batch: int, max_new: int, max_len: int, heads: int, causal: bool = True,
                 window: int = 0, scale: float | None = None, force_kernel: int = -1, force_split: int = 0):
        self.cache, self.heads = cache, heads
        self.scale = cache.head_dim ** -0.5 if scale is None else float(scale)
        with torch.cuda.device(cache.k.device):
            sms = device_sms()
        self.plan = B.cbs_weighed_plan(B.cbs_attn_desc(batch, max_new, max_len, heads, cache.kv_heads, cache.head_dim, cache.prec,
                                                       int(causal), window, sms, force_kernel, force_split))
        self._plan_at = ctypes.addressof(self.plan)
        self._make_workspace()

    def _zeroed_bytes(self) -> int:
        return int(self.plan.attention.workspace_bytes)

    def __call__(self, q: torch.Tensor, new_start: torch.Tensor, seq_lens: torch.Tensor, page_table: torch.Tensor,
                 mass: torch.Tensor, decay: float = 1.0, out: torch.Tensor | None = None) -> torch.Tensor:
        """As PagedAttention, and mass (float32 [num_pages, kv_heads, page_size])
        becomes decay * mass plus the softmax weights that the call's tokens gave each
        position, summed over the query heads of its key head; positions that are new
        in the call count from zero."""
        return _done(_calls().weighed_attention(self._plan_at, *self.cache._at, q, new_start, seq_lens, page_table, self.scale, out,
                                                self.workspace, self._stream, mass, decay), "cbs_weighed_attention")


class SharedPrefixAttention(PagedAttention):
    """Attention of sequences that go on from prefixes which groups of them share
    (several answers about one image, streams with one instruction): a prefix's
    keys and values are read once for its group.  Workspaces and `fork` as
    PagedAttention's."""

    def __init__(self, cache: PagedCache, batch: int, groups: int, max_new: int, max_len: int, max_prefix: int, heads: int,
                 max_group_new: int | None = None, scale: float | None = None):
        self.cache, self.heads = cache, heads
        self.scale = cache.head_dim ** -0.5 if scale is None else float(scale)
        with torch.cuda.device(cache.k.device):
            sms = device_sms()
        if max_group_new is None:
            max_group_new = batch * max_new
        self.plan = B.cbs_shared_plan(B.cbs_shared_desc(batch, groups, max_new, max_group_new, max_len, max_prefix, heads,
                                                        cache.kv_heads, cache.head_dim, cache.prec, sms))
        self._plan_at = ctypes.addressof(self.plan)
        self._make_workspace()

    def _zeroed_bytes(self) -> int:
        return int(self.plan.zeroed_bytes)

    def __call__(self, q: torch.Tensor, new_start: torch.Tensor, seq_lens: torch.Tensor, page_table: torch.Tensor,
                 group_start: torch.Tensor, prefix_lens: torch.Tensor, prefix_table: torch.Tensor,
                 out: torch.Tensor | None = None) -> torch.Tensor:
        """q: bfloat16 [tokens, heads, head_dim].  Sequences group_start[g] to
        group_start[g + 1] - 1 share prefix_lens[g] positions in prefix_table[g]'s
        pages; seq_lens and page_table are their own, behind it.  A new token sees its
        whole prefix, and its own sequence up to itself."""
        return _done(_calls().shared_attention(self._plan_at, *self.cache._at, q, new_start, seq_lens, page_table, self.scale, out,
                                               self.workspace, self._stream, group_start, prefix_lens, prefix_table),
                     "cbs_shared_attention")
