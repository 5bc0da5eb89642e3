"""A small token head over the chain's deepest feature map, built of the token
operators: each image's 20x20 cells are a prefix that answers attend to, and
the answer follows token by token (greedily).

    python -m conv_bn_silu_gb300.token_head [--images 4] [--tokens 32]

One layer, for a prefix as for one new token:

    h, y8   = rmsnorm(h + delta)                 sum, norm and 8-bit rows in one pass
    q, k, v = qkv(y8)                            4-bit weights
    cache.write(k, v)                            8-bit pages
    a       = attention(q)                       over the sequence's pages
    h, y8   = rmsnorm(h + out(a))
    delta   = down(silu(up(y8)))

`AnswerHead` gives several answers about each image: the cells go through 8-bit
products, a row's weight for the others is added up while they attend to one another,
and the heaviest of them stay as the one prefix that all of an image's answers share.

    python -m conv_bn_silu_gb300.token_head --answers 6 [--keep 100]

The weights are random: there is nothing to learn here, only to run.  PyTorch
looks up embeddings, picks the largest logit and holds the buffers; a step of
one token each is captured in a CUDA graph, whose launches all read the same
buffers.
"""
from __future__ import annotations

import argparse

import torch

from . import _binding as B
from .tokens import (LinearW4, LinearW8, PagedAttention, PagedCache, SharedPrefixAttention, WeighedAttention, dequantize_rows,
                     rmsnorm)

EPS = 1e-5


class Layer:
    def __init__(self, width, heads, kv_heads, head_dim, hidden, weights):
        q_width, kv_width = heads * head_dim, kv_heads * head_dim
        self.norm1, self.norm2 = weights.norm(width), weights.norm(width)
        self.qkv = weights.linear(q_width + 2 * kv_width, width)
        self.out = weights.linear(width, q_width)
        self.up = weights.linear(hidden, width, activation=B.CBS_ACT_SILU)
        self.down = weights.linear(width, hidden)


class _Weights:
    """Random weights of unit gain."""

    def __init__(self, seed, device):
        self.g, self.device = torch.Generator(device).manual_seed(seed), device

    def normal(self, *shape):
        return torch.randn(shape, device=self.device, generator=self.g)

    def norm(self, width):
        return 1 + 0.1 * self.normal(width)

    def linear(self, n, k, activation=B.CBS_ACT_IDENTITY):
        return LinearW4.quantize(self.normal(n, k) * k ** -0.5, group=64, activation=activation)


class TokenHead:
    """batch sequences of up to max_len positions over prefixes of `cells`."""

    def __init__(self, batch: int, cells: int = 400, width: int = 256, max_len: int = 512, layers: int = 2, heads: int = 8,
                 kv_heads: int = 2, head_dim: int = 64, hidden: int = 1024, vocabulary: int = 512, page: int = 16,
                 seed: int = 0, device="cuda"):
        if cells < 1 or cells >= max_len:
            raise ValueError(f"{cells} cells leave no room in {max_len} positions")
        weights = _Weights(seed, device)
        self.batch, self.cells, self.max_len, self.heads, self.kv_heads, self.head_dim = batch, cells, max_len, heads, kv_heads, head_dim
        self.layers = [Layer(width, heads, kv_heads, head_dim, hidden, weights) for _ in range(layers)]
        self.norm, self.logits_of = weights.norm(width), weights.linear(vocabulary, width)
        self.embedding = weights.normal(vocabulary, width).to(torch.bfloat16)
        pages = -(-max_len // page)
        self.page_table = torch.arange(batch * pages, dtype=torch.int32, device=device).view(batch, pages)
        self.seq_lens = torch.zeros(batch, dtype=torch.int32, device=device)
        self.caches = [PagedCache.empty(batch * pages, kv_heads, page, head_dim, device=device) for _ in self.layers]
        # The cells of a map see one another; an answer's token sees all before it.
        self.prefix = self._attentions(cells, cells, causal=False)
        self.single = self._attentions(1, max_len, causal=True)
        self.starts = {n: torch.arange(0, batch * n + 1, n, dtype=torch.int32, device=device) for n in (1, cells)}
        self.token = torch.zeros(batch, dtype=torch.int64, device=device)
        self.graph = None

    def _attentions(self, max_new, max_len, causal):
        return [PagedAttention(c, self.batch, max_new, max_len, self.heads, causal=causal) for c in self.caches]

    def _run(self, h, attentions, new):
        """The layers over `new` tokens of each sequence (rows of h, in order);
        the logits of each sequence's last one."""
        starts, delta = self.starts[new], None
        for layer, cache, attention in zip(self.layers, self.caches, attentions):
            y, scale, h = rmsnorm(h, layer.norm1, EPS, residual=delta, int8=True)
            qkv = layer.qkv(y, scale).view(-1, self.heads + 2 * self.kv_heads, self.head_dim)
            q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), dim=1)
            cache.write(k, v, starts, self.seq_lens, self.page_table)
            a = attention(q, starts, self.seq_lens, self.page_table)
            y, scale, h = rmsnorm(h, layer.norm2, EPS, residual=layer.out(a.flatten(1)), int8=True)
            delta = layer.down(layer.up(y, scale))
        if new > 1:
            h, delta = h[new - 1::new].contiguous(), delta[new - 1::new].contiguous()
        self.answer_rows = rmsnorm(h, self.norm, EPS, residual=delta, int8=True)
        return self.logits_of(self.answer_rows.y, self.answer_rows.scale, dtype=torch.float32)

    def start(self, cells: torch.Tensor) -> torch.Tensor:
        """The prefixes (bfloat16 [batch, ..., width], their cells in order)
        into the caches; the logits after each one's last cell."""
        h = cells.reshape(-1, cells.shape[-1])
        if h.shape[0] != self.batch * self.cells:
            raise ValueError(f"{h.shape[0]} cells for {self.batch} prefixes of {self.cells}")
        self.seq_lens.fill_(self.cells)
        return self._run(h, self.prefix, self.cells)

    def step(self, token: torch.Tensor) -> torch.Tensor:
        """One token (int64) of each sequence; the logits that follow it."""
        self.seq_lens += 1
        return self._run(self.embedding[token], self.single, 1)

    def _advance(self):
        self.token.copy_(self.step(self.token).argmax(1))

    def answer(self, cells: torch.Tensor, tokens: int) -> torch.Tensor:
        """The next `tokens` tokens of each sequence, int64 [batch, tokens]."""
        if tokens < 1 or self.cells + tokens - 1 > self.max_len:
            raise ValueError(f"{tokens} tokens after {self.cells} cells: at most {self.max_len} positions")
        if self.graph is None:
            self.start(cells)
            self._advance()   # (everything a launch needs is set up before a capture)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                self._advance()
            self.graph = graph
            self.step_rows = self.answer_rows   # the buffers that each launch writes
        out = torch.empty((self.batch, tokens), dtype=torch.int64, device=self.token.device)
        self.token.copy_(self.start(cells).argmax(1))
        out[:, 0] = self.token
        for i in range(1, tokens):
            self.graph.replay()
            out[:, i] = self.token
        if tokens > 1:
            self.answer_rows = self.step_rows
        return out

    def features(self) -> torch.Tensor:
        """What the last logits were made of: float32 [batch, width]."""
        return dequantize_rows(self.answer_rows.y, self.answer_rows.scale, torch.float32)

    def history(self, layer: int):
        """A layer's keys and values in order, [batch, max_len, kv_heads, head_dim]."""
        return self.caches[layer].read(self.seq_lens, self.page_table, self.max_len)


class AnswerLayer:
    """As Layer; products whose inputs are 8-bit rows have 8-bit weights, for a
    prefix's thousands of rows as for an answer's token."""

    def __init__(self, width, heads, kv_heads, head_dim, hidden, weights):
        q_width, kv_width = heads * head_dim, kv_heads * head_dim
        self.norm1, self.norm2 = weights.norm(width), weights.norm(width)
        self.qkv = LinearW8.quantize(weights.normal(q_width + 2 * kv_width, width) * width ** -0.5)
        self.out = weights.linear(width, q_width)
        self.up = LinearW8.quantize(weights.normal(hidden, width) * width ** -0.5, activation=B.CBS_ACT_SILU)
        self.down = weights.linear(width, hidden)


class AnswerHead:
    """`answers` sequences of up to max_answer tokens about each of `images`, over
    the `keep` cells of the image's prefix that the others looked at most (each
    key head's own choice)."""

    def __init__(self, images: int, answers: int, cells: int = 400, keep: int = 100, width: int = 256, max_answer: int = 64,
                 layers: int = 2, heads: int = 8, kv_heads: int = 2, head_dim: int = 64, hidden: int = 1024, vocabulary: int = 512,
                 page: int = 16, seed: int = 0, device="cuda"):
        if images < 1 or answers < 1 or cells < 1 or max_answer < 1 or not 1 <= keep <= cells:
            raise ValueError(f"{answers} answers of {max_answer} about {images} images of {cells} cells, {keep} kept")
        weights = _Weights(seed, device)
        self.images, self.answers, self.cells, self.keep, self.max_answer = images, answers, cells, keep, max_answer
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.layers = [AnswerLayer(width, heads, kv_heads, head_dim, hidden, weights) for _ in range(layers)]
        self.norm, self.logits_of = weights.norm(width), LinearW8.quantize(weights.normal(vocabulary, width) * width ** -0.5)
        self.embedding = weights.normal(vocabulary, width).to(torch.bfloat16)
        # Pages: the images' cells, what of them stays, the answers' own tokens.
        batch = images * answers
        counts = [(images, -(-cells // page)), (images, -(-keep // page)), (batch, -(-max_answer // page))]
        tables, first = [], 0
        for rows, pages in counts:
            tables.append(torch.arange(first, first + rows * pages, dtype=torch.int32, device=device).view(rows, pages))
            first += rows * pages
        self.cell_table, self.prefix_table, self.page_table = tables
        int32 = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=device)   # noqa: E731
        self.cell_lens = int32(images) + cells
        self.prefix_lens, self.seq_lens = int32(images) + keep, int32(batch)
        self.cell_starts = torch.arange(0, images * cells + 1, cells, dtype=torch.int32, device=device)
        self.starts = torch.arange(batch + 1, dtype=torch.int32, device=device)
        self.group_start = torch.arange(0, batch + 1, answers, dtype=torch.int32, device=device)
        self.caches = [PagedCache.empty(first, kv_heads, page, head_dim, device=device) for _ in self.layers]
        self.mass = torch.zeros((first, kv_heads, page), device=device)
        self.prefix = [WeighedAttention(c, images, cells, cells, heads, causal=False) for c in self.caches]
        self.single = [SharedPrefixAttention(c, batch, images, 1, max_answer, keep, heads, max_group_new=answers) for c in self.caches]
        self.kept = [None] * layers
        self.token = torch.zeros(batch, dtype=torch.int64, device=device)
        self.graph = None

    def _run(self, h, attend):
        delta = None
        for i, layer in enumerate(self.layers):
            y, scale, h = rmsnorm(h, layer.norm1, EPS, residual=delta, int8=True)
            qkv = layer.qkv(y, scale).view(-1, self.heads + 2 * self.kv_heads, self.head_dim)
            a = attend(i, *qkv.split((self.heads, self.kv_heads, self.kv_heads), dim=1))
            y, scale, h = rmsnorm(h, layer.norm2, EPS, residual=layer.out(a.flatten(1)), int8=True)
            delta = layer.down(layer.up(y, scale))
        return h, delta

    def start(self, cells: torch.Tensor):
        """The images' cells (bfloat16 [images, ..., width]) into the caches, and
        what stays of them into the prefixes."""
        h = cells.reshape(-1, cells.shape[-1])
        if h.shape[0] != self.images * self.cells:
            raise ValueError(f"{h.shape[0]} cells for {self.images} images of {self.cells}")

        def attend(i, q, k, v):
            cache = self.caches[i]
            cache.write(k, v, self.cell_starts, self.cell_lens, self.cell_table)
            a = self.prefix[i](q, self.cell_starts, self.cell_lens, self.cell_table, self.mass, decay=0.0)
            self.kept[i], _ = cache.evict(self.mass, self.cell_lens, self.cell_table, self.prefix_table, self.keep)
            return a
        self._run(h, attend)
        self.seq_lens.zero_()

    def step(self, token: torch.Tensor) -> torch.Tensor:
        """One token (int64 [images * answers]) of each answer; the logits that
        follow it."""
        self.seq_lens += 1

        def attend(i, q, k, v):
            self.caches[i].write(k, v, self.starts, self.seq_lens, self.page_table)
            return self.single[i](q, self.starts, self.seq_lens, self.page_table, self.group_start, self.prefix_lens, self.prefix_table)
        h, delta = self._run(self.embedding[token], attend)
        y, scale, _ = rmsnorm(h, self.norm, EPS, residual=delta, int8=True)
        return self.logits_of(y, scale, dtype=torch.float32)

    def _advance(self):
        self.token.copy_(self.step(self.token).argmax(1))

    def answer(self, cells: torch.Tensor, first: torch.Tensor, tokens: int) -> torch.Tensor:
        """The `tokens` tokens that follow each answer's first one (int64 [images,
        answers], what it is asked), int64 [images, answers, tokens]."""
        if tokens < 1 or tokens > self.max_answer:
            raise ValueError(f"{tokens} tokens: at most {self.max_answer}")
        if first.numel() != self.images * self.answers:
            raise ValueError(f"{first.numel()} first tokens for {self.images} images of {self.answers} answers")
        self.start(cells)
        if self.graph is None:
            self._advance()   # (everything a launch needs is set up before a capture)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                self._advance()
            self.graph = graph
            self.seq_lens.zero_()
        self.token.copy_(first.reshape(-1))
        out = torch.empty((self.images * self.answers, tokens), dtype=torch.int64, device=self.token.device)
        for i in range(tokens):
            self.graph.replay()
            out[:, i] = self.token
        return out.view(self.images, self.answers, tokens)


def main():
    from .chain import Chain
    parser = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    parser.add_argument("--images", type=int, default=4)
    parser.add_argument("--tokens", type=int, default=32)
    parser.add_argument("--answers", type=int, default=0, help="answers about each image (0: one, over the whole prefix)")
    parser.add_argument("--keep", type=int, default=100, help="cells of an image that its answers see")
    args = parser.parse_args()
    chain = Chain("bf16", args.images)
    frame = torch.randn((args.images, 3, 640, 640), device="cuda")
    head = AnswerHead(args.images, args.answers, keep=args.keep, max_answer=args.tokens) if args.answers else TokenHead(args.images)
    first = torch.arange(args.images * args.answers, device="cuda").view(args.images, args.answers) if args.answers else None
    start, seen, done = (torch.cuda.Event(enable_timing=True) for _ in range(3))
    for _ in range(3):
        start.record()
        cells = chain.run(frame)[-1]   # [images, 20, 20, 256]
        seen.record()
        answer = head.answer(cells, first % 512, args.tokens).flatten(0, 1) if args.answers else head.answer(cells, args.tokens)
        done.record()
    torch.cuda.synchronize()
    status = B.cbs_read_device_status(True, torch.cuda.current_stream().cuda_stream)
    if status != B.CBS_OK:
        raise RuntimeError(f"a kernel reported {B.status_name(status)}")
    print(f"{args.images} frames {start.elapsed_time(seen):.3f} ms, {args.tokens} tokens each {seen.elapsed_time(done):.3f} ms")
    for row in answer.tolist():
        print(*row)


if __name__ == "__main__":
    main()
