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

The weights are random: there is nothing to learn here, only to run.  PyTorch
looks up embeddings, picks the largest logit and holds the buffers; a step of
one token each is captured in a CUDA graph, whose launches all read the same
buffers.
"""
from __future__ import annotations

import argparse

import torch

from . import _binding as B
from .tokens import LinearW4, PagedAttention, PagedCache, dequantize_rows, rmsnorm

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


def main():
    from .chain import Chain
    parser = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    parser.add_argument("--images", type=int, default=4)
    parser.add_argument("--tokens", type=int, default=32)
    args = parser.parse_args()
    chain = Chain("bf16", args.images)
    frame = torch.randn((args.images, 3, 640, 640), device="cuda")
    head = TokenHead(args.images)
    start, seen, done = (torch.cuda.Event(enable_timing=True) for _ in range(3))
    for _ in range(3):
        start.record()
        cells = chain.run(frame)[-1]   # [images, 20, 20, 256]
        seen.record()
        answer = head.answer(cells, args.tokens)
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
