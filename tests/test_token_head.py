"""The token operators run together: a small head over feature maps."""
import pytest
import torch

from conv_bn_silu_gb300 import _binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def token_calls(cuda_lib):
    from conv_bn_silu_gb300 import build
    build.build_tokens()


def weights_of(layer):
    """A 4-bit layer's weights in 64 bits."""
    b = layer.packed.view(layer.n, layer.k // 8, 4).long()
    low, high = b & 15, b >> 4
    nibbles = torch.stack([low, high], -1).view(layer.n, layer.k // 8, 8)
    codes = nibbles[..., [0, 4, 1, 5, 2, 6, 3, 7]].reshape(layer.n, layer.k)
    zero = 8 if layer.zeros is None else layer.zeros.t().repeat_interleave(layer.group, 1).double()
    return (codes.double() - zero) * layer.scales.t().double().repeat_interleave(layer.group, 1)


def plain(head, cells, answer):
    """The logits after the prefix and each token of `answer`, in 64 bits and
    without 8-bit rows or caches: [batch, 1 + tokens, vocabulary]."""
    batch, n = head.batch, head.cells
    h = torch.cat([cells.reshape(batch, n, -1).double(), head.embedding[answer].double()], 1)
    total, group = h.shape[1], head.heads // head.kv_heads
    at = torch.arange(total, device=h.device)
    seen = (at[None] < n) | (at[None] <= at[:, None])

    def norm(x, w):
        return x * w.double() / (x.square().mean(-1, keepdim=True) + 1e-5).sqrt()

    for layer in head.layers:
        qkv = (norm(h, layer.norm1) @ weights_of(layer.qkv).t()).view(batch, total, -1, head.head_dim).transpose(1, 2)
        q, k, v = qkv.split((head.heads, head.kv_heads, head.kv_heads), 1)
        k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
        scores = (q @ k.transpose(2, 3) * head.head_dim ** -0.5).masked_fill(~seen, float("-inf"))
        a = (scores.softmax(-1) @ v).transpose(1, 2).flatten(2)
        h = h + a @ weights_of(layer.out).t()
        h = h + torch.nn.functional.silu(norm(h, layer.norm2) @ weights_of(layer.up).t()) @ weights_of(layer.down).t()
    return norm(h[:, n - 1:], head.norm) @ weights_of(head.logits_of).t()


def test_an_answer_follows_the_plain_model(cuda_lib):
    """8-bit rows and caches move a product's result by about 0.7% of its size
    (a largest value of three standard deviations in 127 steps), five times a
    layer and once at the end, besides bfloat16's 0.2%: 2.4% together for two
    layers.  Four times that is the bound on the logits' relative error."""
    from conv_bn_silu_gb300.token_head import TokenHead
    batch, tokens = 3, 5
    head = TokenHead(batch, cells=100, max_len=112, seed=3)
    cells = torch.randn((batch, 10, 10, 256), dtype=torch.bfloat16, device="cuda",
                        generator=torch.Generator("cuda").manual_seed(4))
    logits = [head.start(cells)]
    answer = []
    for _ in range(tokens):
        answer.append(logits[-1].argmax(1))
        logits.append(head.step(answer[-1]))
    got = torch.stack(logits, 1).double()
    ref = plain(head, cells, torch.stack(answer, 1))
    err = (got - ref).norm(dim=-1) / ref.norm(dim=-1)
    assert (err <= 0.1).all(), err
    assert B.cbs_read_device_status(True, torch.cuda.current_stream().cuda_stream) == B.CBS_OK

    # The same tokens through the captured step, and what it leaves behind.
    assert torch.equal(head.answer(cells, tokens), torch.stack(answer, 1))
    assert head.seq_lens.tolist() == [100 + tokens - 1] * batch
    assert head.features().shape == (batch, 256) and head.features().isfinite().all()
    keys, values = head.history(0)
    assert keys.shape == (batch, 112, 2, 64) and keys[:, :104].float().norm(dim=-1).min() > 0
    assert not keys[:, 104:].any() and not values[:, 104:].any()


def test_a_head_over_the_chain(cuda_lib):
    from conv_bn_silu_gb300.chain import Chain
    from conv_bn_silu_gb300.token_head import TokenHead
    chain, head = Chain("bf16", 2), TokenHead(2)
    frame = torch.randn((2, 3, 640, 640), device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    first = head.answer(chain.run(frame)[-1], 8)
    again = head.answer(chain.run(frame)[-1], 8)
    assert torch.equal(first, again) and first.shape == (2, 8)
    with pytest.raises(ValueError):
        head.answer(chain.outs[-1], 200)
    with pytest.raises(ValueError):
        head.start(chain.outs[-1][:1])


def test_a_capture_that_fails_leaves_no_graph(cuda_lib):
    from conv_bn_silu_gb300.token_head import TokenHead
    head = TokenHead(2, cells=20, max_len=32, layers=1)
    cells = torch.randn((2, 20, 256), dtype=torch.bfloat16, device="cuda", generator=torch.Generator("cuda").manual_seed(6))
    step, calls = head.step, []

    def failing(token):
        calls.append(torch.cuda.is_current_stream_capturing())
        if calls[-1]:
            raise KeyboardInterrupt
        return step(token)
    head.step = failing
    with pytest.raises(KeyboardInterrupt):
        head.answer(cells, 4)
    assert calls == [False, True] and head.graph is None
    head.step = step
    answer = head.answer(cells, 4)
    assert torch.equal(answer, TokenHead(2, cells=20, max_len=32, layers=1).answer(cells, 4))
