"""Embedding, head norms and dropout past 2^32 elements and bytes: offsets, launches
of many work-groups, strides that reach far."""
import pytest
import torch

import layers_reference as ref
from bit_adamw_update_amd import layers

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _memory():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def test_results_of_an_embedding_past_32_bits():
    tokens, cols = (1 << 21) + 3, 2056   # 4.3 G elements
    table = torch.randn(50, cols, device=DEV).to(BF)
    ids = torch.arange(tokens, device=DEV) % 50
    y = layers.embedding(ids, table)
    for at in (0, 1, tokens // 2, tokens - 2):
        assert torch.equal(y[at:at + 2], table[ids[at:at + 2]])
    # all rows, a slice of columns at a time
    assert bool((y.view(tokens, cols)[:, -8:] == table[ids][:, -8:]).all())


def test_gradients_of_many_tokens_past_32_bits():
    tokens, cols = (1 << 21) + 3, 2056
    dy = torch.ones(tokens, cols, dtype=BF, device=DEV)
    dy[tokens - 1] = 3
    ids = torch.full((tokens,), 7, device=DEV)
    ids[: 1 << 20] = 2
    ids[tokens - 1] = 4
    g = layers.embedding_grad(ids, dy, 9, dtype=torch.float32)
    # whole numbers below 2^24: every sum of them is exact
    want = torch.zeros(9, cols, device=DEV)
    want[2], want[7], want[4] = 1 << 20, tokens - 1 - (1 << 20), 3
    assert torch.equal(g, want)


def test_heads_that_lie_far_apart():
    far = (1 << 31) + 64
    buf = torch.zeros(2 * far + 4096, dtype=BF, device=DEV)
    q = buf.as_strided((3, 2, 64), (far, 128, 1))
    k = buf.as_strided((3, 2, 64), (64, far, 1), 1024)
    q.copy_(torch.randn(3, 2, 64)), k.copy_(torch.randn(3, 2, 64))
    gain, pos, f = torch.rand(64, device=DEV) + 0.5, torch.arange(3, device=DEV), layers.rope_frequencies(64)
    args = gain, gain, pos, f
    near = layers.head_norm_rope(q.contiguous(), k.contiguous(), *args)
    dq, dk = torch.randn(3, 2, 64, device=DEV).to(BF), torch.randn(3, 2, 64, device=DEV).to(BF)
    grads = layers.head_norm_rope_backward(q.contiguous(), k.contiguous(), *args, dq, dk)
    for a, b in zip(grads, layers.head_norm_rope_backward(q, k, *args, dq, dk)):
        assert torch.equal(a, b)
    for a, b in zip(near, layers.head_norm_rope(q, k, *args)):
        assert torch.equal(a, b)
    for a, b in zip(near, layers.head_norm_rope(q, k, *args, out=(q, k))):
        assert torch.equal(a, b)


def test_many_short_heads():
    tokens = (1 << 28) + 5   # work-groups in several rows of a launch
    q = torch.ones(tokens, 1, 2, dtype=BF, device=DEV)
    k = torch.ones(tokens, 1, 2, dtype=BF, device=DEV)
    q[-1] = torch.tensor([3.0, 4.0])
    one, f = torch.ones(2, device=DEV), layers.rope_frequencies(2)
    pos = torch.zeros(1, dtype=torch.int32, device=DEV).expand(tokens)
    layers.head_norm_rope(q, k, one, one, pos, f, out=(q, k))
    assert bool((q[:-1].view(-1) == 1).all()) and bool((k.view(-1) == 1).all())
    want = ref.head_norm_rope(torch.tensor([[[3.0, 4.0]]]), one, pos[-1:], f, 1e-6, False)
    assert torch.allclose(q[-1:].double().cpu(), want, rtol=2.0 ** -8)
    got = layers.head_norm_rope_backward(k, k, one, one, pos, f, q, k, dtype=torch.float32)
    # of equal elements n = 1: dn - n mean(dn n) = 0, and each gain's element gets the sum over the tokens
    assert bool((got[1].view(-1).float().abs() <= 2e-6).all())
    assert abs(float(got[3][0]) / tokens - 1) <= 2e-6


def test_dropout_past_32_bits():
    rows, cols = (1 << 21) + 1, 2056
    x = torch.ones(rows, cols, dtype=BF, device=DEV)
    y = layers.dropout(x, 0.25, 11, 5, 3, out=x)
    for at in (0, 1 << 20, rows - 3):
        part = layers.dropout(torch.ones(3, cols, dtype=BF, device=DEV), 0.25, 11, 5, 3, offset=at * cols)
        assert torch.equal(y[at:at + 3], part)
    kept = ref.dropout(torch.ones(1, cols), 0.25, 11, 5, 3, offset=(rows - 1) * cols)[1]
    assert torch.equal(y[-1].cpu() != 0, kept[0])
