"""Forms of embedding, head norms and dropout that test_layers_gpu.py's sizes do
not reach, with its tolerances."""
import pytest
import torch

from bit_adamw_update_amd import api, layers
from test_layers_gpu import (BF, DEV, F32, _check_back, _check_grad, _check_heads, _drawn, _heads_case, _laid, _normal,
                             _say)

pytestmark = pytest.mark.gpu


# ---- head norms -----------------------------------------------------------------

@pytest.mark.parametrize("layout,batch", [("split", None), ("by head", 3), ("gaps", 3)])
def test_gradients_in_the_place_of_the_inputs(layout, batch):
    tokens = 601   # several rows to a lane
    q, k, gq, gk, pos, f, how = case = _heads_case(tokens, 4, 2, 64, 64, False, layout, 300, batch=batch)
    dq, dk = _laid(tokens, 4, 64, "split", 301, batch), _laid(tokens, 2, 64, layout, 302, batch)
    want = _check_back(*case, dq, dk)
    got = layers.head_norm_rope_backward(q, k, gq.to(DEV), gk.to(DEV), pos.to(DEV), f, dq, dk, out=(q, k), **how)
    assert got[0] is q and got[1] is k
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("tokens,hq,hk,dim,rotary", [(701, 8, 4, 130, 130), (701, 8, 4, 514, 258), (1, 70, 9, 130, 66),
                                                     (1, 70, 1, 1022, 1022), (350, 3, 5, 258, 0)])
def test_several_rows_of_single_pairs(tokens, hq, hk, dim, rotary, inter):
    """Heads of more than 64 pairs that no vector divides: eight pairs to a lane, a wave to a row, several rows to a wave."""
    _say("heads", tokens, hq, hk, dim, rotary, inter)
    case = _heads_case(tokens, hq, hk, dim, rotary, inter, "split", 310)
    _check_heads(*case)
    dq, dk = _laid(tokens, hq, dim, "split", 311), _laid(tokens, hk, dim, "split", 312)
    _check_back(*case, dq, dk)
    _check_back(*case, dq, dk, dtype=F32)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim,rotary", [(64, 64), (80, 80), (10, 6)])
@pytest.mark.parametrize("layout,shared", [("by head", False), ("split", True), ("gaps", True)])
def test_batches_of_many_tokens(layout, shared, dim, rotary, inter):
    """Batches that do not follow each other (by their strides, or by positions that they share): several tokens to a
    work-group, the last of each batch with fewer."""
    _say("batches", layout, shared, dim, rotary, inter)
    q, k, gq, gk, pos, f, how = _heads_case(1501, 2, 1, dim, rotary, inter, layout, 320, batch=3)
    if shared:
        pos = pos[:1].expand(3, 1501)
    _check_heads(q, k, gq, gk, pos, f, how)
    dq, dk = _laid(1501, 2, dim, layout, 321, 3), _laid(1501, 1, dim, "split", 322, 3)
    _check_back(q, k, gq, gk, pos, f, how, dq, dk, dtype=F32)


def test_gradients_of_zero_rows():
    """1 / sqrt(eps) = 1000 times what comes in: FP32 is off by few of its steps, far less than half of BF16's 4."""
    q, k = torch.zeros(5, 2, 64, dtype=BF, device=DEV), torch.full((5, 1, 64), 1e-30, dtype=BF, device=DEV)
    one, pos, f = torch.ones(64, device=DEV), torch.zeros(5, dtype=torch.int64, device=DEV), layers.rope_frequencies(64)
    dq, dk, gq, gk = layers.head_norm_rope_backward(q, k, one, one, pos, f, torch.ones_like(q), -torch.ones_like(k),
                                                    dtype=F32)
    assert bool((dq == 1000).all()) and bool((dk == -1000).all()) and bool((gq == 0).all())
    # five tokens' n = 1000 x each
    want = -5 * 1000 * float(k[0, 0, 0])
    assert bool(((gk.double() - want).abs() <= 16 * 2.0 ** -24 * abs(want)).all())


# ---- the table's gradient: few tokens in the form of several launches ----------------
# A table of more than 8 MB, or columns that take more than 256 work-groups, is not for the form in one launch.

@pytest.mark.parametrize("how", ["same", "text", "falling", "none", "padded"])
@pytest.mark.parametrize("tokens", [1, 2, 31, 32, 33, 64, 65, 97, 1000, 1024])
def test_embedding_grad_of_few_tokens_into_a_large_table(tokens, how):
    _say("few into large", tokens, how)
    ids, dy = _drawn(how, tokens, 9000, tokens), _normal(tokens, 512, seed=tokens)
    _check_grad(ids, dy, 9000, 1.0, BF)
    _check_grad(ids.to(torch.int32), dy, 9000, 0.3125, F32)


@pytest.mark.parametrize("rows,cols", [(700_000, 7), (9000, 513)])
def test_embedding_grad_of_few_tokens_into_a_large_table_of_odd_columns(rows, cols):
    for tokens, how in ((1, "same"), (33, "same"), (97, "text")):
        ids, dy = _drawn(how, tokens, rows, 331), _normal(tokens, cols, seed=332)
        _check_grad(ids, dy, rows, -0.5, BF)


@pytest.mark.parametrize("tokens,cols", [(1, 131600), (32, 131600), (33, 66000), (97, 33300), (300, 13320)])
def test_embedding_grad_of_few_tokens_of_very_many_columns(tokens, cols):
    for how in ("same", "text", "padded"):
        ids, dy = _drawn(how, tokens, 6, 333), _normal(tokens, cols, seed=334)
        _check_grad(ids, dy, 6, 1.0, BF)
        start = _normal(6, cols, seed=335)
        _check_grad(ids, dy, 6, 0.5, F32, start, out=start.float().to(DEV), accumulate=True)


# ---- the same in graphs, on streams, two at once --------------------------------------
# Each takes its workspace: runs that are merged, a sort that needs no merges beside a large table's fill, two merges,
# few tokens into a large table.  Rows of more than 32 tokens are joined from it.
SEVERAL = {"merged": (5000, 300, 72), "ranked": (3000, 60000, 320), "merged twice": (20000, 500, 40),
           "few into large": (1000, 9000, 512)}


def _several(which, seed):
    tokens, rows, cols = SEVERAL[which]
    ids = _drawn("text", tokens, rows, seed).to(DEV)
    assert int(torch.bincount(ids).max()) > 32
    return [ids, _normal(tokens, cols, seed=seed + 1).to(DEV)], rows


def _grad(operands, rows, start=None, **kw):
    """The gradient, or with start added to it."""
    return layers.embedding_grad(*operands, rows, scale=0.5, out=start, accumulate=start is not None, **kw)


@pytest.mark.parametrize("which", SEVERAL)
def test_several_launches_captured_and_replayed(which):
    _say("graph", which)
    operands, rows = _several(which, 1)
    cols = operands[1].shape[1]
    start = _normal(rows, cols, seed=9, dtype=F32).to(DEV)
    added = start.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _grad(operands, rows)
        _grad(operands, rows, added)
    for seed in (2, 3, 2, 4):
        for o, n in zip(operands, _several(which, seed)[0]):
            o.copy_(n)
        added.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, _grad(operands, rows)), seed
        assert torch.equal(added, _grad(operands, rows, start.clone())), seed
        torch.cuda.synchronize()
    _check_grad(operands[0].cpu(), operands[1], rows, 0.5, BF)


@pytest.mark.parametrize("which", SEVERAL)
def test_several_launches_on_another_stream(which):
    _say("stream", which)
    operands, rows = _several(which, 5)
    start = _normal(rows, operands[1].shape[1], seed=9, dtype=F32).to(DEV)
    want, want_added = _grad(operands, rows), _grad(operands, rows, start.clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(10_000_000)
    got = _grad(operands, rows, stream=side)
    added = _grad(operands, rows, start, stream=side)
    assert added is start
    fresh = [o.clone() for o in operands]
    del operands
    for _ in range(3):   # the operands' and the workspaces' memory, were it not held
        [torch.empty_like(o).zero_() for o in fresh]
        torch.empty(1 << 22, dtype=torch.uint8, device=DEV).fill_(255)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want) and torch.equal(added, want_added)


@pytest.mark.parametrize("which", SEVERAL)
def test_several_launches_two_at_once(which):
    """Two calls on two streams, each with a workspace of its own."""
    calls = [_several(which, s) for s in (6, 7)]
    want = [_grad(*c) for c in calls]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[_grad(*c, stream=s) for c, s in zip(calls, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for run in got for a, b in zip(want, run))


@pytest.mark.parametrize("which", SEVERAL)
def test_workspaces_of_exactly_their_size(which):
    """What lies behind a workspace stays, whatever it held before."""
    (ids, dy), rows = _several(which, 8)
    tokens, cols = dy.shape
    want = _grad((ids, dy), rows)
    need = api.q4nn_embedding_grad_workspace_bytes(tokens, rows, cols)
    for byte in (0, 255):
        ws = torch.full((need + 4096,), byte, dtype=torch.uint8, device=DEV)
        got = torch.empty_like(want)
        api.q4nn_embedding_grad(ids, api.NN_I64, tokens, dy, cols, 0.5, rows, cols, got, api.MX_BF16, cols, 0, ws, need)
        assert torch.equal(got, want) and bool((ws[need:] == byte).all())


@pytest.mark.parametrize("tokens,hq,hk,dim,batch", [(1, 16, 8, 128, None), (701, 8, 4, 130, None), (1501, 2, 1, 80, 3)])
def test_workspaces_of_the_gains_gradients(tokens, hq, hk, dim, batch):
    q, k, gq, gk, pos, f, how = _heads_case(tokens, hq, hk, dim, dim, False, "by head" if batch else "split", 340, batch=batch)
    dq, dk = _laid(tokens, hq, dim, "split", 341, batch), _laid(tokens, hk, dim, "split", 342, batch)
    gq, gk, pos = gq.to(DEV), gk.to(DEV), pos.to(DEV)
    want = layers.head_norm_rope_backward(q, k, gq, gk, pos, f, dq, dk, **how)
    packed = [layers._heads(n, t) for n, t in (("q", q), ("k", k), ("dq", dq), ("dk", dk))]
    rope = layers._rope(q, k, gq, gk, pos, f, how["eps"], how["interleaved"])
    need = api.q4nn_head_norm_rope_backward_workspace_bytes(rope)
    for byte in (0, 255):
        ws = torch.full((need + 4096,), byte, dtype=torch.uint8, device=DEV)
        got = [torch.empty_like(w) for w in want]
        api.q4nn_head_norm_rope_backward(rope, *packed, layers._heads("dq", got[0]), layers._heads("dk", got[1]), got[2],
                                         got[3], api.MX_BF16, 0, ws, need)
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and bool((ws[need:] == byte).all())
