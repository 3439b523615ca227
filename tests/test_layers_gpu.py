"""Embedding, head norms with rotation, and dropout on the GPU against plain
64-bit implementations (layers_reference.py), at the sizes and values where
they can go wrong.

Tolerances.  A result's rounding is half a step of its type (2^-8 relative for
BF16, 2^-24 for FP32) of a value that FP32 arithmetic has moved before.  Lookups
and dropout round a product (and a scale, and a sum with the residual) in FP32:
3 half steps of its terms.  A row of the table's gradient is a sum of n BF16
values in FP32: at most n - 1 additions, each off by at most half a step of a
partial sum of at most the sum of magnitudes, and a product.  The bounds of
the head norms are written in layers_reference.py.
"""
import math

import pytest
import torch

import layers_reference as ref
from bit_adamw_update_amd import api, layers, mx

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, D = torch.bfloat16, torch.float32, torch.float64
S24 = 2.0 ** -24


def _say(*a):
    print(*a, flush=True)


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _normal(*shape, seed=0, dtype=BF, scale=1.0):
    return (torch.randn(*shape, generator=_gen(seed)) * scale).to(dtype)


def _strided(x, gap, shift, fill=7.0):
    """x (2-D) on the GPU with `gap` elements between rows, `shift` past an aligned address; (view, whole buffer)."""
    rows, cols = x.shape
    ld = cols + gap
    buf = torch.full((shift + rows * ld + 8,), fill, dtype=x.dtype, device=DEV)
    view = buf[shift:shift + rows * ld].view(rows, ld)[:, :cols]
    view.copy_(x)
    return view, buf


def _untouched(view, buf, fill=7.0):
    """Whether the buffer around the view still holds the fill."""
    inside = torch.zeros(buf.numel(), dtype=torch.bool, device=DEV)
    torch.as_strided(inside, view.shape, view.stride(), view.storage_offset()).fill_(True)
    return bool((buf[~inside] == fill).all())


def _close(got, want, moved, dtype):
    assert got.dtype == dtype
    got = got.to(D).cpu()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    tol = want.abs() * ref.HALF[dtype] + moved * (1 + ref.HALF[dtype]) + 1e-38   # and a value below the normal ones
    off = (got - want).abs()
    bad = ~(off <= tol) & ~nan
    assert not bool(bad.any()), (f"{int(bad.sum())} off, by at most {off[bad].max().item()}, first at "
                                 f"{tuple(bad.nonzero()[0].tolist())}: {got[bad][0].item()} for {want[bad][0].item()}")


# ---- embedding --------------------------------------------------------------

def _ids(tokens, rows, seed, dtype=torch.int64, strange=True):
    g = _gen(seed)
    ids = torch.randint(0, rows, (tokens,), generator=g)
    if strange and tokens > 4:
        ids[1], ids[2], ids[3], ids[-1] = -1, rows, rows - 1, -7
    return ids.to(dtype)


def _table(kind, rows, cols, seed):
    """(the operand, its values in 64 bits)."""
    x = _normal(rows, cols, seed=seed, dtype=F32, scale=0.02)
    if kind in ("fp4", "fp8"):
        t = mx.quantize(x.to(DEV), kind)
        return t, mx.dequantize(t, dtype=F32).to(D).cpu()
    x = x.to({"float32": F32, "bfloat16": BF}[kind])
    return x.to(DEV), x.to(D)


@pytest.mark.parametrize("kind", ["float32", "bfloat16", "fp4", "fp8"])
@pytest.mark.parametrize("tokens,rows,cols", [(1, 1, 1), (1, 50, 1024), (7, 33, 8), (300, 100, 9), (65, 40, 100),
                                              (257, 1000, 129), (33, 64, 2056)])
def test_embedding(tokens, rows, cols, kind):
    _say("embedding", tokens, rows, cols, kind)
    table, values = _table(kind, rows, cols, 1)
    for dtype, id_type, scale in ((BF, torch.int64, 1.0), (F32, torch.int32, math.sqrt(cols)), (BF, torch.int32, -0.37)):
        ids = _ids(tokens, rows, tokens, id_type)
        y = layers.embedding(ids.to(DEV), table, scale=scale, dtype=dtype)
        want = ref.embedding(ids, values, float(torch.tensor(scale, dtype=F32)))
        _close(y, want, 3 * S24 * want.abs().nan_to_num(), dtype)
        if scale == 1.0:
            assert torch.equal(y.cpu().nan_to_num(nan=5.0), want.to(F32).to(dtype).nan_to_num(nan=5.0))


@pytest.mark.parametrize("gap,shift", [(3, 1), (8, 8), (5, 0)])
@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
def test_embedding_between_strided_rows(kind, gap, shift):
    values = _normal(40, 77, seed=2).to({"float32": F32, "bfloat16": BF}[kind])
    table, _ = _strided(values, gap, shift)
    for dtype in (BF, F32):
        out, buf = _strided(torch.zeros(130, 77, dtype=dtype), gap, shift)
        ids = _ids(130, 40, 3)
        assert layers.embedding(ids.to(DEV), table, out=out) is out
        _close(out, ref.embedding(ids, values, 1.0), torch.zeros(1, dtype=D), dtype)
        assert _untouched(out, buf)


def test_embedding_of_nothing():
    t = torch.zeros(4, 8, device=DEV)
    none = torch.zeros(0, dtype=torch.int64, device=DEV)
    assert layers.embedding(none, t).shape == (0, 8)
    assert layers.embedding(none + 0, t[:, :0]).shape == (0, 0)
    ids = torch.tensor([0, -1, 3], device=DEV)
    y = layers.embedding(ids, t[:0])   # a table without rows
    assert torch.isnan(y[0]).all() and (y[1] == 0).all() and torch.isnan(y[2]).all()


def test_embedding_keeps_special_values():
    t = torch.tensor([[math.inf, -math.inf, math.nan, -0.0, 3e38, 1e-40, 1.0, 2.0]], device=DEV)
    y = layers.embedding(torch.zeros(1, dtype=torch.int64, device=DEV), t, dtype=F32)
    assert torch.equal(y.view(torch.int32)[0, [0, 1, 3, 4, 5, 6, 7]], t.view(torch.int32)[0, [0, 1, 3, 4, 5, 6, 7]])
    assert torch.isnan(y[0, 2])


def test_a_table_past_32_bits():
    rows, cols = (1 << 21) + 5, 2048   # 2^32 elements and more
    table = torch.zeros(rows, cols, dtype=BF, device=DEV)
    at = [0, 1, rows - 1, 1 << 20, (1 << 21) + 1]
    for i, r in enumerate(at):
        table[r] = torch.arange(cols, device=DEV).to(BF) + i
    y = layers.embedding(torch.tensor(at, device=DEV), table)
    assert torch.equal(y, table[torch.tensor(at, device=DEV)])
    ids = torch.tensor(at * 20, device=DEV)
    g = layers.embedding_grad(ids, y.repeat(20, 1) / 256, rows, out=table)
    want = (y[:, None].repeat(1, 1, 1).float().squeeze(1) / 256).to(BF).double() * 20
    assert torch.equal(g[torch.tensor(at, device=DEV)], want.to(BF))
    g[torch.tensor(at, device=DEV)] = 0
    assert float(g.view(-1, 1024).abs().amax()) == 0.0


# ---- its gradient -------------------------------------------------------------

def _drawn(how, tokens, rows, seed):
    g = _gen(seed)
    if how == "same":
        return torch.full((tokens,), rows // 2)
    if how == "text":
        return ((rows + 1) ** torch.rand(tokens, generator=g, dtype=D)).long().sub(1).clamp(0, rows - 1)
    if how == "falling":
        return torch.arange(tokens, 0, -1) % rows
    if how == "none":
        return torch.where(torch.arange(tokens) % 2 == 0, -1, rows + 3)
    ids = torch.randint(0, rows, (tokens,), generator=g)
    return torch.where(torch.rand(tokens, generator=g) < 0.2, -1, ids)   # "padded"


def _check_grad(ids, dy, rows, scale, dtype, start=None, **kw):
    want, mag, n = ref.embedding_grad(ids, dy, rows, scale)
    moved = (n[:, None] + 3) * S24 * mag
    if start is not None:
        want = want + start.to(D).cpu()
        moved = moved + S24 * (mag + start.to(D).cpu().abs())
    got = layers.embedding_grad(ids.to(DEV), dy.to(DEV) if not dy.is_cuda else dy, rows, scale=scale, dtype=dtype, **kw)
    _close(got, want, moved, dtype)
    return got


@pytest.mark.parametrize("how", ["same", "text", "falling", "none", "padded"])
@pytest.mark.parametrize("tokens", [1, 2, 31, 32, 33, 64, 65, 97, 1000, 1024, 1025, 2500])
def test_embedding_grad_by_tokens(tokens, how):
    _say("embedding_grad", tokens, how)
    rows, cols = 37, 70
    ids, dy = _drawn(how, tokens, rows, tokens), _normal(tokens, cols, seed=tokens)
    _check_grad(ids, dy, rows, 1.0, BF)
    _check_grad(ids.to(torch.int32), dy, rows, 0.3125, F32)
    start = _normal(rows, cols, seed=9)
    out = start.to(DEV)
    assert _check_grad(ids, dy, rows, -2.0, BF, start, out=out, accumulate=True) is out
    start = start.float()
    _check_grad(ids, dy, rows, 1.0, F32, start, out=start.to(DEV), accumulate=True)


@pytest.mark.parametrize("tokens,how", [(16384, "text"), (16385, "same"), (20000, "padded"), (40000, "text"), (300001, "text")])
def test_embedding_grad_over_several_merges(tokens, how):
    _say("embedding_grad", tokens, how)
    ids, dy = _drawn(how, tokens, 5000, 4), _normal(tokens, 24, seed=5)
    a = _check_grad(ids, dy, 5000, 1.0, F32)
    b = layers.embedding_grad(ids.to(DEV), dy.to(DEV), 5000, dtype=F32)
    assert torch.equal(a, b)   # whatever the order of the work-groups


@pytest.mark.parametrize("cols", [1, 2, 7, 8, 9, 255, 256, 257, 511, 512, 513, 1030, 2561])
def test_embedding_grad_by_columns(cols):
    for how in ("text", "same"):
        ids, dy = _drawn(how, 200, 20, 6), _normal(200, cols, seed=7)
        _check_grad(ids, dy, 20, 1.0, BF)


@pytest.mark.parametrize("gap,shift", [(1, 0), (3, 1), (8, 8)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_embedding_grad_between_strided_rows(dtype, gap, shift):
    ids = _drawn("text", 150, 90, 8)
    dy, _ = _strided(_normal(150, 101, seed=9), gap, shift)
    for add in (False, True):
        out, buf = _strided(torch.ones(90, 101, dtype=dtype), gap, shift)
        _check_grad(ids, dy, 90, 1.0, dtype, torch.ones(90, 101) if add else None, out=out, accumulate=add)
        assert _untouched(out, buf)


def test_embedding_grad_of_nothing():
    none = torch.zeros(0, dtype=torch.int64, device=DEV)
    dy = torch.zeros(0, 40, dtype=BF, device=DEV)
    out = torch.ones(9, 40, dtype=BF, device=DEV)
    assert float(layers.embedding_grad(none, dy, 9, out=out).abs().amax()) == 0
    out.fill_(3)
    layers.embedding_grad(none, dy, 9, out=out, accumulate=True)
    assert bool((out == 3).all())
    assert layers.embedding_grad(none, dy, 0).shape == (0, 40)
    assert layers.embedding_grad(torch.zeros(5, dtype=torch.int64, device=DEV), dy.new_zeros(5, 0), 9).shape == (9, 0)


def test_embedding_grad_leaves_rows_alone_and_passes_on_what_is_not_finite():
    ids = torch.tensor([3, 3, 5, -1, 3, 900])
    dy = torch.ones(6, 16, dtype=BF)
    dy[2, 1], dy[2, 2] = math.inf, math.nan
    dy[3] = math.nan     # padding: counts for no row
    dy[5] = math.nan     # names no row
    out = torch.full((8, 16), -0.0, dtype=BF, device=DEV)
    out[6] = math.nan
    before = out.clone()
    layers.embedding_grad(ids.to(DEV), dy.to(DEV), 8, out=out, accumulate=True)
    for r in (0, 1, 2, 4, 6, 7):
        assert torch.equal(out[r].view(torch.int16), before[r].view(torch.int16))
    assert bool((out[3] == 3).all())
    assert out[5, 1] == math.inf and torch.isnan(out[5, 2]) and out[5, 0] == 1
    g = layers.embedding_grad(ids.to(DEV), dy.to(DEV), 8)
    assert torch.isfinite(g[[0, 1, 2, 3, 4, 6, 7]]).all()


# ---- head norms with rotation ---------------------------------------------------

def _laid(tokens, h, dim, layout, seed, batch=None):
    x = _normal(*([] if batch is None else [batch]), tokens, h, dim, seed=seed, scale=2.0)
    if layout == "split":
        return x.to(DEV)
    if layout == "by head":
        return x.to(DEV).transpose(-3, -2).contiguous().transpose(-3, -2)
    wide = torch.full(x.shape[:-1] + (dim + 3,), 5.0, dtype=BF, device=DEV)   # misaligned heads with gaps
    wide[..., 1:dim + 1] = x.to(DEV)
    return wide[..., 1:dim + 1]


def _heads_case(tokens, hq, hk, dim, rotary, inter, layout, seed, batch=None, far=False, wide=True, eps=1e-6):
    q, k = _laid(tokens, hq, dim, layout, seed, batch), _laid(tokens, hk, dim, layout, seed + 1, batch)
    gq, gk = 1 + 0.5 * _normal(dim, seed=seed + 2, dtype=F32), 1 + 0.5 * _normal(dim, seed=seed + 3, dtype=F32)
    lead = (tokens,) if batch is None else (batch, tokens)
    top = (1 << 30) if far else 4096
    pos = torch.randint(-top, top, lead, generator=_gen(seed + 4), dtype=torch.int64 if wide else torch.int32)
    f = layers.rope_frequencies(rotary, theta=1e4)
    return q, k, gq, gk, pos, f, {"eps": eps, "interleaved": inter}


def _check_heads(q, k, gq, gk, pos, f, how, gain_dtype=F32, **kw):
    gq, gk = gq.to(gain_dtype), gk.to(gain_dtype)
    out = layers.head_norm_rope(q, k, gq.to(DEV), gk.to(DEV), pos.to(DEV), f, **how, **kw)
    for x, g, y in ((q, gq, out[0]), (k, gk, out[1])):
        _close(y, ref.head_norm_rope(x, g, pos, f, **how), ref.forward_off(x, g, pos, f, **how), BF)
    return out


def _check_back(q, k, gq, gk, pos, f, how, dq, dk, dtype=BF, start=None, **kw):
    got = layers.head_norm_rope_backward(q, k, gq.to(DEV), gk.to(DEV), pos.to(DEV), f, dq, dk, **how, dtype=dtype, **kw)
    for i, (x, g, dy) in enumerate(((q, gq, dq), (k, gk, dk))):
        dx, dw, off, off_w = ref.head_norm_rope_backward(x, g, pos, f, dy, **how)
        _close(got[i], dx, off, BF)
        if start is not None:
            dw, off_w = dw + start[i].to(D).cpu(), off_w + S24 * (dw.abs() + start[i].to(D).cpu().abs())
        _close(got[2 + i], dw, off_w, dtype)
    return got


HEADS = [(1, 16, 8, 128, 128), (3, 4, 1, 64, 64), (5, 12, 12, 80, 80), (33, 3, 2, 72, 72), (17, 4, 2, 96, 48),
         (6, 2, 2, 256, 256), (9, 5, 1, 128, 32), (4, 2, 1, 2, 2), (7, 3, 1, 10, 4), (5, 1, 1, 1024, 1024),
         (5, 2, 1, 514, 510), (3, 1, 2, 130, 66), (2, 70, 1, 16, 16), (1, 1, 1, 64, 0), (4, 1, 3, 126, 62)]


@pytest.mark.parametrize("layout", ["split", "by head", "gaps"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("tokens,hq,hk,dim,rotary", HEADS)
def test_head_norm_rope(tokens, hq, hk, dim, rotary, inter, layout):
    _say("heads", tokens, hq, hk, dim, rotary, inter, layout)
    case = _heads_case(tokens, hq, hk, dim, rotary, inter, layout, 20)
    _check_heads(*case)
    dq, dk = _laid(tokens, hq, dim, "split", 30), _laid(tokens, hk, dim, layout, 31)
    _check_back(*case, dq, dk)
    _check_back(*case, dq, dk, dtype=F32)


@pytest.mark.parametrize("tokens,hq,hk,dim,rotary,inter", [(5000, 2, 1, 64, 64, False), (3001, 4, 1, 128, 64, True),
                                                           (2049, 3, 3, 80, 80, False), (4099, 1, 2, 10, 6, True)])
def test_many_tokens(tokens, hq, hk, dim, rotary, inter):
    """Several tokens to a work-group, several blocks of them, a ragged last one."""
    _say("heads", tokens, hq, hk, dim, rotary, inter)
    case = _heads_case(tokens, hq, hk, dim, rotary, inter, "split", 40)
    _check_heads(*case)
    dq, dk = _laid(tokens, hq, dim, "split", 50), _laid(tokens, hk, dim, "split", 51)
    a = _check_back(*case, dq, dk, dtype=F32)
    b = layers.head_norm_rope_backward(case[0], case[1], case[2].to(DEV), case[3].to(DEV), case[4].to(DEV), case[5], dq,
                                       dk, **case[6], dtype=F32)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("layout", ["split", "by head", "gaps"])
def test_batches(layout):
    case = _heads_case(37, 4, 2, 64, 64, False, layout, 60, batch=3, wide=False)
    _check_heads(*case)
    dq, dk = _laid(37, 4, 64, layout, 61, 3), _laid(37, 2, 64, "split", 62, 3)
    _check_back(*case, dq, dk)
    # one row of positions for every batch, and an expanded one
    q, k, gq, gk, pos, f, how = case
    want = _check_heads(q, k, gq, gk, pos[:1].expand(3, 37), f, how)
    got = layers.head_norm_rope(q, k, gq.to(DEV), gk.to(DEV), pos[0].to(DEV), f, **how)
    wide = layers.head_norm_rope(q, k, gq.to(DEV), gk.to(DEV), pos[0].to(DEV).expand(3, 37), f, **how)
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(want, got, wide))


def test_far_positions_and_bfloat16_gains():
    _check_heads(*_heads_case(50, 2, 2, 128, 128, False, "split", 70, far=True), gain_dtype=BF)
    _check_heads(*_heads_case(50, 2, 2, 36, 20, True, "split", 71, far=True), gain_dtype=BF)


def test_in_place_and_strided_outputs():
    q, k, gq, gk, pos, f, how = case = _heads_case(19, 4, 2, 64, 64, False, "gaps", 80)
    want = _check_heads(*case)
    q2, k2 = q.clone(memory_format=torch.preserve_format), _laid(19, 2, 64, "by head", 81)
    k2.copy_(k)
    got = _check_heads_into(q, k, gq, gk, pos, f, how, (q2, k2))
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    dq, dk = _laid(19, 4, 64, "gaps", 82), _laid(19, 2, 64, "gaps", 83)
    grads = _check_back(*case, dq, dk)
    other = layers.head_norm_rope_backward(q, k, gq.to(DEV), gk.to(DEV), pos.to(DEV), f, dq, dk, out=(dq, dk), **how)
    assert other[0] is dq and all(torch.equal(a, b) for a, b in zip(grads, other))
    same = layers.head_norm_rope(q, k, gq.to(DEV), gk.to(DEV), pos.to(DEV), f, out=(q, k), **how)
    assert same[0] is q and all(torch.equal(a, b) for a, b in zip(want, same))


def _check_heads_into(q, k, gq, gk, pos, f, how, out):
    got = layers.head_norm_rope(q, k, gq.to(DEV), gk.to(DEV), pos.to(DEV), f, out=out, **how)
    assert got[0] is out[0] and got[1] is out[1]
    return got


def test_shared_inputs_and_results_between_others():
    """Heads that share their memory (stride 0) as inputs; results in a wider buffer, whose rest stays."""
    x = _laid(11, 1, 64, "split", 90)
    gq, gk = torch.ones(64), torch.ones(64)
    pos, f = torch.arange(11), layers.rope_frequencies(64)
    buf = torch.full((11, 9, 64), 7.0, dtype=BF, device=DEV)
    how = {"eps": 1e-6, "interleaved": False}
    _check_heads(x.expand(11, 4, 64), x, gq, gk, pos, f, how, out=(buf[:, 1:5], buf[:, 6:7]))
    assert bool((buf[:, [0, 5, 7, 8]] == 7).all())


def test_gain_gradients_are_added():
    case = _heads_case(40, 3, 2, 64, 32, True, "split", 100)
    dq, dk = _laid(40, 3, 64, "split", 101), _laid(40, 2, 64, "split", 102)
    for dtype in (BF, F32):
        start = (_normal(64, seed=103, dtype=dtype), _normal(64, seed=104, dtype=dtype))
        grads = tuple(s.to(DEV) for s in start)
        got = _check_back(*case, dq, dk, dtype=dtype, start=start, gain_grads=grads, accumulate=True)
        assert got[2] is grads[0]


def test_zero_rows_and_values_that_are_not_finite():
    q = torch.zeros(3, 2, 64, dtype=BF, device=DEV)
    q[1, 0, 5], q[2, 1, 7] = math.nan, math.inf
    k = torch.full((3, 1, 64), 1e-30, dtype=BF, device=DEV)
    one, pos, f = torch.ones(64, device=DEV), torch.arange(3, device=DEV), layers.rope_frequencies(64)
    y, z = layers.head_norm_rope(q, k, one, one, pos, f)
    assert bool((y[0] == 0).all() and (y[1, 1] == 0).all() and (y[2, 0] == 0).all())
    assert bool(torch.isnan(y[1, 0]).all()) and bool(torch.isnan(y[2, 1, [7, 39]]).any())
    assert torch.isfinite(z).all()
    dq, dk, gq, gk = layers.head_norm_rope_backward(q[:1], k[:1], one, one, pos[:1], f, torch.ones_like(q[:1]),
                                                    torch.ones_like(k[:1]))
    assert bool((gq == 0).all()) and bool((dq.float() - 1000 <= 8).all()) and torch.isfinite(dk).all()


def test_no_tokens_and_no_heads():
    one, f = torch.ones(64, device=DEV), layers.rope_frequencies(64)
    q = torch.zeros(0, 2, 64, dtype=BF, device=DEV)
    pos = torch.zeros(0, dtype=torch.int64, device=DEV)
    assert layers.head_norm_rope(q, q, one, one, pos, f)[0].shape == (0, 2, 64)
    g = (torch.ones(64, device=DEV), torch.ones(64, device=DEV))
    layers.head_norm_rope_backward(q, q, one, one, pos, f, q, q, gain_grads=g, accumulate=True)
    assert bool((g[0] == 1).all())
    layers.head_norm_rope_backward(q, q, one, one, pos, f, q, q, gain_grads=g)
    assert bool((g[0] == 0).all() and (g[1] == 0).all())
    q, k = _laid(5, 2, 64, "split", 110), torch.zeros(5, 0, 64, dtype=BF, device=DEV)
    pos = torch.arange(5, device=DEV)
    y, z = layers.head_norm_rope(q, k, one, one, pos, f)
    _close(y, ref.head_norm_rope(q, one, pos, f, 1e-6, False), ref.forward_off(q, one, pos, f, 1e-6, False), BF)
    got = layers.head_norm_rope_backward(k, q, one, one, pos, f, k, q)
    assert got[0].shape == (5, 0, 64) and bool((got[2] == 0).all())


def test_gradients_match_differences():
    """Directional derivatives of the 64-bit forward pass against the kernel's gradients, which are rounded to BF16."""
    q, k, gq, gk, pos, f, how = _heads_case(7, 3, 2, 64, 64, False, "split", 120)
    dq, dk = _laid(7, 3, 64, "split", 121), _laid(7, 2, 64, "split", 122)
    got = layers.head_norm_rope_backward(q, k, gq.to(DEV), gk.to(DEV), pos.to(DEV), f, dq, dk, **how, dtype=F32)
    for x, g, dy, dx, dw in ((q, gq, dq, got[0], got[2]), (k, gk, dk, got[1], got[3])):
        x, g, dy = x.to(D).cpu(), g.to(D), dy.to(D).cpu()
        loss = lambda a, w: float((ref.head_norm_rope(a, w, pos, f, **how) * dy).sum())  # noqa: E731, B023
        v, w, h = torch.randn(x.shape, generator=_gen(1), dtype=D), torch.randn(g.shape, generator=_gen(2), dtype=D), 1e-5
        slope = (loss(x + h * v, g) - loss(x - h * v, g)) / (2 * h)
        # each of the gradient's elements is off by a rounding; the difference by h^2 and the sums' last bits over h
        assert abs(slope - float((dx.to(D).cpu() * v).sum())) <= 2 ** -8 * float((dx.to(D).cpu() * v).abs().sum()) + 1e-5 * abs(slope)
        slope = (loss(x, g + h * w) - loss(x, g - h * w)) / (2 * h)
        assert abs(slope - float((dw.to(D).cpu() * w).sum())) <= 1e-5 * float((dw.to(D).cpu() * w).abs().sum()) + 1e-5 * abs(slope)


# ---- dropout ----------------------------------------------------------------------

KEY = {"seed": 0x123456789ABCDEF0, "step": 77, "layer": 5}


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (3, 8), (5, 9), (2, 2049), (33, 100), (7, 1024)])
def test_dropout(rows, cols, dtype):
    _say("dropout", rows, cols, dtype)
    x, r = _normal(rows, cols, seed=1, dtype=dtype), _normal(rows, cols, seed=2, dtype=dtype)
    for p, residual, offset in ((0.1, None, 0), (0.5, r, 0), (0.25, r, 8 * 12345)):
        want, kept = ref.dropout(x, p, **KEY, residual=residual, offset=offset)
        terms = torch.where(kept, x.to(D).abs() / (1 - p), 0.0) + (0 if residual is None else residual.to(D).abs())
        got = layers.dropout(x.to(DEV), p, **KEY, residual=None if residual is None else residual.to(DEV), offset=offset)
        _close(got, want, 3 * S24 * terms, dtype)
        if residual is None:
            assert torch.equal(got.cpu() != 0, kept & (x != 0))


@pytest.mark.parametrize("cols", [40, 45, 3, 1])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_dropout_of_strided_rows_is_that_of_the_whole(dtype, cols):
    x, r = _normal(70, cols, seed=3, dtype=dtype), _normal(70, cols, seed=4, dtype=dtype)
    want = layers.dropout(x.to(DEV), 0.3, **KEY, residual=r.to(DEV))
    for gap, shift in ((1, 1), (8, 0), (3, 5)):
        xs, rs = _strided(x, gap, shift)[0], _strided(r, gap + 1, shift)[0]
        out, buf = _strided(torch.zeros(70, cols, dtype=dtype), gap, shift)
        assert layers.dropout(xs, 0.3, **KEY, residual=rs, out=out) is out
        assert torch.equal(out, want) and _untouched(out, buf)
        assert torch.equal(layers.dropout(xs, 0.3, **KEY, residual=rs), want)
        assert torch.equal(layers.dropout(xs, 0.3, **KEY, residual=rs, out=rs), want)   # in place of the residual
        assert torch.equal(layers.dropout(xs, 0.3, **KEY, residual=r.to(DEV), out=xs), want)   # of x


def test_dropout_in_shards():
    x = _normal(48, 90, seed=5)
    want = layers.dropout(x.to(DEV), 0.4, **KEY)
    for at in (4, 20, 44):   # 4 rows of 90: a multiple of 8
        a, b = layers.dropout(x[:at].to(DEV), 0.4, **KEY), layers.dropout(x[at:].to(DEV), 0.4, **KEY, offset=at * 90)
        assert torch.equal(torch.cat((a, b)), want)


def test_dropout_at_the_ends_of_its_range():
    x = _normal(9, 50, seed=6).to(DEV)
    r = _normal(9, 50, seed=7).to(DEV)
    assert torch.equal(layers.dropout(x, 0.0, **KEY), x)
    assert torch.equal(layers.dropout(x, 2.0 ** -18, **KEY), x)      # rounds to 0
    assert bool((layers.dropout(x, 1.0, **KEY) == 0).all())
    assert torch.equal(layers.dropout(x, 1.0, **KEY, residual=r), r)
    last = layers.dropout(x, 0.5, **KEY, offset=(1 << 35) - 456)
    want, _ = ref.dropout(x.cpu(), 0.5, **KEY, offset=(1 << 35) - 456)
    assert torch.equal(last.to(D).cpu(), want)
    assert layers.dropout(x[:0], 0.5, **KEY).shape == (0, 50)
    big = dict(seed=(1 << 64) - 1, step=(1 << 32) + 3, layer=(1 << 32) - 1)
    assert torch.equal(layers.dropout(x, 0.5, **big).to(D).cpu(), ref.dropout(x.cpu(), 0.5, **big)[0])
    assert torch.equal(layers.dropout(x, 0.5, **{**big, "step": 3}), layers.dropout(x, 0.5, **big))


def test_dropped_values_that_are_not_finite_are_zero():
    x = torch.full((8, 64), math.nan, dtype=BF, device=DEV)
    x[::2] = math.inf
    y = layers.dropout(x, 0.5, **KEY)
    kept = ref.dropout(torch.ones(8, 64), 0.5, **KEY)[1].to(DEV)
    assert bool((y[~kept] == 0).all()) and not torch.isfinite(y[kept]).any()


def test_dropout_keeps_the_share_and_differs_by_key():
    x = torch.ones(512, 1024, device=DEV)
    base = layers.dropout(x, 0.3, **KEY)
    n = x.numel()
    share = float((base != 0).double().mean())
    assert abs(share - (1 - round(0.3 * 65536) / 65536)) <= 5 * math.sqrt(0.21 / n)   # five standard deviations
    for other in ({"seed": 1}, {"step": 78}, {"layer": 6}):
        y = layers.dropout(x, 0.3, **{**KEY, **other})
        same = float(((y != 0) == (base != 0)).double().mean())
        assert abs(same - (0.7 ** 2 + 0.3 ** 2)) <= 0.01
    assert torch.equal(layers.dropout(x, 0.3, **{**KEY, "step": torch.tensor([77], device=DEV)}), base)


# ---- streams, graphs, refusals ----------------------------------------------------------

def _calls(seed):
    """(name, results of the call on its operands), all of one seed."""
    ids = _drawn("text", 700, 300, seed).to(DEV)
    table, dy = _normal(300, 72, seed=seed, dtype=F32).to(DEV), _normal(700, 72, seed=seed + 1).to(DEV)
    q, k, gq, gk, pos, f, how = _heads_case(50, 4, 2, 64, 64, False, "split", seed)
    dq, dk = _laid(50, 4, 64, "split", seed + 5), _laid(50, 2, 64, "split", seed + 6)
    heads = [q, k, gq.to(DEV), gk.to(DEV), pos.to(DEV), f]
    step = torch.tensor([seed], device=DEV)
    return [("embedding", [ids, table], lambda a, b, **kw: (layers.embedding(a, b, **kw),)),
            ("embedding_grad", [ids, dy], lambda a, b, **kw: (layers.embedding_grad(a, b, 300, **kw),)),
            ("head_norm_rope", heads, lambda *a, **kw: layers.head_norm_rope(*a, **how, **kw)),
            ("head_norm_rope_backward", heads + [dq, dk], lambda *a, **kw: layers.head_norm_rope_backward(*a, **how, **kw)),
            ("dropout", [dy, step, dy * 2], lambda a, s, r, **kw: (layers.dropout(a, 0.2, 9, s, 3, residual=r, **kw),))]


@pytest.mark.parametrize("which", range(5))
def test_captured_and_replayed(which):
    name, operands, call = _calls(1)[which]
    _say("graph", name)
    call(*operands)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(*operands)
    for seed in (2, 3, 2, 4):
        for o, n in zip(operands, _calls(seed)[which][1]):
            o.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        want = call(*operands)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), seed
        torch.cuda.synchronize()


@pytest.mark.parametrize("which", range(5))
def test_on_another_stream(which):
    name, operands, call = _calls(5)[which]
    _say("stream", name)
    want = call(*operands)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(10_000_000)
    got = call(*operands, stream=side)
    fresh = [o.clone() for o in operands]
    del operands
    for _ in range(3):   # the operands' memory, were it not held
        [torch.empty_like(o).zero_() for o in fresh]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))

    class Other:
        device = torch.device("cuda", torch.cuda.current_device() + 1)

    with pytest.raises(ValueError, match="the stream is on"):
        call(*fresh, stream=Other())


def test_given_results_on_another_stream():
    ids, rows = _drawn("text", 500, 90, 1).to(DEV), 90
    table, dy = _normal(90, 64, seed=2, dtype=F32).to(DEV), _normal(500, 64, seed=3).to(DEV)
    q, k, gq, gk, pos, f, how = _heads_case(500, 1, 1, 64, 64, True, "split", 4)
    heads = (q, k, gq.to(DEV), gk.to(DEV), pos.to(DEV), f)

    def outs():
        e = lambda *s, dt=BF: torch.ones(*s, dtype=dt, device=DEV)   # noqa: E731
        return [e(500, 64, dt=F32), e(rows, 64, dt=F32), (e(500, 1, 64), e(500, 1, 64)), (e(500, 1, 64), e(500, 1, 64)),
                (e(64, dt=F32), e(64, dt=F32)), e(500, 64)]

    def run(o, **kw):
        return [layers.embedding(ids, table, 2.0, o[0], F32, **kw),
                layers.embedding_grad(ids, dy, rows, 2.0, o[1], True, F32, **kw),
                layers.head_norm_rope(*heads, 1e-6, True, o[2], **kw),
                layers.head_norm_rope_backward(*heads, q, k, 1e-6, True, list(o[3]), list(o[4]), True, F32, **kw),
                layers.dropout(dy, 0.3, 1, 2, 3, dy, 16, o[5], **kw)]

    want = run(outs())
    side = torch.cuda.Stream()
    given = outs()
    side.wait_stream(torch.cuda.current_stream())
    got = run(given, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    flat = lambda v: [t for x in v for t in (x if isinstance(x, tuple) else (x,))]   # noqa: E731
    assert all(torch.equal(a, b) for a, b in zip(flat(want), flat(got)))
    assert got[0] is given[0] and got[2][0] is given[2][0] and got[3][2] is given[4][0] and got[4] is given[5]


@pytest.mark.parametrize("which", range(5))
def test_two_at_once_do_not_meet(which):
    """Two calls on two streams, each with a workspace of its own."""
    calls = [_calls(s)[which] for s in (6, 7)]
    want = [c[2](*c[1]) for c in calls]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[c[2](*c[1], stream=s) for c, s in zip(calls, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for run in got for w, g in zip(want, run) for a, b in zip(w, g))


def test_refusals():
    ids = torch.zeros(4, dtype=torch.int64, device=DEV)
    t = torch.zeros(5, 8, device=DEV)
    dy = torch.zeros(4, 8, dtype=BF, device=DEV)
    h = torch.zeros(4, 2, 8, dtype=BF, device=DEV)
    one, f = torch.ones(8, device=DEV), layers.rope_frequencies(8)
    rope = lambda q=h, k=h, g=one, p=ids, fr=f, **kw: layers.head_norm_rope(q, k, g, one, p, fr, **kw)  # noqa: E731
    for call, text in [(lambda: layers.embedding(ids[None], t), "1-D"),
                       (lambda: layers.embedding(ids[::2], t), "contiguous"),
                       (lambda: layers.embedding(ids, t.t()), "consecutive"),
                       (lambda: layers.embedding(ids, t.half()), "float16"),
                       (lambda: layers.embedding(ids, t, out=t), "shape"),
                       (lambda: layers.embedding(ids, t, dtype=torch.float16), "dtype"),
                       (lambda: layers.embedding(ids, t.cpu()), "GPU"),
                       (lambda: layers.embedding(ids, t.clone().requires_grad_()), "gradient"),
                       (lambda: layers.embedding_grad(ids, dy[:3], 5), "entries"),
                       (lambda: layers.embedding_grad(ids, dy.float(), 5), "bfloat16"),
                       (lambda: layers.embedding_grad(ids, dy, 5, accumulate=True), "needs out"),
                       (lambda: layers.embedding_grad(ids, dy, 5, out=dy), "shape"),
                       (lambda: rope(k=h[:3]), "differ"), (lambda: rope(q=h[..., ::2]), "consecutive"),
                       (lambda: rope(g=one[:7]), "8 elements"), (lambda: rope(g=one.to(BF)), "float32|bfloat16"),
                       (lambda: rope(p=ids[:3]), "positions"), (lambda: rope(p=ids[0]), "positions"), (lambda: rope(p=ids.float()), "int32"),
                       (lambda: rope(fr=f.float()), "float64"), (lambda: rope(out=h), "pair"),
                       (lambda: rope(out=(h, h[:, :1])), "shape"),
                       (lambda: rope(g=one.clone().requires_grad_()), "gradient"),
                       (lambda: layers.head_norm_rope_backward(h, h, one, one, ids, f, h, h, accumulate=True), "needs gain_grads"),
                       (lambda: layers.head_norm_rope_backward(h, h, one, one, ids, f, h, h, dtype=torch.float16), "dtype"),
                       (lambda: layers.dropout(t, 0.1, -1, 0, 0), "seed"), (lambda: layers.dropout(t, 0.1, 0, 0, 1 << 32), "layer"),
                       (lambda: layers.dropout(t, 0.1, 0, ids, 0), "one element"),
                       (lambda: layers.dropout(t, 0.1, 0, 0, 0, residual=t.to(BF)), "float32"),
                       (lambda: layers.dropout(t, 0.1, 0, 0, 0, residual=t[:4]), "shape"),
                       (lambda: layers.dropout(t, 0.1, 0, 0, 0, out=t.to(BF)), "float32"),
                       (lambda: layers.dropout(t.expand(5, 8).t(), 0.1, 0, 0, 0), "consecutive")]:
        with pytest.raises(ValueError, match=text):
            call()
    for call, status in [(lambda: layers.dropout(t, 1.5, 0, 0, 0), 1), (lambda: layers.dropout(t, 0.5, 0, 0, 0, offset=4), 2),
                         (lambda: layers.embedding(ids, t, scale=math.inf), 1), (lambda: layers.embedding_grad(ids, dy, -1), 2),
                         (lambda: rope(eps=0.0), 1), (lambda: rope(out=(h[:, :1].expand(4, 2, 8), torch.zeros_like(h))), 2),
                         (lambda: rope(fr=layers.rope_frequencies(10)), 2), (lambda: rope(out=(h, h)), 4),
                         (lambda: layers.head_norm_rope_backward(h, h, one, one, ids, f, h, h, gain_grads=(one, one)), 4)]:
        with pytest.raises(api.Q4Error) as e:
            call()
        assert e.value.status == status


# ---- together -----------------------------------------------------------------------------

def test_a_layers_ends_between_masters_and_gradients():
    """Embedding, dropout, the fused projection from 4-bit weights, head norms on views of its result, and back into
    the optimizer's BF16 gradients: every call's result against the plain one of what it was given."""
    rows, d, hq, hk, dim, tokens = 211, 128, 4, 2, 64, 150
    g = _gen(130)
    table, wqkv = (torch.randn(s, generator=g).mul(0.05).to(DEV) for s in ((rows, d), (d, (hq + 2 * hk) * dim)))
    gq, gk = (1 + 0.1 * torch.randn(dim, generator=g) for _ in range(2))
    ids, pos = _drawn("padded", tokens, rows, 131), torch.arange(tokens) % 70
    f, how = layers.rope_frequencies(dim), {"eps": 1e-6, "interleaved": False}
    drop = {"p": 0.1, "seed": 17, "step": 4, "layer": 0}
    tied = mx.quantize(table, "fp4")
    x0 = layers.embedding(ids.to(DEV), tied, scale=math.sqrt(d))
    x1 = layers.dropout(x0, **drop)
    xq, w = mx.quantize(x1, "fp8"), mx.quantize(wqkv, "fp4", transpose=True)
    qkv = mx.linear(xq, w)
    q, k = qkv[:, :hq * dim].view(tokens, hq, dim), qkv[:, hq * dim:(hq + hk) * dim].view(tokens, hk, dim)
    _check_heads(q, k, gq, gk, pos, f, how)
    want = ref.embedding(ids, mx.dequantize(tied, dtype=F32).to(D).cpu(), float(torch.tensor(math.sqrt(d), dtype=F32)))
    _close(x0, want, 3 * S24 * want.abs(), BF)
    want, kept = ref.dropout(x0, **drop)
    _close(x1, want, 3 * S24 * want.abs(), BF)
    # backward: the head norms' gradients go straight into the projection's
    dqkv = _normal(tokens, (hq + 2 * hk) * dim, seed=132, scale=1e-3).to(DEV)
    dq, dk = dqkv[:, :hq * dim].view(tokens, hq, dim), dqkv[:, hq * dim:(hq + hk) * dim].view(tokens, hk, dim)
    before = dqkv.clone()
    gain_grads = (torch.zeros(dim, dtype=BF, device=DEV), torch.zeros(dim, dtype=BF, device=DEV))
    plain = [ref.head_norm_rope_backward(a, b, pos, f, c.clone(), **how) for a, b, c in ((q, gq, dq), (k, gk, dk))]
    layers.head_norm_rope_backward(q, k, gq.to(DEV), gk.to(DEV), pos.to(DEV), f, dq, dk, out=(dq, dk),
                                   gain_grads=gain_grads, accumulate=True, **how)
    for got, gain, (dx, dw, off, off_w) in zip((dq, dk), gain_grads, plain):
        _close(got, dx, off, BF)
        _close(gain, dw, off_w, BF)
    assert torch.equal(dqkv[:, (hq + hk) * dim:], before[:, (hq + hk) * dim:])
    dx1 = mx.linear_dgrad(dqkv, w)
    dx0 = layers.dropout(dx1, **drop)
    want, again = ref.dropout(dx1, **drop)
    assert torch.equal(kept, again)
    _close(dx0, want, 3 * S24 * want.abs(), BF)
    grad = torch.full((rows, d), 9.0, dtype=BF, device=DEV)
    _check_grad(ids, dx0, rows, math.sqrt(d), BF, out=grad)
    start = grad.clone()
    _check_grad(ids, dx0, rows, math.sqrt(d), BF, start, out=grad, accumulate=True)   # a second micro-batch's


# ---- sorting without merges: tokens of several tiles beside the fill of a large table ----------

@pytest.mark.parametrize("how", ["same", "text", "falling", "none", "padded"])
@pytest.mark.parametrize("tokens,rows,cols", [(1025, 40000, 320), (3000, 60000, 320), (5000, 100000, 320), (16384, 320000, 320)])
def test_embedding_grad_of_large_tables(tokens, rows, cols, how):
    _say("large table", tokens, rows, cols, how)
    ids, dy = _drawn(how, tokens, rows, tokens).to(DEV), _normal(tokens, cols, seed=3).to(DEV)
    got = layers.embedding_grad(ids, dy, rows, scale=0.5)
    # added to zeros, which sorts with merges and sums in the same order
    want = torch.zeros(rows, cols, dtype=BF, device=DEV)
    layers.embedding_grad(ids, dy, rows, scale=0.5, out=want, accumulate=True)
    assert torch.equal(got, want)
    real = (ids >= 0) & (ids < rows)
    seen = torch.unique(ids[real])
    want, mag, n = ref.embedding_grad(torch.searchsorted(seen, ids[real]), dy[real], len(seen), 0.5)
    _close(got[seen], want, (n[:, None] + 3) * S24 * mag, BF)
    got[seen] = 0
    assert float(got.abs().amax()) == 0


# ---- more than a tile's tokens, and 1024 tokens of many columns: not the form in one launch ------

@pytest.mark.parametrize("cols", [1, 2, 7, 8, 9, 255, 256, 257, 511, 512, 513, 1030])
def test_embedding_grad_of_many_tokens_by_columns(cols):
    for how in ("text", "same", "padded"):
        ids, dy = _drawn(how, 1500, 40, 6), _normal(1500, cols, seed=7)
        _check_grad(ids, dy, 40, 1.0, BF)
        start = _normal(40, cols, seed=8)
        _check_grad(ids, dy, 40, 0.5, BF, start, out=start.to(DEV), accumulate=True)


@pytest.mark.parametrize("tokens", [1, 33, 40, 300, 1024])
@pytest.mark.parametrize("how", ["same", "text", "padded"])
def test_embedding_grad_of_wide_rows(tokens, how):
    ids, dy = _drawn(how, tokens, 30, 6), _normal(tokens, 8200, seed=7)
    _check_grad(ids, dy, 30, 1.0, BF)
    start = _normal(30, 8200, seed=8)
    _check_grad(ids, dy, 30, 0.5, BF, start, out=start.to(DEV), accumulate=True)


@pytest.mark.parametrize("gap,shift", [(1, 0), (3, 1), (8, 8)])
@pytest.mark.parametrize("cols", [5, 96, 101])
def test_embedding_grad_of_many_tokens_between_strided_rows(cols, gap, shift):
    ids = _drawn("text", 3000, 900, 8)
    dy, _ = _strided(_normal(3000, cols, seed=9), gap, shift)
    for add, dtype in ((False, BF), (True, BF), (False, F32), (True, F32)):
        out, buf = _strided(torch.ones(900, cols, dtype=dtype), gap, shift)
        _check_grad(ids, dy, 900, 1.0, dtype, torch.ones(900, cols) if add else None, out=out, accumulate=add)
        assert _untouched(out, buf)


@pytest.mark.parametrize("lengths", [(33, 33, 33), (32, 1, 31, 64, 1, 33), (1, 1000, 23), (40, 60, 80, 100, 5, 5, 5, 500), (31, 34, 2, 200, 32)])
def test_embedding_grad_of_rows_around_the_lengths_that_are_split(lengths):
    ids = torch.cat([torch.full((n,), 3 * i + 1) for i, n in enumerate(lengths)])
    for tokens in (len(ids), 2200):   # either form: padding behind
        padded = torch.cat((ids, torch.full((tokens - len(ids),), -1)))[torch.randperm(tokens, generator=_gen(9))]
        dy = _normal(tokens, 72, seed=10)
        _check_grad(padded, dy, 40, 1.0, F32)
        start = _normal(40, 72, seed=11)
        _check_grad(padded, dy, 40, 1.0, BF, start, out=start.to(DEV), accumulate=True)
