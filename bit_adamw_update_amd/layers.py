"""Embedding, head norms with rotation, and dropout on torch tensors.

What a training step does with the optimizer's masters and gradients beside
the products of ``mx``: the functions allocate results and workspaces with
torch and forward to the ``q4nn_*`` calls ("beside the products" in
``include/q4adamw.h``).  They compute nothing themselves::

    x = layers.embedding(ids, master)                     # or the MXMatrix of a tied table
    x = layers.dropout(h, 0.1, seed, step, layer, residual=x)
    f = layers.rope_frequencies(128, theta=1e6)           # once
    q, k = layers.head_norm_rope(q, k, q_gain, k_gain, positions, f)
    ...
    dq, dk, _, _ = layers.head_norm_rope_backward(q_in, k_in, q_gain, k_gain, positions, f, dq, dk,
                                                  gain_grads=(q_gain_grad, k_gain_grad))
    dh = layers.dropout(dx, 0.1, seed, step, layer)       # the same mask
    layers.embedding_grad(ids, dx, rows, out=grad)        # grad: the optimizer's BF16 gradient

Streams, memory and autograd are as in ``mx``: the calls run on the current
stream of their operands' device or on ``stream``, and refuse an operand or
result whose gradient autograd would lose.
"""
from __future__ import annotations

import struct

import torch

from . import api
from .mx import _BOTH, _DTYPES, MXMatrix, _dense, _elsewhere, _entered, _lost_gradient, _raw, _result, _same_device

_CONTIGUOUS = torch.contiguous_format
_INTS = {torch.int32: api.NN_I32, torch.int64: api.NN_I64}
_PACK_HEADS = struct.Struct("@Pqqq").pack           # a q4nn_heads
_PACK_ROPE = struct.Struct("@qqiiiiiiifPPPqqP").pack   # a q4nn_rope


def _ints(name, t):
    """A GPU tensor of integers; returns its type's code."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _INTS:
        raise ValueError(f"{name} must be an int32 or int64 tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU")
    return _INTS[t.dtype]


def _tokens(ids):
    code = _ints("ids", ids)
    if ids.dim() != 1 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous 1-D tensor")
    return code


def _new(like, rows, cols, dtype):
    """(an uninitialized result, its dtype code, its row stride); like: a tensor of its device."""
    if dtype not in _DTYPES:
        raise ValueError(f"dtype must be torch.float32 or torch.bfloat16, not {dtype}")
    t = like.new_empty((rows, cols)) if like.dtype == dtype else like.new_empty((rows, cols), dtype=dtype)
    return t, _DTYPES[dtype], max(1, cols)


def _room(like, nbytes):
    """A workspace, in elements of like's type, and where it is."""
    if nbytes == 0:
        return None, None
    t = like.new_empty(nbytes // like.element_size() + 1)
    return t, t.data_ptr()


def embedding(ids, table, scale: float = 1.0, out=None, dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """scale * table[ids] [tokens, cols]: table a float32 (a master) or
    bfloat16 tensor [rows, cols] or an MXMatrix.  An id below 0 is padding (a
    row of zeros), one of rows or more gives a row of NaN."""
    id_type = _tokens(ids)
    coded = isinstance(table, MXMatrix)
    if coded:
        rows, cols = table.rows, table.cols
    else:
        ld = _dense("table", table, _BOTH)
        rows, cols = table.shape
    device = _same_device(table, ids, out)
    if _elsewhere(device, stream):
        return _entered(device, stream, (ids, table, out), embedding, ids, table, scale, out, dtype)
    tokens = ids.shape[0]
    if out is None:
        out, code, ldo = _new(ids if coded else table, tokens, cols, dtype)
    else:
        out, code, ldo = _result(out, (tokens, cols), dtype, device)
    lib = api.load_library()
    if coded:
        api._check(lib.q4nn_embedding_mx(ids.data_ptr(), id_type, tokens, table.packed, scale, out.data_ptr(), code, ldo,
                                         _raw(device)))
    else:
        api._check(lib.q4nn_embedding(ids.data_ptr(), id_type, tokens, table.data_ptr(), _DTYPES[table.dtype], rows,
                                      cols, ld, scale, out.data_ptr(), code, ldo, _raw(device)))
    return out


def embedding_grad(ids, dy, rows: int, scale: float = 1.0, out=None, accumulate: bool = False, dtype=torch.bfloat16,
                   stream=None) -> torch.Tensor:
    """The gradient [rows, cols] of embedding's table from dy, bfloat16
    [tokens, cols]: all of it, or with accumulate added to out."""
    id_type = _tokens(ids)
    lddy = _dense("dy", dy)
    device = _same_device(dy, ids, out)
    tokens, cols = dy.shape
    if ids.shape[0] != tokens:
        raise ValueError(f"dy has {tokens} rows, ids {ids.shape[0]} entries")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if _elsewhere(device, stream):
        return _entered(device, stream, (ids, dy, out), embedding_grad, ids, dy, rows, scale, out, accumulate, dtype)
    need = api.q4nn_embedding_grad_workspace_bytes(tokens, rows, cols)
    if out is None:
        out, code, ld = _new(dy, rows, cols, dtype)
    else:
        out, code, ld = _result(out, (rows, cols), dtype, device)
    ws, at = _room(dy, need)
    api._check(api.load_library().q4nn_embedding_grad(
        ids.data_ptr(), id_type, tokens, dy.data_ptr(), lddy, scale, rows, cols, out.data_ptr(), code, ld,
        api.NN_ADD if accumulate else 0, at, need, _raw(device)))
    return out


def rope_frequencies(rotary: int, theta: float = 10000.0, device="cuda") -> torch.Tensor:
    """theta^(-2 i / rotary) for the pairs i of head_norm_rope, in float64."""
    if rotary < 0 or rotary % 2:
        raise ValueError(f"rotary must be even, not {rotary}")
    return (theta ** (torch.arange(rotary // 2, dtype=torch.float64) * (-2.0 / max(1, rotary)))).to(device)


def _heads(name, t, like=None):
    """A [tokens, heads, dim] or [batch, tokens, heads, dim] operand for a call."""
    if not isinstance(t, torch.Tensor) or t.dim() not in (3, 4):
        raise ValueError(f"{name} must be a tensor [tokens, heads, dim] or [batch, tokens, heads, dim]")
    if t.dtype is not torch.bfloat16:
        raise ValueError(f"{name} must be torch.bfloat16, not {t.dtype}")
    if _lost_gradient(t):
        raise ValueError(f"{name} has a gradient, which autograd would lose here; call under torch.no_grad() or detach it")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU")
    if like is not None and t.shape != like.shape:
        raise ValueError(f"{name} must have shape {tuple(like.shape)}, not {tuple(t.shape)}")
    shape, stride = t.shape, t.stride()
    if shape[-1] > 1 and stride[-1] != 1:
        raise ValueError(f"{name} must have consecutive elements in a head (stride 1)")
    # the stride of a single entry means nothing
    return _PACK_HEADS(t.data_ptr(), stride[0] if len(shape) == 4 and shape[0] > 1 else 0,
                       stride[-3] if shape[-3] > 1 else 0, stride[-2] if shape[-2] > 1 else 0)


def _vector(name, t, n, dtypes=_BOTH):
    if not isinstance(t, torch.Tensor) or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of {n} elements")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if _lost_gradient(t):
        raise ValueError(f"{name} has a gradient, which autograd would lose here; call under torch.no_grad() or detach it")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU")


def _pair(name, v):
    if not isinstance(v, (tuple, list)) or len(v) != 2:
        raise ValueError(f"{name} must be a pair of tensors")
    return tuple(v)


def _rope(q, k, q_gain, k_gain, positions, frequencies, eps, interleaved):
    """The packed q4nn_rope of a call."""
    shape, k_shape = q.shape, k.shape
    *lead, q_heads, dim = shape
    if k_shape[:-2] != shape[:-2] or k_shape[-1] != dim:
        raise ValueError(f"q {tuple(shape)} and k {tuple(k_shape)} differ in more than their heads")
    _vector("q_gain", q_gain, dim)
    gain_dtype = q_gain.dtype
    _vector("k_gain", k_gain, dim, (gain_dtype,))
    position_type = _ints("positions", positions)
    at, step = list(positions.shape), positions.stride()
    if at == lead:
        batch_step = step[0] if len(at) == 2 and at[0] > 1 else 0
    elif len(lead) == 2 and at == lead[1:]:   # of every batch
        batch_step = 0
    else:
        raise ValueError(f"positions must have shape {tuple(lead)}, not {tuple(at)}")
    if not isinstance(frequencies, torch.Tensor) or frequencies.dim() != 1:
        raise ValueError("frequencies must be a 1-D tensor")
    pairs = frequencies.shape[0]
    _vector("frequencies", frequencies, pairs, (torch.float64,))
    return _PACK_ROPE(lead[0] if len(lead) == 2 else 1, lead[-1], q_heads, k_shape[-2], dim, 2 * pairs,
                      1 if interleaved else 0, _DTYPES[gain_dtype], position_type, eps, q_gain.data_ptr(),
                      k_gain.data_ptr(), positions.data_ptr(), batch_step, step[-1] if at[-1] > 1 else 0,
                      frequencies.data_ptr())


def _new_heads(like):
    """An uninitialized result of like's shape, and its description."""
    t = torch.empty_like(like, memory_format=_CONTIGUOUS)
    heads, dim = t.shape[-2:]
    row = heads * dim
    return t, _PACK_HEADS(t.data_ptr(), row * t.shape[-3], row, dim)


def head_norm_rope(q, k, q_gain, k_gain, positions, frequencies, eps: float = 1e-6, interleaved: bool = False,
                   out=None, stream=None) -> tuple:
    """(q', k'): every head of q and k (bfloat16 [tokens, heads, dim] or [batch,
    tokens, heads, dim], any strides but the last) divided by its root mean
    square, times its gain (dim elements, float32 or bfloat16), the first
    2 * len(frequencies) elements turned by position: pair i (elements i and
    i + len(frequencies), or with interleaved 2 i and 2 i + 1) by position *
    frequencies[i].  positions: integers, one per token (and batch).
    out: the two results' tensors, which may be q and k."""
    pq, pk = _heads("q", q), _heads("k", k)
    rope = _rope(q, k, q_gain, k_gain, positions, frequencies, eps, interleaved)
    if out is not None:
        out = qo, ko = _pair("out", out)
        pqo, pko = _heads("out[0]", qo, q), _heads("out[1]", ko, k)
        device = _same_device(q, k, q_gain, k_gain, positions, frequencies, qo, ko)
    else:
        device = _same_device(q, k, q_gain, k_gain, positions, frequencies)
    if _elsewhere(device, stream):
        return _entered(device, stream, (q, k, q_gain, k_gain, positions, frequencies, out), head_norm_rope, q, k,
                        q_gain, k_gain, positions, frequencies, eps, interleaved, out)
    if out is None:
        (qo, pqo), (ko, pko) = _new_heads(q), _new_heads(k)
    api._check(api.load_library().q4nn_head_norm_rope(rope, pq, pk, pqo, pko, _raw(device)))
    return qo, ko


def head_norm_rope_backward(q, k, q_gain, k_gain, positions, frequencies, dq, dk, eps: float = 1e-6,
                            interleaved: bool = False, out=None, gain_grads=None, accumulate: bool = False,
                            dtype=torch.bfloat16, stream=None) -> tuple:
    """(dq, dk, dq_gain, dk_gain): the gradients of head_norm_rope's q, k and
    gains from its inputs and the gradients dq, dk of its results.  out: the
    tensors of the first two, which may be dq and dk, or q and k; gain_grads:
    those of the others (bfloat16 or float32), to which accumulate adds."""
    pq, pk, pdq, pdk = _heads("q", q), _heads("k", k), _heads("dq", dq, q), _heads("dk", dk, k)
    rope = _rope(q, k, q_gain, k_gain, positions, frequencies, eps, interleaved)
    held = [q, k, q_gain, k_gain, positions, frequencies, dq, dk]
    if out is not None:
        out = qo, ko = _pair("out", out)
        pqo, pko = _heads("out[0]", qo, q), _heads("out[1]", ko, k)
        held += [qo, ko]
    if gain_grads is not None:
        gain_grads = gq, gk = _pair("gain_grads", gain_grads)
        _vector("gain_grads[0]", gq, q.shape[-1])
        _vector("gain_grads[1]", gk, q.shape[-1], (gq.dtype,))
        held += [gq, gk]
    elif accumulate:
        raise ValueError("accumulate needs gain_grads")
    elif dtype not in _DTYPES:
        raise ValueError(f"dtype must be torch.float32 or torch.bfloat16, not {dtype}")
    device = _same_device(*held)
    if _elsewhere(device, stream):
        return _entered(device, stream, tuple(held), head_norm_rope_backward, q, k, q_gain, k_gain, positions,
                        frequencies, dq, dk, eps, interleaved, out, gain_grads, accumulate, dtype)
    if out is None:
        (qo, pqo), (ko, pko) = _new_heads(q), _new_heads(k)
    if gain_grads is None:
        gq, gk = (torch.empty_like(t, dtype=dtype) for t in (q_gain, k_gain))
    need = api.q4nn_head_norm_rope_backward_workspace_bytes(rope)
    ws, at = _room(q, need)
    api._check(api.load_library().q4nn_head_norm_rope_backward(
        rope, pq, pk, pdq, pdk, pqo, pko, gq.data_ptr(), gk.data_ptr(), _DTYPES[gq.dtype],
        api.NN_ADD if accumulate else 0, at, need, _raw(device)))
    return qo, ko, gq, gk


def dropout(x, p: float, seed: int, step, layer: int, residual=None, offset: int = 0, out=None,
            stream=None) -> torch.Tensor:
    """x / (1 - p) where an element is kept, 0 where it is dropped (with
    probability p, rounded to a multiple of 2^-16), plus residual; x float32 or
    bfloat16 [rows, cols], residual and out of its type (out may be either).
    The mask follows from seed, step, layer and the element's index, counted
    from offset (a multiple of 8); it is never stored, and the backward pass is
    the same call on the gradient.  step: a number, or an int64 tensor of one
    element on the GPU (a captured graph's replays read it anew)."""
    ldx = _dense("x", x, _BOTH)
    ldr, at = 0, None
    if residual is not None:
        ldr = _dense("residual", residual, (x.dtype,))
        if residual.shape != x.shape:
            raise ValueError(f"residual must have shape {tuple(x.shape)}, not {tuple(residual.shape)}")
    on_gpu = isinstance(step, torch.Tensor)
    if on_gpu and (step.dtype != torch.int64 or step.numel() != 1 or not step.is_cuda):
        raise ValueError("step must be a number or an int64 tensor of one element on the GPU")
    if not 0 <= seed < 1 << 64 or not 0 <= layer < 1 << 32 or not (on_gpu or 0 <= step < 1 << 64):
        raise ValueError("seed and step must be in [0, 2^64), layer in [0, 2^32)")
    if out is not None and out.dtype != x.dtype:
        raise ValueError(f"out must be {x.dtype}, not {out.dtype}")
    device = _same_device(x, residual, out, step if on_gpu else None)
    if _elsewhere(device, stream):
        return _entered(device, stream, (x, residual, out, step if on_gpu else None), dropout, x, p, seed, step, layer,
                        residual, offset, out)
    rows, cols = x.shape
    if out is None:
        out, code, ldo = torch.empty_like(x, memory_format=_CONTIGUOUS), _DTYPES[x.dtype], max(1, cols)
    else:
        out, code, ldo = _result(out, (rows, cols), x.dtype, device)
    if on_gpu:
        at, step = step.data_ptr(), 0
    api._check(api.load_library().q4nn_dropout(
        p, seed, step, at, layer, offset, x.data_ptr(), ldx, None if residual is None else residual.data_ptr(), ldr, rows,
        cols, out.data_ptr(), ldo, code, _raw(device)))
    return out
