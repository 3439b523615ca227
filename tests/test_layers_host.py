"""Refusals and host arithmetic of embedding, head norms and dropout: every call
here is refused, or has nothing to do, before any device work, so no GPU is
needed.  The plain implementations are held to published values and to
differences."""
import ctypes
import math
import os

import pytest
import torch

import layers_reference as ref
from bit_adamw_update_amd import api, layers

INVALID, SHAPE, ALIGNMENT, CONFLICT, WORKSPACE = 1, 2, 3, 4, 7
P = 0x10000000   # plausible aligned addresses: refused before any is used
BIG = 1 << 31


def refused(status, text, fn, *args, **kw):
    with pytest.raises(api.Q4Error) as e:
        fn(*args, **kw)
    assert e.value.status == status, str(e.value)
    assert text in str(e.value), str(e.value)


def lookup(ids=P, id_type=api.NN_I64, tokens=8, table=P, dtype=api.MX_F32, rows=100, cols=64, ld=64, scale=1.0, out=P,
           out_dtype=api.MX_BF16, ldo=64):
    api.q4nn_embedding(ids, id_type, tokens, table, dtype, rows, cols, ld, scale, out, out_dtype, ldo, 0)


def test_lookups_are_checked():
    refused(INVALID, "ids is NULL", lookup, ids=None)
    refused(INVALID, "integer type", lookup, id_type=2)
    refused(ALIGNMENT, "ids", lookup, ids=P + 4)
    refused(ALIGNMENT, "ids", lookup, ids=P + 2, id_type=api.NN_I32)
    refused(SHAPE, "ids", lookup, tokens=-1)
    refused(SHAPE, "ids", lookup, tokens=BIG)
    refused(INVALID, "table is NULL", lookup, table=None)
    refused(INVALID, "dtype", lookup, dtype=7)
    refused(INVALID, "dtype", lookup, out_dtype=-1)
    refused(SHAPE, "stride", lookup, ld=63)
    refused(SHAPE, "stride", lookup, ldo=63)
    refused(SHAPE, "table", lookup, rows=BIG)
    refused(ALIGNMENT, "table", lookup, table=P + 2)
    refused(ALIGNMENT, "out", lookup, out=P + 1)
    refused(INVALID, "scale", lookup, scale=math.inf)
    refused(INVALID, "scale", lookup, scale=math.nan)
    refused(SHAPE, "2^38", lookup, tokens=1 << 20, cols=1 << 18, ld=1 << 18, ldo=1 << 18)
    mx = lambda **k: api.q4nn_embedding_mx(P, 1, 8, api.Q4MXMatrix(**{**dict(format=1, reserved=0, rows=9, cols=64, codes=P, scales=P), **k}), 1.0, P, 1, 64, 0)  # noqa: E731
    refused(INVALID, "format", mx, format=2)
    refused(INVALID, "NULL", mx, codes=None)
    refused(ALIGNMENT, "16-byte", mx, scales=P + 4)
    refused(SHAPE, "stride", mx, cols=65)


def test_a_lookup_in_the_place_of_its_table():
    # a row is read by any work-group, after others have written theirs
    for k in (dict(), dict(tokens=100), dict(tokens=1), dict(dtype=api.MX_BF16)):
        refused(CONFLICT, "in the place of the table", lookup, table=P, out=P, **k)
    for out in (2 * P, 3 * P):
        refused(CONFLICT, "in the place of the table", api.q4nn_embedding_mx, P, 1, 8,
                api.Q4MXMatrix(format=1, reserved=0, rows=9, cols=64, codes=2 * P, scales=3 * P), 1.0, out, 1, 64, 0)
    # not where nothing is read
    lookup(tokens=0, table=P, out=P)
    lookup(cols=0, table=P, out=P)


def grad(ids=P, id_type=api.NN_I64, tokens=40, dy=P, lddy=64, scale=1.0, rows=100, cols=64, out=P, dtype=api.MX_BF16,
         ldg=64, flags=0, ws=P, n=1 << 40):
    api.q4nn_embedding_grad(ids, id_type, tokens, dy, lddy, scale, rows, cols, out, dtype, ldg, flags, ws, n, 0)


def test_gradients_of_tables_are_checked():
    need = api.q4nn_embedding_grad_workspace_bytes(40, 100, 64)
    assert need >= 40 * 16 + 2 * 2 * 64 * 4
    refused(WORKSPACE, "NULL", grad, ws=None)
    refused(WORKSPACE, str(need), grad, n=need - 1)
    refused(ALIGNMENT, "workspace", grad, ws=P + 8)
    refused(INVALID, "flags", grad, flags=2)
    refused(INVALID, "ids is NULL", grad, ids=None)
    refused(INVALID, "dy is NULL", grad, dy=None)
    refused(INVALID, "grad is NULL", grad, out=None)
    refused(SHAPE, "dy", grad, lddy=63)
    refused(SHAPE, "grad", grad, ldg=63)
    refused(SHAPE, "outside", grad, rows=-1)
    refused(INVALID, "scale", grad, scale=math.nan)
    refused(SHAPE, "2^38", grad, rows=1 << 20, cols=1 << 18, lddy=1 << 18, ldg=1 << 18)
    refused(SHAPE, "outside", api.q4nn_embedding_grad_workspace_bytes, BIG, 1, 1)
    refused(SHAPE, "2^38", api.q4nn_embedding_grad_workspace_bytes, 1 << 30, 1, 1 << 10)
    assert api.q4nn_embedding_grad_workspace_bytes(0, 5, 5) == 0
    assert api.q4nn_embedding_grad_workspace_bytes(5, 0, 5) == 0


def test_a_tables_gradient_in_the_place_of_its_operand():
    # zeros are written before dy is summed, and a row's sum before another row's dy is read
    for rows, flags in ((40, 0), (40, api.NN_ADD), (100, 0), (7, 0)):
        refused(CONFLICT, "in the place of dy", grad, rows=rows, out=P, dy=P, flags=flags)
    # not where dy has nothing to read
    grad(rows=0, out=P, dy=P)
    grad(tokens=0, out=P, dy=P, flags=api.NN_ADD)


def rope(**k):
    d = dict(batches=2, tokens=5, q_heads=4, k_heads=2, dim=64, rotary=64, interleaved=0, gain_dtype=0,
             position_type=1, eps=1e-6, q_gain=P, k_gain=P, positions=P, position_batch=5, position_token=1,
             frequencies=P)
    return api.Q4NNRope(**{**d, **k})


def view(heads, dim=64, tokens=5, **k):
    return api.Q4NNHeads(**{**dict(p=P, batch=tokens * heads * dim, token=heads * dim, head=dim), **k})


def heads(r=None, q=None, k=None, qo=None, ko=None):
    api.q4nn_head_norm_rope(r or rope(), q or view(4), k or view(2), qo or view(4, p=2 * P), ko or view(2, p=3 * P), 0)


def back(r=None, dq=None, dqi=None, dki=None, gq=P, gk=2 * P, dtype=api.MX_BF16, flags=0, ws=P, n=1 << 40):
    api.q4nn_head_norm_rope_backward(r or rope(), view(4), view(2), dq or view(4, p=2 * P), view(2, p=3 * P),
                                     dqi or view(4, p=4 * P), dki or view(2, p=5 * P), gq, gk, dtype, flags, ws, n, 0)


@pytest.mark.parametrize("call", [heads, back])
def test_ropes_are_checked(call):
    for status, text, k in [(SHAPE, "batches", dict(batches=-1)), (SHAPE, "batches", dict(batches=1 << 16, tokens=1 << 15)),
                            (SHAPE, "heads", dict(q_heads=4097)), (SHAPE, "heads", dict(k_heads=-1)),
                            (SHAPE, "dim", dict(dim=63, rotary=62)), (SHAPE, "dim", dict(dim=1026)),
                            (SHAPE, "dim", dict(dim=0, rotary=0)), (SHAPE, "rotary", dict(rotary=66)),
                            (SHAPE, "rotary", dict(rotary=31)), (SHAPE, "rotary", dict(rotary=-2)),
                            (INVALID, "interleaved", dict(interleaved=2)), (INVALID, "dtype", dict(gain_dtype=2)),
                            (INVALID, "integer type", dict(position_type=2)), (INVALID, "eps", dict(eps=0.0)),
                            (INVALID, "eps", dict(eps=1e-40)), (INVALID, "eps", dict(eps=math.nan)),
                            (INVALID, "eps", dict(eps=math.inf)), (INVALID, "q_gain", dict(q_gain=None)),
                            (INVALID, "k_gain", dict(k_gain=None)), (INVALID, "positions", dict(positions=None)),
                            (INVALID, "frequencies", dict(frequencies=None)), (ALIGNMENT, "gain", dict(q_gain=P + 2)),
                            (ALIGNMENT, "positions", dict(positions=P + 4)),
                            (ALIGNMENT, "frequencies", dict(frequencies=P + 4)),
                            (SHAPE, "stride", dict(position_token=-1)), (SHAPE, "stride", dict(position_batch=BIG))]:
        refused(status, text, call, rope(**k))


def test_head_operands_are_checked():
    refused(INVALID, "q.p", heads, q=view(4, p=None))
    refused(ALIGNMENT, "k is", heads, k=view(2, p=P + 1))
    refused(SHAPE, "stride", heads, q=view(4, head=-1))
    refused(SHAPE, "stride", heads, q=view(4, token=1 << 40))
    refused(SHAPE, "2^50", heads, rope(batches=1, tokens=1 << 20), q=view(4, token=1 << 39))
    refused(SHAPE, "overlap", heads, qo=view(4, p=2 * P, head=63))
    refused(SHAPE, "overlap", heads, qo=view(4, p=2 * P, token=0))
    refused(SHAPE, "overlap", heads, ko=view(2, p=3 * P, batch=64))
    refused(SHAPE, "in place", heads, q=view(4, p=2 * P, token=300), qo=view(4, p=2 * P))
    refused(SHAPE, "in place", back, dq=view(4, p=4 * P, token=300))
    need = api.q4nn_head_norm_rope_backward_workspace_bytes(rope())
    assert need >= 2 * 64 * 4
    refused(WORKSPACE, "NULL", back, ws=None)
    refused(WORKSPACE, str(need), back, n=need - 1)
    refused(INVALID, "flags", back, flags=4)
    refused(INVALID, "dq_gain", back, gq=None)
    refused(CONFLICT, "one buffer", back, gk=P)
    refused(CONFLICT, "one buffer", back, dki=view(2, p=4 * P))
    refused(CONFLICT, "one buffer", heads, ko=view(2, p=2 * P))
    refused(CONFLICT, "the other", heads, k=view(2, p=2 * P))
    refused(CONFLICT, "the other", heads, ko=view(2, p=P))
    refused(CONFLICT, "the other", back, dqi=view(4, p=3 * P))
    refused(CONFLICT, "the other", back, dki=view(2, p=2 * P))
    refused(CONFLICT, "the other", back, dki=view(2, p=P))
    refused(INVALID, "dtype", back, dtype=3)
    refused(ALIGNMENT, "dk_gain", back, gk=P + 1)
    refused(SHAPE, "overlap", back, dki=view(2, p=5 * P, head=0))


def test_gradients_in_the_place_of_an_input_have_its_strides():
    # q's and k's addresses are P: a permuted view of equal extents, and other strides
    refused(SHAPE, "in place", back, rope(tokens=4), dqi=view(4, p=P, batch=1024, token=64, head=256))
    refused(SHAPE, "in place", back, dqi=view(4, p=P, token=300, batch=1500))
    refused(SHAPE, "in place", back, rope(k_heads=0), dqi=view(4, p=P, token=300, batch=1500))
    refused(SHAPE, "in place", back, rope(q_heads=0), dki=view(2, p=P, token=300, batch=1500))
    # with its strides it is not: the next thing to refuse is the workspace
    refused(WORKSPACE, "NULL", back, rope(k_heads=0), dqi=view(4, p=P), ws=None)
    refused(WORKSPACE, "NULL", back, rope(q_heads=0), dki=view(2, p=P), ws=None)


def test_strides_of_a_single_head_and_of_none_mean_nothing():
    def one(**k):
        return view(1, **{**dict(batch=320, token=64, head=64), **k})
    r = rope(q_heads=1, k_heads=0)
    for call in (lambda: api.q4nn_head_norm_rope_backward(r, one(), view(2), one(p=2 * P), view(2), one(p=P, head=0), view(2),
                                                          P, 2 * P, 1, 0, None, 0, 0),
                 lambda: api.q4nn_head_norm_rope_backward(r, one(), view(2), one(p=2 * P, head=7), view(2), one(p=2 * P),
                                                          view(2, p=P, token=999), P, 2 * P, 1, 0, None, 0, 0)):
        refused(WORKSPACE, "NULL", call)   # the next thing to refuse
    refused(SHAPE, "in place", api.q4nn_head_norm_rope, r, one(token=65), view(2), one(head=1), view(2), 0)


def drop(p=0.1, step_at=None, offset=0, x=P, ldx=64, res=None, ldr=64, rows=10, cols=64, out=2 * P, ldo=64, dtype=1):
    api.q4nn_dropout(p, 1, 1, step_at, 0, offset, x, ldx, res, ldr, rows, cols, out, ldo, dtype, 0)


def test_dropouts_are_checked():
    for p in (-0.01, 1.01, math.nan, math.inf):
        refused(INVALID, "p is outside", drop, p=p)
    refused(ALIGNMENT, "step_at", drop, step_at=P + 4)
    refused(SHAPE, "multiple of 8", drop, offset=4)
    refused(SHAPE, "multiple of 8", drop, offset=-8)
    refused(SHAPE, "2^35", drop, offset=(1 << 35) - 632)
    refused(SHAPE, "2^35", drop, rows=1 << 30, cols=64)
    refused(INVALID, "x is NULL", drop, x=None)
    refused(INVALID, "dtype", drop, dtype=2)
    refused(SHAPE, "x: row stride", drop, ldx=63)
    refused(SHAPE, "residual: row stride", drop, res=3 * P, ldr=63)
    refused(SHAPE, "out: row stride", drop, ldo=60)
    refused(SHAPE, "in place", drop, out=P, ldo=72)
    refused(SHAPE, "in place", drop, res=2 * P, ldr=72)
    refused(ALIGNMENT, "out", drop, out=P + 1)


def test_nothing_to_do_needs_no_pointers():
    lookup(ids=None, tokens=0, out=None)
    lookup(table=None, out=None, cols=0)
    grad(rows=0, out=None)
    grad(tokens=0, ids=None, dy=None, flags=api.NN_ADD)
    none = view(4, p=None)
    heads(rope(tokens=0, positions=None), none, none, none, none)
    back(rope(tokens=0, positions=None), flags=api.NN_ADD, ws=None, n=0)
    drop(x=None, out=None, rows=0)


def test_structures_match_the_packed_forms():
    assert ctypes.sizeof(api.Q4NNHeads) == layers.struct.calcsize("@Pqqq")
    assert ctypes.sizeof(api.Q4NNRope) == layers.struct.calcsize("@qqiiiiiiifPPPqqP")
    r = rope(eps=0.5)
    packed = layers._PACK_ROPE(2, 5, 4, 2, 64, 64, 0, 0, 1, 0.5, P, P, P, 5, 1, P)
    assert bytes(r) == packed


def test_tensors_are_checked():
    ids, t = torch.zeros(4, dtype=torch.int64), torch.zeros(3, 8)
    for call, text in [(lambda: layers.embedding(ids.float(), t), "int32 or int64"),
                       (lambda: layers.embedding(ids, t), "GPU"),
                       (lambda: layers.embedding([1], t), "int32 or int64"),
                       (lambda: layers.embedding_grad(ids, t.bfloat16(), 5), "GPU"),
                       (lambda: layers.head_norm_rope(t, t, t, t, ids, t), r"\[tokens, heads, dim\]"),
                       (lambda: layers.head_norm_rope(t[None], t[None], t, t, ids, t), "bfloat16"),
                       (lambda: layers.rope_frequencies(3), "even"),
                       (lambda: layers.dropout(t[0], 0.1, 0, 0, 0), "2-D"),
                       (lambda: layers.dropout(t.half(), 0.1, 0, 0, 0), "float16"),
                       (lambda: layers.dropout(t, 0.1, 0, 0, 0), "GPU")]:
        with pytest.raises(ValueError, match=text):
            call()
    x = torch.zeros(2, 2, 8, dtype=torch.bfloat16, requires_grad=True)
    for call in (lambda: layers.head_norm_rope(x, x, t[0], t[0], ids, t), lambda: layers.dropout(x[0], 0.1, 0, 0, 0)):
        with pytest.raises(ValueError, match="gradient"):
            call()


def test_frequencies():
    f = layers.rope_frequencies(6, theta=100.0, device="cpu")
    assert f.dtype == torch.float64 and f.tolist() == pytest.approx([1.0, 100 ** (-1 / 3), 100 ** (-2 / 3)], rel=1e-15)
    assert layers.rope_frequencies(0, device="cpu").shape == (0,)


# ---- the plain implementations themselves -----------------------------------

def test_plain_philox_gives_the_published_values():
    path = os.path.join(os.path.dirname(__file__), "golden", "philox4x32_10_kat.txt")
    seen = 0
    with open(path) as f:
        for line in f:
            words = line.split("#")[0].split()
            if len(words) < 10:
                continue
            v = [int(w, 16) for w in words[-10:]]
            assert ref.philox(v[:4], v[4:6]) == v[6:]
            seen += 1
    assert seen >= 3


@pytest.mark.parametrize("interleaved", [False, True])
def test_plain_gradients_match_differences(interleaved):
    g = torch.Generator().manual_seed(3)
    x, dy = (torch.randn(5, 3, 12, generator=g, dtype=torch.float64) for _ in range(2))
    gain = torch.randn(12, generator=g, dtype=torch.float64)
    pos, f = torch.tensor([0, 1, 7, -3, 100]), layers.rope_frequencies(8, device="cpu")
    loss = lambda a, w: float((ref.head_norm_rope(a, w, pos, f, 1e-3, interleaved) * dy).sum())  # noqa: E731
    dx, dw, _, _ = ref.head_norm_rope_backward(x, gain, pos, f, dy, 1e-3, interleaved)
    for _ in range(5):
        v, w = torch.randn(x.shape, generator=g, dtype=torch.float64), torch.randn(12, generator=g, dtype=torch.float64)
        h = 1e-5
        assert (loss(x + h * v, gain) - loss(x - h * v, gain)) / (2 * h) == pytest.approx(float((dx * v).sum()), rel=1e-6)
        assert (loss(x, gain + h * w) - loss(x, gain - h * w)) / (2 * h) == pytest.approx(float((dw * w).sum()), rel=1e-6)
