"""Refusals and host arithmetic of the microscaled linear layer's C ABI: every
call here is refused, or has nothing to do, before any device work, so no GPU
is needed."""
import pytest

from bit_adamw_update_amd import api, mx

INVALID, SHAPE, ALIGNMENT, CONFLICT, DEVICE, WORKSPACE = 1, 2, 3, 4, 6, 7
P = 0x10000000   # plausible aligned addresses: refused before any is used


def M(fmt=api.MX_FP8, rows=64, cols=256, codes=P, scales=2 * P, reserved=0):
    return api.Q4MXMatrix(fmt, reserved, rows, cols, codes, scales)


def W(**k):
    return M(fmt=api.MX_FP4, **k)


def refused(status, text, fn, *args):
    with pytest.raises(api.Q4Error) as e:
        fn(*args)
    assert e.value.status == status, str(e.value)
    assert text in str(e.value)


@pytest.mark.parametrize("fmt,rows,cols,codes,scales", [
    (api.MX_FP4, 1, 1, 64, 4), (api.MX_FP8, 1, 1, 128, 4), (api.MX_FP4, 3, 129, 384, 24), (api.MX_FP8, 7, 128, 896, 28),
    (api.MX_FP8, 0, 5, 0, 0), (api.MX_FP4, 5, 0, 0, 0), (api.MX_FP8, 2 ** 26, 255, 2 ** 34 // 1, None)])
def test_matrix_bytes(fmt, rows, cols, codes, scales):
    if scales is None:   # 2^34 padded elements
        refused(SHAPE, "2^34", api.q4mx_matrix_bytes, fmt, rows, cols)
        api.q4mx_matrix_bytes(fmt, rows - 1, cols)
        return
    assert api.q4mx_matrix_bytes(fmt, rows, cols) == (codes, scales)


def test_matrices_are_checked():
    q = lambda m, *a: api.q4mx_dequantize(m, P, api.MX_F32, 256, 0)  # noqa: E731
    refused(INVALID, "format", q, M(fmt=2))
    refused(INVALID, "format", q, M(fmt=-1))
    refused(INVALID, "reserved", q, M(reserved=1))
    refused(INVALID, "NULL", q, None)
    refused(INVALID, "NULL", q, M(codes=None))
    refused(INVALID, "NULL", q, M(scales=None))
    refused(ALIGNMENT, "16-byte", q, M(codes=P + 8))
    refused(ALIGNMENT, "16-byte", q, M(scales=P + 1))
    refused(SHAPE, "outside", q, M(rows=-1))
    refused(SHAPE, "outside", q, M(cols=2 ** 31))
    refused(SHAPE, "2^34", q, M(rows=2 ** 30))


def test_dense_operands_are_checked():
    q = lambda p=P, dt=api.MX_F32, ld=256, t=False, m=None: api.q4mx_quantize(p, dt, ld, t, m or M(), 0)  # noqa: E731
    refused(INVALID, "dtype", q, P, 2)
    refused(INVALID, "NULL", q, None)
    refused(ALIGNMENT, "aligned", q, P + 2)
    refused(ALIGNMENT, "aligned", q, P + 1, api.MX_BF16)
    refused(SHAPE, "stride", q, P, api.MX_F32, 255)
    refused(SHAPE, "stride", q, P, api.MX_F32, 63, True)
    refused(SHAPE, "stride", q, P, api.MX_F32, 2 ** 31)
    with pytest.raises(api.Q4Error):
        api._check(api.load_library().q4mx_quantize(P, 0, 256, 2, api._mx(M()), None))


def test_products_are_checked():
    lin = lambda x, w, y=P, dt=api.MX_BF16, ld=512: api.q4mx_linear(x, w, y, dt, ld, None, None, 0)  # noqa: E731
    refused(CONFLICT, "FP4", lin, M(), M())
    refused(SHAPE, "columns", lin, M(cols=128), W())
    refused(SHAPE, "stride", lin, M(), W(rows=600))
    refused(INVALID, "NULL", lin, M(), W(), None)
    refused(INVALID, "dtype", lin, M(), W(), P, 9)
    b = lambda x=P, ld=256, t=40, w=None, ws=None, n=0: api.q4mx_linear_bf16(  # noqa: E731
        x, ld, t, w or W(), P, api.MX_BF16, 64, ws, n, 0)
    need = api.q4mx_linear_bf16_workspace_bytes(40, W())
    assert need >= 40 * 256 + 40 * 8
    refused(WORKSPACE, "NULL", b)
    refused(WORKSPACE, str(need), b, P, 256, 40, None, P, need - 1)
    refused(ALIGNMENT, "workspace", b, P, 256, 40, None, P + 8, need)
    refused(SHAPE, "outside", b, P, 256, -1)
    refused(SHAPE, "stride", b, P, 255)
    refused(ALIGNMENT, "aligned", b, P + 1)
    d = lambda dy=P, ld=64, t=40, w=None, dx=P: api.q4mx_dgrad(  # noqa: E731
        dy, ld, t, w or W(), dx, api.MX_BF16, 256, P, 1 << 40, 0)
    refused(CONFLICT, "FP4", d, P, 64, 40, M())
    refused(SHAPE, "stride", d, P, 63)
    refused(SHAPE, "outside", d, P, 64, -5)
    refused(INVALID, "NULL", d, P, 64, 40, None, None)
    g = lambda dy=P, ld=300, n=300, x=None, dw=P, lddw=300, flags=0: api.q4mx_wgrad(  # noqa: E731
        dy, ld, n, x or M(), dw, api.MX_BF16, lddw, flags, P, 1 << 40, 0)
    refused(INVALID, "flags", g, P, 300, 300, None, P, 300, 4)
    refused(SHAPE, "stride", g, P, 299)
    refused(SHAPE, "outside", g, P, 300, -1)
    refused(SHAPE, "dw", g, P, 300, 300, None, P, 255)
    refused(SHAPE, "dw", g, P, 300, 300, None, P, 299, api.MX_WGRAD_TRANSPOSED)
    refused(ALIGNMENT, "dy", g, P + 1)


def test_activations_are_checked():
    f = lambda act=0, x=P, up=None, y=P, ymx=None, kx=None, ku=None, r=64, c=256, ld=256: api.q4mx_act_forward(  # noqa: E731
        act, x, ld, up, ld, r, c, y, ld, ymx, kx, ku, 0)
    refused(INVALID, "activation", f, 3)
    refused(INVALID, "activation", f, -1)
    refused(CONFLICT, "SWIGLU", f, 0, P, P)
    refused(CONFLICT, "SWIGLU", f, 1, P, None, P, None, None, M())
    refused(INVALID, "up is NULL", f, 2)
    refused(INVALID, "no output", f, 0, P, None, None)
    refused(CONFLICT, "FP8", f, 0, P, None, P, None, W())
    refused(SHAPE, "kept_x", f, 0, P, None, P, None, M(rows=63))
    refused(SHAPE, "y_mx", f, 0, P, None, P, M(cols=128))
    refused(SHAPE, "stride", f, 0, P, None, P, None, None, None, 64, 256, 200)
    b = lambda act=0, kx=M(), ku=None, dy=P, dx=P, dup=None, lddx=256: api.q4mx_act_backward(  # noqa: E731
        act, kx, ku, dy, 256, dx, lddx, dup, 256, 0)
    refused(INVALID, "activation", b, 7)
    refused(INVALID, "kept_x", b, 0, None)
    refused(CONFLICT, "FP8", b, 0, W())
    refused(CONFLICT, "SWIGLU", b, 0, M(), M())
    refused(CONFLICT, "SWIGLU", b, 0, M(), None, P, P, P)
    refused(INVALID, "kept_up", b, 2)
    refused(SHAPE, "kept_up", b, 2, M(), M(rows=2), P, P, P)
    refused(INVALID, "dup", b, 2, M(), M())
    refused(SHAPE, "row stride", b, 0, M(), None, P, P, None, 264)


def test_nothing_to_do_needs_no_pointers():
    none = M(rows=0, codes=None, scales=None)
    api.q4mx_quantize(None, api.MX_F32, 0, False, none, 0)
    api.q4mx_dequantize(none, None, api.MX_F32, 0, 0)
    api.q4mx_linear(none, W(), None, api.MX_BF16, 0, None, None, 0)
    api.q4mx_linear_bf16(None, 0, 0, W(), None, api.MX_BF16, 0, None, None, 0)
    api.q4mx_dgrad(None, 0, 0, W(), None, api.MX_BF16, 0, None, None, 0)
    api.q4mx_wgrad(P, 8, 0, M(), None, api.MX_BF16, 0, 0, None, None, 0)
    api.q4mx_act_forward(0, None, 0, None, 0, 0, 5, None, 0, stream=0)
    api.q4mx_act_backward(0, none, None, None, 0, None, 0, stream=0)


def test_tensors_are_checked():
    import torch
    with pytest.raises(ValueError, match="format"):
        mx.MXMatrix(4, 4, "fp6", device="cpu")
    with pytest.raises(api.Q4Error):
        mx.MXMatrix(-1, 4, "fp4", device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        mx.MXMatrix(4, 4, "fp4", device="cpu")
    with pytest.raises(ValueError, match="together"):
        mx.MXMatrix(4, 4, "fp4", codes=torch.zeros(4, 64, dtype=torch.uint8))
    with pytest.raises(ValueError, match="shape"):
        mx.MXMatrix(4, 4, "fp4", codes=torch.zeros(4, 2, dtype=torch.uint8),
                    scales=torch.zeros(1, 4, 4, dtype=torch.uint8))
    for bad, text in ((torch.zeros(3), "2-D"), (torch.zeros(3, 3, dtype=torch.float16), "bfloat16"),
                      (torch.zeros(3, 3), "GPU"), ([1.0], "2-D")):
        with pytest.raises(ValueError, match=text):
            mx.quantize(bad, "fp4")
    with pytest.raises(ValueError, match="MXMatrix"):
        mx.dequantize(torch.zeros(3, 3))
    with pytest.raises(ValueError, match="unknown activation"):
        mx.act_forward("relu", torch.zeros(3, 3))
