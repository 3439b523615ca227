"""Every code under every scale through the products: with the identity as the
other operand a result is one product and zeros, so it is the code's value as
it enters the product, exact in FP32 above 2^-126 and BF16's value of it below.

Values past FP32's range and NaN codes are left out: times the identity's
zeros they reach the whole row, as they should.
"""
import pytest
import torch

import mx_reference as ref
from bit_adamw_update_amd import mx

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _all_codes(fmt):
    """(MXMatrix 255 x 256, its values): row e has scale e, column c code c (fp4: c % 16)."""
    codes = torch.arange(256, dtype=torch.uint8).repeat(255, 1)
    if fmt == "fp4":
        codes = codes % 16
    scales = torch.arange(255, dtype=torch.uint8)[:, None].repeat(1, 8)
    values = ref.values(codes, scales, 256, fmt)
    codes[~(values.abs() < 2.0 ** 128)] = 0
    values = ref.values(codes, scales, 256, fmt)
    packed = codes[:, 0::2] | (codes[:, 1::2] << 4) if fmt == "fp4" else codes
    return (mx.MXMatrix(255, 256, fmt, codes=packed.contiguous().to(DEV),
                        scales=scales.view(255, -1, 4).transpose(0, 1).contiguous().to(DEV)), values)


def _rows(m, rows):
    return mx.MXMatrix(len(rows), m.cols, m.format, codes=m.codes[rows].contiguous(),
                       scales=m.scales[:, rows].contiguous())


def _same(got, values):
    want = values.float().to(torch.bfloat16).float()   # FP32 holds every value
    wrong = (got.cpu() != want).nonzero()
    assert len(wrong) == 0, (len(wrong), wrong[:3].tolist())


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_codes_of_x_in_linear(fmt):
    x, values = _all_codes(fmt)
    eye = mx.quantize(torch.eye(256, device=DEV), "fp4")
    assert torch.equal(mx.dequantize(eye, torch.float32).cpu(), torch.eye(256))
    _same(mx.linear(x, eye, dtype=torch.float32), values)
    for at in range(0, 255, 15):
        rows = list(range(at, at + 15))
        _same(mx.linear(_rows(x, rows), eye, dtype=torch.float32), values[rows])


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_codes_of_w_in_linear(fmt):
    w, values = _all_codes("fp4")
    eye = mx.quantize(torch.eye(256, device=DEV), fmt)
    _same(mx.linear(eye, w, dtype=torch.float32).t(), values)
    for at in (0, 128, 240):
        _same(mx.linear(_rows(eye, list(range(at, at + 16))), w, dtype=torch.float32).t(), values[:, at:at + 16])


def test_codes_in_the_gradients():
    eye = torch.eye(255, dtype=torch.bfloat16, device=DEV)
    w, values = _all_codes("fp4")
    _same(mx.linear_dgrad(eye, w, dtype=torch.float32), values)
    for fmt in ("fp8", "fp4"):
        x, values = _all_codes(fmt)
        _same(mx.linear_wgrad(eye, x, dtype=torch.float32), values)
