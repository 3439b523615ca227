"""Copied and pickled MXMatrix objects describe memory of their own."""
import copy
import io

import pytest
import torch

from bit_adamw_update_amd import mx

pytestmark = pytest.mark.gpu


def _points_at_its_own(m):
    d = m.desc
    if m.codes.numel() == 0:   # no memory to point at
        return (d.rows, d.cols) == m.shape
    return (d.codes, d.scales) == (m.codes.data_ptr(), m.scales.data_ptr()) and (d.rows, d.cols) == m.shape


def _saved(m):
    f = io.BytesIO()
    torch.save(m, f)
    f.seek(0)
    return torch.load(f, weights_only=False)   # written above


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("rows,cols", [(37, 200), (1, 1), (5, 128), (0, 64), (4, 0)])
@pytest.mark.parametrize("how", [copy.deepcopy, _saved])
def test_a_copy_outlives_the_original(how, rows, cols, fmt, given):
    x = torch.randn(rows, cols, device="cuda")
    m = mx.quantize(x, fmt)
    if given:
        m = mx.MXMatrix(rows, cols, fmt, codes=m.codes.clone(), scales=m.scales.clone())
    want = mx.dequantize(m)
    c = how(m)
    assert _points_at_its_own(c) and _points_at_its_own(m)
    assert c.codes.numel() == 0 or c.codes.data_ptr() != m.codes.data_ptr()
    if m.codes.numel():
        m.codes.fill_(0x11)   # the original's memory, other values
    del m
    assert torch.equal(mx.dequantize(c), want)


def test_a_shallow_copy_shares_the_memory():
    m = mx.quantize(torch.randn(20, 64, device="cuda"), "fp8")
    c = copy.copy(m)
    assert _points_at_its_own(c) and c.codes.data_ptr() == m.codes.data_ptr()
    want = mx.dequantize(m)
    del m
    assert torch.equal(mx.dequantize(c), want)
