"""linear's sums are FP32 sums of exact products, whatever the format of x.

Two products of far-apart sizes: E4M3 256 and 2^-9 (its smallest value), E2M1
1 and 0.5, so 256 + 2^-10, 19 bits, which FP32 holds.  FP32 additions in any
order, zeros among them, give exactly that; a sum on a coarser grid does not.
Random operands: (K + 16) 2^-23 of the sum of magnitudes S, as each of at most
K additions is off by at most a step (2^-23) of a partial sum of at most S, and
half a step of the result's type.
"""
import pytest
import torch

import mx_reference as ref
from bit_adamw_update_amd import mx

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _pairs(n):
    """Every ordered pair of different columns of the first n."""
    a = torch.arange(n)
    i, j = torch.meshgrid(a, a, indexing="ij")
    keep = i != j
    return i[keep], j[keep]


def _two_products():
    """(codes of x, FP4 values of w [2 blocks of rows], pairs): row p of x holds 256 and
    2^-9 in columns i, j of pair p; w has 1 or 0.5 in every column."""
    i, j = _pairs(24)
    codes = torch.zeros(len(i), 128, dtype=torch.uint8)
    codes[torch.arange(len(i)), i] = 0x78   # 2^8
    codes[torch.arange(len(i)), j] = 0x01   # 2^-9
    return codes


@pytest.mark.parametrize("tokens,outs", [(16, 40), (100, 40), (552, 300), (552, 70000)])
def test_two_products_of_far_apart_sizes(tokens, outs):
    print("two products", tokens, outs, flush=True)
    codes = _two_products()
    rows = torch.arange(tokens) * (len(codes) // tokens)
    scales = torch.zeros(1, tokens, 4, dtype=torch.uint8)
    scales[0, :, 0] = 127
    x = mx.MXMatrix(tokens, 128, "fp8", codes=codes[rows].contiguous().to(DEV), scales=scales.to(DEV))
    # output o has 1 in the columns of parity o and 0.5 in the others
    w = torch.full((outs, 128), 0.5)
    w[0::2, 0::2] = 1
    w[1::2, 1::2] = 1
    w[:, 31] = 6.0   # keeps the block's scale at 1
    wq = mx.quantize(w.to(DEV), "fp4")
    assert torch.equal(mx.dequantize(wq, torch.float32).cpu()[:, :31], w[:, :31])
    y = mx.linear(x, wq, dtype=torch.float32)
    want = ref.values_of(x).to(DEV) @ w.double().to(DEV).t()
    wrong = int((y.double() != want).sum())
    assert wrong == 0


@pytest.mark.parametrize("tokens", [1, 16, 17, 40])
def test_two_products_from_bf16(tokens):
    """The same through the quantization on the way: 256 keeps the scale at 1."""
    i, j = _pairs(16)
    x = torch.zeros(tokens, 128)
    t = torch.arange(tokens)
    x[t, i[t * 5]] = 256.0
    x[t, j[t * 5]] = 2.0 ** -9
    w = torch.full((50, 128), 1.0)
    w[:, 31] = 6.0
    y = mx.linear(x.to(DEV, torch.bfloat16), mx.quantize(w.to(DEV), "fp4"), dtype=torch.float32)
    wrong = int((y != 256.0 + 2.0 ** -9).sum())
    assert wrong == 0


SIZES = [(1, 2048, 300), (7, 129, 65), (16, 256, 128), (17, 384, 100), (64, 500, 130), (257, 1000, 300)]


@pytest.mark.parametrize("xfmt", ["fp8", "fp4", "bf16"])
@pytest.mark.parametrize("tokens,cin,cout", SIZES)
def test_sums_of_random_products(tokens, cin, cout, xfmt):
    print("sums", tokens, cin, cout, xfmt, flush=True)
    g = torch.Generator().manual_seed(5)
    x = torch.randn(tokens, cin, generator=g) * torch.where(torch.rand(cin, generator=g) < 0.02, 20.0, 1.0)
    x = x.to(torch.bfloat16)
    w = mx.quantize((torch.randn(cout, cin, generator=g) * 0.02).to(DEV), "fp4")
    wv = ref.values_of(w)
    if xfmt == "bf16":
        operand, xv = x.to(DEV), ref.values(*ref.quantize(x, "fp8"), cin, "fp8")
    else:
        operand = mx.quantize(x.to(DEV), xfmt)
        xv = ref.values_of(operand)
    want, terms = xv @ wv.t(), xv.abs() @ wv.abs().t()
    for dtype in (torch.bfloat16, torch.float32):
        y = mx.linear(operand, w, dtype=dtype).double().cpu()
        tol = (cin + 16) * 2.0 ** -23 * terms * (1 + HALF_STEP[dtype]) + want.abs() * HALF_STEP[dtype]
        worst = ((y - want).abs() / tol.clamp(min=1e-300)).max().item()
        assert worst <= 1
