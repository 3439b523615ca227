"""Gradients that autograd would lose silently are refused, on the CPU (before
the device is looked at) and on the GPU."""
import pytest
import torch
from torch.autograd import forward_ad

from bit_adamw_update_amd import mx

LOST = "gradient"


def _calls(x, w=None, kept=None):
    """Calls with x as a dense operand; those that need a matrix only where there is one."""
    out = [lambda: mx.act_forward("gelu", x)]
    if w is not None:
        xq = mx.quantize(x.detach(), "fp8")
        out += [lambda: mx.act_forward("swiglu", x.detach(), x),
                lambda: mx.linear(x, w), lambda: mx.linear_dgrad(x, w), lambda: mx.linear_wgrad(x, xq),
                lambda: mx.act_backward("gelu", kept, x), lambda: mx.dequantize(xq, out=x),
                lambda: mx.linear(x.detach(), w, out=x)]
    return out


def _refused(calls):
    for call in calls:
        with pytest.raises(ValueError, match=LOST):
            call()


def test_refused_before_the_device_is_looked_at():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, requires_grad=True)
    _refused(_calls(x))
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        mx.act_forward("gelu", x)
    with pytest.raises(ValueError, match="GPU"):
        mx.act_forward("gelu", x.detach())
    with forward_ad.dual_level():
        d = forward_ad.make_dual(torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(4, 64, dtype=torch.bfloat16))
        _refused(_calls(d))
        with pytest.raises(ValueError, match="GPU"):
            mx.act_forward("gelu", torch.zeros(4, 64, dtype=torch.bfloat16))


@pytest.mark.gpu
def test_every_dense_operand():
    w = mx.quantize(torch.randn(64, 64, device="cuda"), "fp4")
    x = torch.randn(64, 64, device="cuda").to(torch.bfloat16)
    kept = mx.act_forward("gelu", x)[1]
    want = mx.linear(x, w)
    x.requires_grad_()
    _refused(_calls(x, w, kept))
    with torch.no_grad():
        assert torch.equal(mx.linear(x, w), want)
    assert torch.equal(mx.linear(x.detach(), w), want)
    with forward_ad.dual_level():
        d = forward_ad.make_dual(x.detach(), torch.ones_like(x))
        with pytest.raises(ValueError, match=LOST):
            mx.linear(d, w)
        assert torch.equal(mx.linear(x.detach(), w), want)


@pytest.mark.gpu
def test_a_parameter_is_quantized():
    p = torch.nn.Parameter(torch.randn(64, 96, device="cuda"))
    w = mx.quantize(p, "fp4", transpose=True)
    assert torch.equal(w.codes, mx.quantize(p.detach(), "fp4", transpose=True).codes)


class _Linear(torch.autograd.Function):
    """The layer in autograd, for a master stored [in, out]."""

    @staticmethod
    def forward(ctx, x, master):
        w, xq = mx.quantize(master, "fp4", transpose=True), mx.quantize(x, "fp8")
        ctx.kept = w, xq
        return mx.linear(xq, w)

    @staticmethod
    def backward(ctx, dy):
        w, xq = ctx.kept
        return mx.linear_dgrad(dy, w), mx.linear_wgrad(dy, xq, transposed=True, dtype=torch.float32)


@pytest.mark.gpu
def test_from_an_autograd_function():
    master = torch.nn.Parameter(torch.randn(64, 96, device="cuda") * 0.1)
    x = torch.randn(20, 64, device="cuda").to(torch.bfloat16).requires_grad_()
    y = _Linear.apply(x, master)
    dy = torch.randn(20, 96, device="cuda").to(torch.bfloat16)
    y.backward(dy)
    w, xq = mx.quantize(master, "fp4", transpose=True), mx.quantize(x, "fp8")
    assert torch.equal(x.grad, mx.linear_dgrad(dy, w))
    assert torch.equal(master.grad, mx.linear_wgrad(dy, xq, transposed=True, dtype=torch.float32))
