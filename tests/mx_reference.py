"""Plain 64-bit implementation of the microscaled formats and of the linear
layer's operators, on the CPU, from the definitions in include/q4adamw.h.
Shares no code with the library."""
import math

import torch

FP4_VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
FP8_VALUES = [math.ldexp(c & 7, -9) if c < 8 else math.ldexp(8 + (c & 7), (c >> 3) - 10) for c in range(127)]
VALUES = {"fp4": FP4_VALUES, "fp8": FP8_VALUES}


def padded(cols):
    return (cols + 127) // 128 * 128


def block_scale(amax, top):
    """Smallest k >= -127 with amax / 2^k <= top; the byte k + 127."""
    k = -127
    if amax > 0:
        k = max(k, math.frexp(amax / top)[1] - 2)   # one below the answer at most
        while math.ldexp(amax, -k) > top:
            k += 1
    return k + 127


def quantize(x, fmt):
    """(codes one per byte [rows, P], scale bytes [rows, P / 32]) of x."""
    x = x.double().cpu()
    rows, cols = x.shape
    grid = torch.tensor(VALUES[fmt], dtype=torch.float64)
    p = torch.zeros(rows, padded(cols), dtype=torch.float64)
    p[:, :cols] = x
    blocks = p.view(-1, 32)
    scales = torch.zeros(blocks.shape[0], dtype=torch.uint8)
    amax = blocks.abs().amax(1)
    for i, a in enumerate(amax.tolist()):
        scales[i] = 255 if not math.isfinite(a) else block_scale(a, VALUES[fmt][-1])
    bad = scales == 255
    s = torch.ldexp(torch.ones(1, dtype=torch.float64), scales.double() - 127)[:, None]
    a = torch.where(bad[:, None], torch.zeros_like(blocks), blocks.abs() / s)
    hi = torch.searchsorted(grid, a.contiguous()).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    dhi, dlo = grid[hi] - a, a - grid[lo]
    code = torch.where((dhi < dlo) | ((dhi == dlo) & (hi % 2 == 0)), hi, lo)
    code = code + torch.signbit(blocks).long() * (8 if fmt == "fp4" else 128)
    code[bad] = 0
    return code.to(torch.uint8).view(rows, -1), scales.view(rows, -1)


def values(codes, scales, cols, fmt):
    """The 64-bit values of codes (one per byte) and scale bytes (natural order)."""
    n, half = len(VALUES[fmt]), 8 if fmt == "fp4" else 128
    t = torch.full((2 * half,), math.nan, dtype=torch.float64)
    t[:n] = torch.tensor(VALUES[fmt], dtype=torch.float64)
    t[half:half + n] = -t[:n]
    s = torch.where(scales == 255, math.nan, torch.ldexp(torch.ones(1, dtype=torch.float64), scales.double() - 127))
    return (t[codes.long()].view(codes.shape[0], -1, 32) * s[:, :, None]).reshape(codes.shape[0], -1)[:, :cols]


def unpack(m):
    """An MXMatrix's codes one per byte and its scale bytes in natural order."""
    c = m.codes.cpu()
    if m.format == "fp4":
        c = torch.stack((c & 15, c >> 4), 2).flatten(1)
    return c, m.scales.cpu().permute(1, 0, 2).reshape(m.rows, -1)


def values_of(m):
    return values(*unpack(m), m.cols, m.format)


def act(kind, x):
    """f(x) and f'(x) in 64 bits."""
    if kind == "swiglu":
        s = torch.sigmoid(x)
        return x * s, s * (1 + x * torch.sigmoid(-x))
    if kind == "gelu":
        k = math.sqrt(2 / math.pi)
        u = k * (x + 0.044715 * x ** 3)
        # 1 + tanh u = 2 sigmoid(2u) keeps the small values of negative x
        s = torch.sigmoid(2 * u)
        return x * s, s + x * s * torch.sigmoid(-2 * u) * 2 * k * (1 + 3 * 0.044715 * x ** 2)
    phi = 0.5 * torch.special.erfc(-x / math.sqrt(2))
    return x * phi, phi + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
