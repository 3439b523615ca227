"""Plain 64-bit implementations of embedding, head norms with rotation, and
dropout, on the CPU, from the definitions in include/q4adamw.h.  They share no
code with the library."""
import math

import numpy as np
import torch

D = torch.float64
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step, relative


def embedding(ids, values, scale):
    """values: the table's, in any type."""
    ids, values = ids.long().cpu(), values.to(D).cpu()
    y = torch.zeros(len(ids), values.shape[1], dtype=D)
    for t, i in enumerate(ids.tolist()):
        if i >= 0:
            y[t] = values[i] * scale if i < values.shape[0] else math.nan
    return y


def embedding_grad(ids, dy, rows, scale):
    """(gradient, the sum of magnitudes behind each element, tokens of each row)."""
    ids, dy = ids.long().cpu(), dy.to(D).cpu()
    real = (ids >= 0) & (ids < rows)
    g, mag = torch.zeros(rows, dy.shape[1], dtype=D), torch.zeros(rows, dy.shape[1], dtype=D)
    g.index_add_(0, ids[real], dy[real])
    mag.index_add_(0, ids[real], dy[real].abs())
    return g * scale, mag * abs(scale), torch.bincount(ids[real], minlength=rows).to(D)


def pairs(dim, rotary, interleaved):
    """(first elements, second elements) of the pairs that turn."""
    i = torch.arange(rotary // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)


def turn(x, angle, interleaved):
    """x [..., heads, dim] with its pairs turned by angle [..., rotary / 2]."""
    a, b = pairs(x.shape[-1], 2 * angle.shape[-1], interleaved)
    c, s = torch.cos(angle)[..., None, :], torch.sin(angle)[..., None, :]
    y = x.clone()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def angles(positions, frequencies):
    return positions.to(D).cpu()[..., None] * frequencies.cpu()


def head_norm_rope(x, gain, positions, frequencies, eps, interleaved):
    x, gain = x.to(D).cpu(), gain.to(D).cpu()
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return turn(n * gain, angles(positions, frequencies), interleaved)


def magnitudes(x, angle, interleaved):
    """|a| + |b| in the place of both elements of a pair that turns, |x| elsewhere: what bounds either after a turn."""
    a, b = pairs(x.shape[-1], 2 * angle.shape[-1], interleaved)
    y = x.abs()
    y[..., a] = y[..., b] = x[..., a].abs() + x[..., b].abs()
    return y


def head_norm_rope_backward(x, gain, positions, frequencies, dy, eps, interleaved):
    """(dx, dgain, and bounds of the errors of the same in FP32)."""
    x, gain, dy = x.to(D).cpu(), gain.to(D).cpu(), dy.to(D).cpu()
    dim, step = x.shape[-1], 2.0 ** -24
    angle = angles(positions, frequencies)
    inv = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n = x * inv
    g = turn(dy, -angle, interleaved)
    big = magnitudes(dy, angle, interleaved)
    dn = g * gain
    dx = inv * (dn - n * (dn * n).mean(-1, keepdim=True))
    rows = dy.numel() // dim
    # inv: half of the sum's dim roundings and a few; g: the angle's cosine and sine, three roundings each;
    # the mean: its own sum of dim terms, each as far off as dn and n are
    mean_mag = (big * gain.abs() * n.abs()).mean(-1, keepdim=True)
    off = inv * step * ((dim / 2 + 24) * big * gain.abs() + (2 * dim + 48) * n.abs() * mean_mag)
    over = tuple(range(dy.dim() - 1))
    return dx, (g * n).sum(over), off, (rows + dim / 2 + 48) * step * (big * n.abs()).sum(over)


def forward_off(x, gain, positions, frequencies, eps, interleaved):
    """A bound of the error of head_norm_rope in FP32: half of the sum's dim roundings and a few, on either of a pair."""
    x, gain = x.to(D).cpu(), gain.to(D).cpu()
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return (x.shape[-1] / 2 + 24) * 2.0 ** -24 * magnitudes(n * gain, angles(positions, frequencies), interleaved)


def philox(counter, key):
    """Philox4x32-10 of one counter, in Python's integers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        p, q = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(q >> 32) ^ c[1] ^ k[0], q & 0xFFFFFFFF, (p >> 32) ^ c[3] ^ k[1], p & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def draws(count, seed, step, layer, offset=0):
    """The 16 random bits of elements offset .. offset + count - 1."""
    out = []
    for g in range(offset // 8, (offset + count + 7) // 8):
        for w in philox((g, step & 0xFFFFFFFF, layer, 2), (seed & 0xFFFFFFFF, seed >> 32)):
            out += [w & 0xFFFF, w >> 16]
    return np.array(out[:count], dtype=np.int64)


def dropout(x, p, seed, step, layer, residual=None, offset=0):
    """(y, kept) in 64 bits."""
    rows, cols = x.shape
    below = int(np.rint(p * 65536))
    kept = torch.from_numpy(draws(rows * cols, seed, step, layer, offset).reshape(rows, cols) >= below)
    y = torch.zeros(rows, cols, dtype=D)
    if below < 65536:
        y[kept] = x.to(D).cpu()[kept] * 65536 / (65536 - below)
    return (y if residual is None else y + residual.to(D).cpu()), kept
