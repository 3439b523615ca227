"""The operators beside a training step's products: real calls, their plain forms
and their definitions in 64 bits.

* embed: rows of the embedding table at the tokens' numbers, times a scale,
  from the FP32 masters, a BF16 copy or a matrix in a microscaled format (for
  every run of 32 columns one power of two, a byte e: 2^(e-127), and 32 codes,
  E2M1 (fp4, two to a byte, the even column in the low half) or E4M3 (fp8);
  the layout is bit_adamw_update_amd.mx.MXMatrix's).  A token below 0 is
  padding and reads zeros;
* embed_grad: the table's gradient, for every row the scale times the sum of
  the result's gradients over the tokens that read it, the whole table in BF16
  as the optimizer takes it;
* heads: queries and keys divided by their root mean square over the head,
  times a gain per element, and rotated by their position: pair i of the
  rotary elements turns by position * frequency[i], pairs being elements i and
  i + R/2, or 2i and 2i + 1 (interleaved); forward, and with "train" backward
  too, from the inputs;
* dropout: an element is kept if 16 random bits are not below p 2^16, and then
  divided by the kept share; on a residual stream added to it.  The bits come
  from Philox4x32-10 under the key (seed), counter (i / 8, step, layer, 2) for
  element i of the row-major matrix: half i mod 8 of its 128 bits.  Backward
  is the same call on the gradient.
"""
import math

import numpy as np
import torch

own = False

FP4, FP8 = "fp4", "fp8"
EPS = 1e-6
THETA = 1e6


# ---- cases ----------------------------------------------------------------

def listed():
    return [
        # a decoding step's token from a tied table in 4 bits: latency
        {"name": "embed one token", "op": "embed", "tokens": 1, "rows": 151936, "cols": 1024, "table": FP4,
         "scaled": False, "ids": "int64"},
        # a micro-batch from the masters of a 2.7 G parameter model
        {"name": "embed 16384x2560", "op": "embed", "tokens": 16384, "rows": 50304, "cols": 2560, "table": "float32",
         "scaled": False, "ids": "int64"},
        # a packed batch of odd length, the result scaled by the width's root
        {"name": "embed 5003x2048 scaled", "op": "embed", "tokens": 5003, "rows": 32000, "cols": 2048,
         "table": "bfloat16", "scaled": True, "ids": "int32"},
        # the gradient of a large vocabulary's table: most of it is rows that no token read
        {"name": "embed_grad 8192 of 151936", "op": "embed_grad", "tokens": 8192, "rows": 151936, "cols": 1024,
         "scaled": False, "ids": "int64"},
        # of a 2.7 G parameter model's
        {"name": "embed_grad 16384 of 50304", "op": "embed_grad", "tokens": 16384, "rows": 50304, "cols": 2560,
         "scaled": False, "ids": "int64"},
        # a small model's on an odd batch, padding behind it
        {"name": "embed_grad 301 of 1000", "op": "embed_grad", "tokens": 301, "rows": 1000, "cols": 100,
         "scaled": True, "ids": "int32"},
        # a decoding step's queries and keys
        {"name": "heads one token", "op": "heads", "tokens": 1, "hq": 16, "hk": 8, "dim": 128, "rotary": 128,
         "interleaved": False, "layout": "fused", "train": False},
        # a micro-batch, forward and backward, out of the fused projection's result
        {"name": "heads 8192 train", "op": "heads", "tokens": 8192, "hq": 16, "hk": 8, "dim": 128, "rotary": 128,
         "interleaved": False, "layout": "fused", "train": True},
        # an odd batch, pairs side by side, half of the head rotated, a head's tokens together
        {"name": "heads 2047 interleaved", "op": "heads", "tokens": 2047, "hq": 32, "hk": 4, "dim": 64, "rotary": 32,
         "interleaved": True, "layout": "by head", "train": True},
        # a long prompt
        {"name": "heads 16001 prompt", "op": "heads", "tokens": 16001, "hq": 32, "hk": 32, "dim": 80, "rotary": 80,
         "interleaved": False, "layout": "split", "train": False},
        # a sublayer's result onto the residual stream and the gradient back
        {"name": "dropout 8192x2560", "op": "dropout", "rows": 8192, "cols": 2560, "dtype": "bfloat16", "p": 0.1,
         "residual": True},
        # an FP32 stream of a small model, odd sizes
        {"name": "dropout 333x771 float32", "op": "dropout", "rows": 333, "cols": 771, "dtype": "float32", "p": 0.25,
         "residual": False},
    ]


def _between(rng, lo, hi):
    """A size spread over the logarithm of [lo, hi]; half of them multiples of 64 where that fits."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if n >= 64 and rng.random() < 0.5:
        n = n // 64 * 64
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "heads", "dropout"])
    if op in ("embed", "embed_grad"):
        cols = _between(rng, 32, 2560)
        c = {"op": op, "tokens": _between(rng, 1, 16384), "rows": _between(rng, 256, min(151936, 128_000_000 // cols)),
             "cols": cols, "scaled": rng.random() < 0.5, "ids": rng.choice(["int64", "int32"])}
        if op == "embed":
            c["table"] = rng.choice(["float32", "bfloat16", FP4, FP8])
        return c
    if op == "heads":
        dim = rng.choice([32, 64, 72, 80, 96, 128, 256])
        hq = rng.choice([4, 8, 12, 16, 32])
        hk = rng.choice([h for h in (1, 2, 4, 8, 12, 16, 32) if hq % h == 0])
        return {"op": op, "tokens": _between(rng, 1, min(16384, 24_000_000 // ((hq + hk) * dim))), "hq": hq, "hk": hk,
                "dim": dim, "rotary": rng.choice([dim, dim, dim // 2]), "interleaved": rng.random() < 0.4,
                "layout": rng.choice(["fused", "split", "by head"]), "train": rng.random() < 0.6}
    return {"op": op, "rows": _between(rng, 1, 8192), "cols": _between(rng, 32, 2560),
            "dtype": rng.choice(["bfloat16", "bfloat16", "float32"]), "p": rng.choice([0.05, 0.1, 0.2, 0.5]),
            "residual": rng.random() < 0.6}


def work(case):
    op = case["op"]
    if op == "embed":
        t, c = case["tokens"], case["cols"]
        held = {"float32": 4, "bfloat16": 2, FP4: 17 / 32, FP8: 33 / 32}[case["table"]]
        # a row that several tokens read is read once
        seen = _distinct(t, case["rows"])
        return {"bytes": int(t * (8 if case["ids"] == "int64" else 4) + c * (held * seen + 2 * t)), "flops": t * c}
    if op == "embed_grad":
        t, c = case["tokens"], case["cols"]
        return {"bytes": int(t * (8 if case["ids"] == "int64" else 4) + 2 * c * (t + case["rows"])), "flops": t * c}
    if op == "heads":
        n = case["tokens"] * (case["hq"] + case["hk"]) * case["dim"]
        # forward: read, write; backward: inputs and gradients in, gradients out
        return {"bytes": n * (4 + (6 if case["train"] else 0)) + 8 * case["tokens"],
                "flops": n * (8 + (20 if case["train"] else 0))}
    n, size = case["rows"] * case["cols"], 2 if case["dtype"] == "bfloat16" else 4
    return {"bytes": n * size * (4 + (1 if case["residual"] else 0)), "flops": 2 * n * 2}


def _distinct(tokens, rows):
    """The number of distinct rows that _ids' tokens are expected to name."""
    edge = np.log(np.arange(1, rows + 2, dtype=np.float64)) / math.log(rows + 1)
    return float(np.sum(-np.expm1(tokens * np.log1p(-np.minimum(np.diff(edge), 1 - 1e-12)))))


# ---- inputs ---------------------------------------------------------------

def _activations(shape, gen):
    """Normal values with a few channels twenty times larger, as residual streams have them."""
    x = torch.randn(shape, generator=gen, device="cuda")
    loud = torch.rand(shape[-1], generator=gen, device="cuda") < 0.005
    return x * torch.where(loud, 20.0, 1.0)


def _gradients(shape, gen):
    """Heavy-tailed values of a loss gradient's size."""
    g = torch.randn(shape, generator=gen, device="cuda")
    chi = torch.randn(shape[:-1] + (1,), generator=gen, device="cuda").abs() + 0.3
    return (g * 1e-3 / chi).to(torch.bfloat16)


def _ids(case, gen):
    """Token numbers with the frequencies of text (the n-th most frequent about 1/n), a few percent of padding at the
    end of a batch of several."""
    t, rows = case["tokens"], case["rows"]
    u = torch.rand(t, generator=gen, device="cuda", dtype=torch.float64)
    rank = ((rows + 1) ** u).long().sub_(1).clamp_(0, rows - 1)
    ids = torch.randperm(rows, generator=gen, device="cuda")[rank]
    if t > 1:
        ids[t - t // 32:] = -1
    return ids.to(getattr(torch, case["ids"]))


def _codes(case, gen):
    """A table in a microscaled format: codes and scale bytes."""
    rows, cols = case["rows"], case["cols"]
    padded = (cols + 127) // 128 * 128
    if case["table"] == FP4:
        c = torch.randint(0, 256, (rows, padded // 2), generator=gen, device="cuda", dtype=torch.uint8)
        if cols % 2:
            c[:, cols // 2] &= 15
        c[:, (cols + 1) // 2:] = 0
    else:
        c = torch.randint(0, 254, (rows, padded), generator=gen, device="cuda", dtype=torch.uint8)
        c += (c >= 127).to(torch.uint8)  # all but the two NaN
        c[:, cols:] = 0
    e = torch.randint(116, 121, (padded // 32, rows), generator=gen, device="cuda", dtype=torch.uint8)
    e[(cols + 31) // 32:] = 0
    return {"rows": rows, "cols": cols, "fmt": case["table"], "codes": c,
            "scales": e.view(padded // 128, 4, rows).transpose(1, 2).contiguous()}


def _laid_out(x, layout):
    """Queries or keys [tokens, heads, dim] as a program has them: "split", a tensor of their own; "by head", a head's
    tokens together."""
    return x.transpose(0, 1).contiguous().transpose(0, 1) if layout == "by head" else x


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    bf, op = torch.bfloat16, case["op"]
    s = {"case": case}
    if op in ("embed", "embed_grad"):
        s["ids"] = _ids(case, gen)
        s["scale"] = math.sqrt(case["cols"]) if case["scaled"] else 1.0
        if op == "embed_grad":
            s["dy"] = _gradients((case["tokens"], case["cols"]), gen)
        elif case["table"] in (FP4, FP8):
            s["table"] = _codes(case, gen)
        else:
            w = torch.randn(case["rows"], case["cols"], generator=gen, device="cuda") * 0.02
            s["table"] = w.to(getattr(torch, case["table"]))
        return s
    if op == "heads":
        t, hq, hk, d = case["tokens"], case["hq"], case["hk"], case["dim"]
        if case["layout"] == "fused":  # views of the projection's result, values behind the keys
            x = _activations((t, (hq + 2 * hk) * d), gen).to(bf)
            s["q"], s["k"] = x[:, :hq * d].view(t, hq, d), x[:, hq * d:(hq + hk) * d].view(t, hk, d)
        else:
            s["q"], s["k"] = (_laid_out(_activations((t, h, d), gen).to(bf), case["layout"]) for h in (hq, hk))
        s["q_gain"], s["k_gain"] = (1 + 0.3 * torch.randn(d, generator=gen, device="cuda") for _ in range(2))
        # a packed batch's positions, or those of a token far into its sequence
        first = int(torch.randint(0, 100_000, (1,), generator=gen, device="cuda"))
        s["positions"] = torch.arange(t, device="cuda") + first
        s["positions"][t // 3:] -= first + t // 3
        s["frequencies"] = THETA ** (-torch.arange(case["rotary"] // 2, device="cuda", dtype=torch.float64)
                                     * 2 / case["rotary"])
        if case["train"]:
            s["dq"], s["dk"] = (_laid_out(_gradients((t, h, d), gen), case["layout"]) for h in (hq, hk))
        return s
    shape, dtype = (case["rows"], case["cols"]), getattr(torch, case["dtype"])
    s["x"], s["dy"] = _activations(shape, gen).to(dtype), _gradients(shape, gen).to(dtype)
    s["residual"] = _activations(shape, gen).to(dtype) if case["residual"] else None
    s["key"] = {"seed": seed * 0x9E3779B97F4A7C15 % (1 << 64), "step": seed % 1000 + 1, "layer": seed % 61}
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own and isinstance(s.get("table"), dict):  # the handle that a program keeps of its codes
        from bit_adamw_update_amd import mx
        h = s["table"]
        s["table"] = mx.MXMatrix(h["rows"], h["cols"], h["fmt"], codes=h["codes"], scales=h["scales"])
    return s


# ---- the plain forms ------------------------------------------------------

def _code_rows(h, ids):
    """The rows at ids of a table in a microscaled format, in FP32."""
    c = h["codes"][ids].int()
    if h["fmt"] == FP4:
        c = torch.stack((c & 15, c >> 4), 2).flatten(1)
        sign, n = c >> 3, c & 7
        a = torch.where(n < 4, n * 0.5, torch.where(n < 6, n - 2.0, n * 2.0 - 8.0))
    else:
        sign, n = c >> 7, c & 127
        man = torch.where(n < 8, n, (n & 7) + 8)
        a = man.float() * torch.exp2((n >> 3).clamp(min=1).float() - 10)
    s = torch.exp2(h["scales"][:, ids].transpose(0, 1).flatten(1).float() - 127).repeat_interleave(32, 1)
    return (torch.where(sign == 1, -a, a) * s)[:, :h["cols"]]


def _turned(x, cos, sin, rotary, interleaved):
    """x [tokens, heads, dim] with its rotary elements turned by the angles of cos and sin [tokens, 1, rotary / 2]."""
    r, rest = x[..., :rotary], x[..., rotary:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r[..., :rotary // 2], r[..., rotary // 2:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, rest), -1)


def _heads_plain(s, x, gain, dy, cos, sin):
    c, bf = s["case"], torch.bfloat16
    x, gain = x.float(), gain.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    out = [_turned(x * r * gain, cos, sin, c["rotary"], c["interleaved"]).to(bf)]
    if dy is not None:
        g = _turned(dy.float(), cos, -sin, c["rotary"], c["interleaved"])
        n = x * r
        dn = g * gain
        out += [(r * (dn - n * (dn * n).mean(-1, keepdim=True))).to(bf), (g * n).sum((0, 1)).to(bf)]
    return out


def _kept(case, key):
    """Which elements dropout keeps: Philox4x32-10 in whole numbers of 64 bits, whose products wrap around."""
    rows, cols = case["rows"], case["cols"]
    low = 0xFFFFFFFF
    x = torch.arange((rows * cols + 7) // 8, device="cuda")
    y, z, w = (torch.full_like(x, v) for v in (key["step"], key["layer"], 2))
    k0, k1 = key["seed"] & low, key["seed"] >> 32
    for _ in range(10):
        p, q = 0xD2511F53 * x, 0xCD9E8D57 * z
        x, y, z, w = ((q >> 32) & low) ^ y ^ k0, q & low, ((p >> 32) & low) ^ w ^ k1, p & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    bits = torch.stack([h for v in (x, y, z, w) for h in (v & 0xFFFF, v >> 16)], 1).flatten()[:rows * cols]
    return bits.view(rows, cols) >= round(case["p"] * 65536)


def _plain(s):
    c, bf = s["case"], torch.bfloat16
    if c["op"] == "embed":
        ids, real = s["ids"].clamp(min=0), (s["ids"] >= 0)[:, None]
        rows = _code_rows(s["table"], ids) if isinstance(s["table"], dict) else s["table"][ids].float()
        return torch.where(real, rows * s["scale"], 0.0).to(bf)
    if c["op"] == "embed_grad":
        real = s["ids"] >= 0
        sums = torch.zeros(c["rows"], c["cols"], device="cuda")
        return (sums.index_add_(0, s["ids"][real], s["dy"][real].float()) * s["scale"]).to(bf)
    if c["op"] == "heads":
        angle = s["positions"].double()[:, None, None] * s["frequencies"]
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
        q = _heads_plain(s, s["q"], s["q_gain"], s.get("dq"), cos, sin)
        k = _heads_plain(s, s["k"], s["k_gain"], s.get("dk"), cos, sin)
        return tuple(v for pair in zip(q, k) for v in pair)
    kept, share = _kept(c, s["key"]), 1 - round(c["p"] * 65536) / 65536
    y = torch.where(kept, s["x"].float() / share, 0.0)
    y = y if s["residual"] is None else y + s["residual"].float()
    return y.to(s["x"].dtype), torch.where(kept, s["dy"].float() / share, 0.0).to(s["x"].dtype)


def _own(s):
    from bit_adamw_update_amd import layers
    c = s["case"]
    if c["op"] == "embed":
        return layers.embedding(s["ids"], s["table"], scale=s["scale"])
    if c["op"] == "embed_grad":
        return layers.embedding_grad(s["ids"], s["dy"], c["rows"], scale=s["scale"])
    if c["op"] == "heads":
        how = {"eps": EPS, "interleaved": c["interleaved"]}
        fixed = s["q"], s["k"], s["q_gain"], s["k_gain"], s["positions"], s["frequencies"]
        out = layers.head_norm_rope(*fixed, **how)
        return out + layers.head_norm_rope_backward(*fixed, s["dq"], s["dk"], **how) if c["train"] else out
    return (layers.dropout(s["x"], c["p"], **s["key"], residual=s["residual"]),
            layers.dropout(s["dy"], c["p"], **s["key"]))


def run(state):
    return _own(state) if own else _plain(state)


# ---- the definition, in 64 bits -------------------------------------------

def _table(fmt):
    """The values of all codes of a format, from its fields."""
    mbits, bias, half = (1, 1, 8) if fmt == FP4 else (3, 7, 128)
    v = [math.ldexp(c & ((1 << mbits) - 1), 1 - bias - mbits) if c >> mbits == 0 else
         math.ldexp((1 << mbits) + (c & ((1 << mbits) - 1)), (c >> mbits) - bias - mbits) for c in range(half)]
    if fmt == FP8:
        v[127] = math.nan
    return torch.tensor(v + [-u for u in v], dtype=torch.float64, device="cuda")


def _row_values(h, ids):
    raw = h["codes"].index_select(0, ids).long()
    if h["fmt"] == FP4:
        wide = torch.empty(raw.shape[0], 2 * raw.shape[1], dtype=torch.long, device=raw.device)
        wide[:, 0::2], wide[:, 1::2] = raw % 16, raw // 16
        raw = wide
    power = torch.exp2(h["scales"].index_select(1, ids).double() - 127).permute(1, 0, 2).reshape(len(ids), -1, 1)
    return (_table(h["fmt"])[raw].view(len(ids), -1, 32) * power).reshape(len(ids), -1)[:, :h["cols"]]


def _rotation(x, z, rotary, interleaved):
    """x's rotary pairs as complex numbers, times z."""
    r = x[..., :rotary]
    pair = (torch.complex(r[..., 0::2].contiguous(), r[..., 1::2].contiguous()) if interleaved else
            torch.complex(r[..., :rotary // 2].contiguous(), r[..., rotary // 2:].contiguous())) * z
    y = x.clone()
    if interleaved:
        y[..., 0:rotary:2], y[..., 1:rotary:2] = pair.real, pair.imag
    else:
        y[..., :rotary // 2], y[..., rotary // 2:rotary] = pair.real, pair.imag
    return y


def _heads_exact(s, x, gain, dy, z):
    c = s["case"]
    x, gain = x.double(), gain.double()
    rms = torch.sqrt((x ** 2).sum(-1, keepdim=True) / c["dim"] + EPS)
    out = [_rotation(x / rms * gain, z, c["rotary"], c["interleaved"])]
    if dy is not None:
        g = _rotation(dy.double(), z.conj(), c["rotary"], c["interleaved"])
        # d(x_j / rms) / dx_i = (i == j) / rms - x_i x_j / (dim rms^3)
        along = (g * gain * x).sum(-1, keepdim=True) / (c["dim"] * rms ** 3)
        out += [g * gain / rms - x * along, (g * x / rms).flatten(0, 1).sum(0)]
    return out


def _philox(x, step, layer, stream, seed):
    """Philox4x32-10's four words for the counters (x, step, layer, stream), by numpy on the host."""
    word, m = np.uint64(32), np.uint64(0xFFFFFFFF)
    c = [x.astype(np.uint64)] + [np.full(x.shape, v, dtype=np.uint64) for v in (step, layer, stream)]
    for r in range(10):
        k0 = np.uint64(((seed & 0xFFFFFFFF) + r * 0x9E3779B9) & 0xFFFFFFFF)
        k1 = np.uint64(((seed >> 32) + r * 0xBB67AE85) & 0xFFFFFFFF)
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> word) ^ c[1] ^ k0, b & m, (a >> word) ^ c[3] ^ k1, a & m]
    return np.stack(c, 1).astype(np.uint32)


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "embed":
        ids = s["ids"].long()
        y = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device="cuda")
        at = torch.nonzero(ids >= 0).flatten()
        rows = _row_values(s["table"], ids[at]) if isinstance(s["table"], dict) else s["table"].index_select(0, ids[at]).double()
        y[at] = rows * s["scale"]
        return y
    if case["op"] == "embed_grad":
        ids = s["ids"].long()
        g = torch.zeros(case["rows"] + 1, case["cols"], dtype=torch.float64, device="cuda")
        g.index_put_((torch.where(ids < 0, case["rows"], ids),), s["dy"].double() * s["scale"], accumulate=True)
        return g[:-1]
    if case["op"] == "heads":
        angle = torch.outer(s["positions"].double(), s["frequencies"])[:, None]
        z = torch.polar(torch.ones_like(angle), angle)
        q = _heads_exact(s, s["q"], s["q_gain"], s.get("dq"), z)
        k = _heads_exact(s, s["k"], s["k_gain"], s.get("dk"), z)
        return (q[0], k[0]) + ((q[1], k[1], q[2], k[2]) if case["train"] else ())
    n, key = case["rows"] * case["cols"], s["key"]
    words = _philox(np.arange((n + 7) // 8), key["step"], key["layer"], 2, key["seed"])
    drawn = torch.from_numpy(words.view("<u2").reshape(-1)[:n].astype(np.int32)).cuda().view(case["rows"], case["cols"])
    below = round(case["p"] * 65536)
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    y, dx = (torch.where(drawn < below, zero, s[v].double() * 65536 / (65536 - below)) for v in ("x", "dy"))
    return (y if s["residual"] is None else y + s["residual"].double()), dx
