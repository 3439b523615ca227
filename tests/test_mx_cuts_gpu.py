"""The products' cuts: tiles of both sizes, whole and split along the sum, one
and many to a work-group, over sums deep enough that the rings of steps wrap.

Operands are whole numbers times small powers of two, and every partial sum is
a number that FP32 holds exactly, so every element of every result is compared
bit for bit with an FP32 product (BF16 results: with its rounding); a lost,
doubled or stale run, step or tile shows.
"""
import pytest
import torch

from bit_adamw_update_amd import api, mx

pytestmark = pytest.mark.gpu
DEV = "cuda"
# values and their codes; the two formats' codes of 0, 1, 2, -1, -2
VALUES = [0.0, 1.0, 2.0, -1.0, -2.0]
CODES = {"fp4": [0, 2, 4, 10, 12], "fp8": [0, 0x38, 0x40, 0xB8, 0xC0]}


def _matrix(rows, cols, fmt, seed):
    """(MXMatrix, its values in FP32): values of VALUES, scales 1/2, 1 or 2."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    padded = (cols + 127) // 128 * 128
    pick = torch.randint(0, 5, (rows, padded), device=DEV, generator=g, dtype=torch.uint8)
    pick[:, cols:] = 0
    codes = torch.tensor(CODES[fmt], dtype=torch.uint8, device=DEV)[pick.int()]
    if fmt == "fp4":
        codes = codes[:, 0::2] | (codes[:, 1::2] << 4)
    e = torch.randint(126, 129, (rows, padded // 32), device=DEV, generator=g, dtype=torch.uint8)
    e[:, (cols + 31) // 32:] = 0
    scales = e.view(rows, -1, 4).transpose(0, 1).contiguous()
    values = torch.tensor(VALUES, device=DEV)[pick.int()].view(rows, -1, 32) * torch.exp2(e.float() - 127)[:, :, None]
    return (mx.MXMatrix(rows, cols, fmt, codes=codes.contiguous(), scales=scales),
            values.view(rows, -1)[:, :cols].contiguous())


def _dense(rows, cols, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-3, 4, (rows, cols), device=DEV, generator=g).to(torch.bfloat16)


def _into(shape, dtype, gap):
    """A result of that shape inside a larger buffer, and the check that only it was written."""
    rows, cols = shape
    buf = torch.full((rows + 2, cols + gap), 77.0, dtype=dtype, device=DEV)
    view = buf[1:rows + 1, gap // 2:gap // 2 + cols]

    def untouched():
        inner = view.clone()
        view.fill_(77.0)
        ok = bool((buf == 77.0).all())
        view.copy_(inner)
        return ok

    return view, untouched


def _check(call, want, add=False):
    for dtype, gap in ((torch.float32, 0), (torch.bfloat16, 0), (torch.float32, 5), (torch.bfloat16, 3)):
        out, untouched = _into(want.shape, dtype, gap)
        if add:
            out.fill_(1.0)
        call(out)
        wrong = int((out != (want + 1 if add else want).to(dtype)).sum())
        assert wrong == 0, (dtype, gap, wrong)
        assert untouched()


# (format of x, tokens, in, out, split): split tells whether the plan joins runs
LINEAR = [("fp8", 39, 2916, 320, True), ("fp8", 512, 5120, 2048, True), ("fp8", 3233, 1245, 2484, True),
          ("fp8", 684, 6850, 5498, True), ("fp8", 6639, 446, 5018, True), ("fp8", 4611, 1283, 4099, False),
          ("fp8", 8200, 1283, 8200, False), ("fp8", 3001, 1100, 5001, False),
          ("fp4", 39, 2916, 320, True), ("fp4", 512, 5120, 2048, True), ("fp4", 3356, 5982, 2337, True),
          ("fp4", 2953, 1879, 5472, True), ("fp4", 4200, 1300, 4100, False), ("fp4", 6458, 33, 2468, False),
          ("fp4", 4037, 3822, 2048, False)]


@pytest.mark.parametrize("fmt,tokens,cin,cout,split", LINEAR)
def test_linear(fmt, tokens, cin, cout, split):
    print("linear", fmt, tokens, cin, cout, flush=True)
    x, xv = _matrix(tokens, cin, fmt, 1)
    w, wv = _matrix(cout, cin, "fp4", 2)
    assert (api.q4mx_linear_workspace_bytes(x.desc, w.desc) > 0) == split
    want = xv @ wv.t()
    _check(lambda out: mx.linear(x, w, out=out), want)


@pytest.mark.parametrize("tokens,cin,cout", [(39, 2916, 320), (512, 5120, 2048), (684, 6850, 5498)])
def test_linear_from_bf16(tokens, cin, cout):
    """Values whose largest of a block is 2 times its scale: quantized exactly."""
    print("linear bf16", tokens, cin, cout, flush=True)
    _, xv = _matrix(tokens, cin, "fp8", 3)
    w, wv = _matrix(cout, cin, "fp4", 4)
    quantized = (tokens * (cin + 127) // 128 * 128) * 33 // 32
    assert api.q4mx_linear_bf16_workspace_bytes(tokens, w.desc) > quantized + 65536
    _check(lambda out: mx.linear(xv.to(torch.bfloat16), w, out=out), xv @ wv.t())


DGRAD = [(41, 32, 491, True), (100, 300, 1000, True), (931, 2721, 6015, True), (7217, 2201, 466, True),
         (4774, 3402, 458, True), (4611, 4099, 1283, False), (6835, 2328, 32, False), (1322, 5934, 200, False)]


@pytest.mark.parametrize("tokens,cin,cout,split", DGRAD)
def test_dgrad(tokens, cin, cout, split):
    print("dgrad", tokens, cin, cout, flush=True)
    w, wv = _matrix(cout, cin, "fp4", 5)
    dy = _dense(tokens, cout, 6)
    copy = 0 if cout % 8 == 0 else tokens * (cout + 7) // 8 * 16 + 256
    assert (api.q4mx_dgrad_workspace_bytes(dy.data_ptr(), cout, tokens, w.desc) > copy + 65536) == split
    _check(lambda out: mx.linear_dgrad(dy, w, out=out), dy.float() @ wv)


WGRAD = [(597, 32, 37, True), (4097, 128, 64, True), (5684, 450, 5484, True), (518, 7416, 2294, True),
         (487, 3394, 4748, True), (1283, 4099, 4611, False), (76, 8189, 898, False), (32, 4754, 3511, False)]


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("tokens,cin,n,split", WGRAD)
def test_wgrad(tokens, cin, n, split, fmt):
    print("wgrad", tokens, cin, n, fmt, flush=True)
    x, xv = _matrix(tokens, cin, fmt, 7)
    dy = _dense(tokens, n, 8)
    copy = 0 if n % 8 == 0 else tokens * ((n + 7) // 8) * 16 + 256
    assert (api.q4mx_wgrad_workspace_bytes(dy.data_ptr(), n, n, x.desc) > copy + 65536) == split
    want = dy.float().t() @ xv
    for transposed in (False, True):
        w = want.t().contiguous() if transposed else want
        for add in (False, True):
            _check(lambda out: mx.linear_wgrad(dy, x, out=out, transposed=transposed, accumulate=add), w, add)


@pytest.mark.parametrize("fill", [0, 127, 255])   # 0, 3.4e38, NaN as FP32; 255 is also a NaN scale byte
def test_split_products_in_a_workspace_of_arbitrary_contents(fill):
    """The calls' workspaces, filled, of exactly the bytes they ask for and with
    bytes behind them that stay."""
    def workspace(n):
        ws = torch.full((n + 256,), fill, dtype=torch.uint8, device=DEV)
        return ws, lambda: bool((ws[n:] == fill).all())

    def check(need, at_least, call, want):
        assert need >= at_least + 65536   # runs' sums, beyond any copy
        ws, behind = workspace(need)
        out = torch.full(want.shape, float("nan"), dtype=torch.bfloat16, device=DEV)
        call(out, ws, need)
        assert int((out != want.to(torch.bfloat16)).sum()) == 0 and behind()

    bf, stream = api.MX_BF16, None
    for fmt in ("fp8", "fp4"):
        x, xv = _matrix(39, 2916, fmt, 9)
        w, wv = _matrix(320, 2916, "fp4", 10)
        check(api.q4mx_linear_workspace_bytes(x.desc, w.desc), 0,
              lambda o, ws, n: api.q4mx_linear(x.desc, w.desc, o, bf, 320, ws, n, stream), xv @ wv.t())
    xb = xv.to(torch.bfloat16)
    check(api.q4mx_linear_bf16_workspace_bytes(39, w.desc), 39 * 2944 * 33 // 32,
          lambda o, ws, n: api.q4mx_linear_bf16(xb, 2916, 39, w.desc, o, bf, 320, ws, n, stream), xv @ wv.t())
    w, wv = _matrix(1001, 300, "fp4", 11)
    dy = _dense(100, 1001, 12)
    check(api.q4mx_dgrad_workspace_bytes(dy, 1001, 100, w.desc), 100 * 1008 * 2,
          lambda o, ws, n: api.q4mx_dgrad(dy, 1001, 100, w.desc, o, bf, 300, ws, n, stream), dy.float() @ wv)
    x, xv = _matrix(4097, 128, "fp8", 13)
    dy = _dense(4097, 61, 14)
    check(api.q4mx_wgrad_workspace_bytes(dy, 61, 61, x.desc), 4097 * 64 * 2,
          lambda o, ws, n: api.q4mx_wgrad(dy, 61, 61, x.desc, o, bf, 128, 0, ws, n, stream), dy.float().t() @ xv)


def test_two_split_products_at_once_in_graphs():
    """Two captured layers with workspaces of their own, replayed on two
    streams at once, against the eager results."""
    x, xv = _matrix(512, 5120, "fp8", 15)
    w, wv = _matrix(2048, 5120, "fp4", 16)
    dy = _dense(512, 2048, 17)
    want = (xv @ wv.t(), dy.float() @ wv, dy.float().t() @ xv)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    held = []
    mx.linear(x, w), mx.linear_dgrad(dy, w), mx.linear_wgrad(dy, x)
    torch.cuda.synchronize()
    for _ in streams:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held.append((graph, mx.linear(x, w, dtype=torch.float32), mx.linear_dgrad(dy, w, dtype=torch.float32),
                         mx.linear_wgrad(dy, x, dtype=torch.float32)))
    for _ in range(4):
        for _, *results in held:
            for r in results:
                r.fill_(float("nan"))
        torch.cuda.synchronize()
        for s, (graph, *_) in zip(streams, held):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for _, *results in held:
            for r, v in zip(results, want):
                assert int((r != v).sum()) == 0


def test_activations_with_some_outputs_only():
    """The C call writes what is given: y, its codes and the checkpoints, each alone."""
    g = torch.Generator(device=DEV).manual_seed(18)
    x = torch.randn(37, 300, device=DEV, generator=g).to(torch.bfloat16)
    up = torch.randn(37, 300, device=DEV, generator=g).to(torch.bfloat16)
    for kind, act in mx.ACTIVATIONS.items():
        u = up if kind == "swiglu" else None
        y, kept = mx.act_forward(kind, x, u)
        ymx, _ = mx.act_forward(kind, x, u, out_format="fp4")
        args = (act, x, 300, u, 300 if u is not None else 0, 37, 300)
        got = torch.full_like(y, 7.0)
        api.q4mx_act_forward(*args, got, 300)
        assert torch.equal(got, y)
        m = mx.MXMatrix(37, 300, "fp4")
        api.q4mx_act_forward(*args, None, 300, m.desc)
        assert torch.equal(m.codes, ymx.codes) and torch.equal(m.scales, ymx.scales)
        for i, k in enumerate(kept):
            if k is not None:
                m = mx.MXMatrix(37, 300, "fp8")
                api.q4mx_act_forward(*args, None, 300, None, *((m.desc, None) if i == 0 else (None, m.desc)))
                assert torch.equal(m.codes, k.codes) and torch.equal(m.scales, k.scales)
