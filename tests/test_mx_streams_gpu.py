"""stream=: memory of temporaries on another stream.  A side stream is kept
busy by a bounded wait (torch's _sleep), so that work queued behind it has not
run when the memory is asked for again."""
import pytest
import torch

from bit_adamw_update_amd import mx

pytestmark = pytest.mark.gpu
DEV = "cuda"
BUSY = 100_000_000   # counts of a clock of 100 MHz or more: at most a second


def _normal(rows, cols, seed, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(rows, cols, generator=g).to(DEV, dtype)


def _span(t):
    if isinstance(t, mx.MXMatrix):
        return t.codes.data_ptr(), t.scales.data_ptr() + t.scales.numel()
    return t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()


def _apart(a, b):
    return a[1] <= b[0] or b[1] <= a[0]


def _keep_busy(stream):
    with torch.cuda.stream(stream):
        torch.cuda._sleep(BUSY)


def _still_busy(stream):
    if stream.query():
        pytest.skip("the host was held up and the stream ran dry: nothing to tell")


def _calls():
    """(name, operands made on the current stream, the call)."""
    w = lambda: mx.quantize(_normal(512, 1024, 1, torch.float32), "fp4")   # noqa: E731
    x8 = lambda: mx.quantize(_normal(600, 1024, 2), "fp8")                  # noqa: E731
    dy = lambda: _normal(600, 512, 3)                                       # noqa: E731
    kept = lambda: mx.act_forward("swiglu", _normal(600, 512, 4), _normal(600, 512, 5))[1]   # noqa: E731
    return [("quantize", [lambda: _normal(600, 1024, 2)], lambda a, **k: mx.quantize(a, "fp8", **k)),
            ("dequantize", [x8], lambda a, **k: mx.dequantize(a, **k)),
            ("linear", [x8, w], lambda a, b, **k: mx.linear(a, b, **k)),
            ("linear from bf16", [lambda: _normal(600, 1024, 2), w], lambda a, b, **k: mx.linear(a, b, **k)),
            ("dgrad", [dy, w], lambda a, b, **k: mx.linear_dgrad(a, b, **k)),
            ("wgrad", [dy, x8], lambda a, b, **k: mx.linear_wgrad(a, b, **k)),
            ("act_forward", [lambda: _normal(600, 512, 4), lambda: _normal(600, 512, 5)],
             lambda a, b, **k: mx.act_forward("swiglu", a, b, **k)),
            ("act_backward", [lambda: list(kept()), dy], lambda a, b, **k: mx.act_backward("swiglu", a, b, **k))]


def _flat(v):
    return [u for t in v for u in _flat(t)] if isinstance(v, (tuple, list)) else [v]


def _values(v):
    return [(t.codes.clone(), t.scales.clone()) if isinstance(t, mx.MXMatrix) else (t.clone(),) for t in _flat(v)]


def _equal(a, b):
    return all(torch.equal(p, q) for s, t in zip(a, b) for p, q in zip(s, t))


@pytest.mark.parametrize("which", range(8))
def test_operands_may_be_dropped_at_once(which):
    name, make, call = _calls()[which]
    print(name, flush=True)
    want = _values(call(*[m() for m in make]))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    operands = [m() for m in make]
    spans = [_span(t) for t in _flat(operands)]
    forms = [(True, t.rows, t.cols, t.format) if isinstance(t, mx.MXMatrix) else (False, t.numel() * t.element_size() // 4)
             for t in _flat(operands)]
    side.wait_stream(torch.cuda.current_stream())
    _keep_busy(side)
    got = call(*operands, stream=side)
    del operands
    # the same sizes on the current stream; nothing here waits for the GPU, whose
    # streams may share a hardware queue
    fresh = [mx.MXMatrix(*f[1:]) if f[0] else torch.empty(*f[1:], device=DEV) for f in forms]
    _still_busy(side)
    assert all(_apart(_span(t), s) for t in fresh for s in spans)
    for t in fresh:
        (t.codes if isinstance(t, mx.MXMatrix) else t.view(torch.uint8)).zero_()
    side.synchronize()
    assert _equal(_values(got), want)


@pytest.mark.parametrize("which", range(8))
def test_results_may_be_dropped_once_their_use_is_queued(which):
    name, make, call = _calls()[which]
    print(name, flush=True)
    operands = [m() for m in make]
    want = _values(call(*operands))
    torch.cuda.synchronize()
    side, main = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(main):
        side.wait_stream(main)
        got = call(*operands, stream=side)
        main.wait_stream(side)
        spans = [_span(t) for t in _flat(got)]
        torch.cuda._sleep(BUSY)
        used = _values(got)                      # queued behind the wait
        del got
        again = call(*operands, stream=side)
        _still_busy(main)
        assert all(_apart(_span(t), s) for t in _flat(again) for s in spans)
    torch.cuda.synchronize()
    assert _equal(used, want) and _equal(_values(again), want)


def test_a_side_stream_with_temporaries_in_a_graph():
    x, m = _normal(70, 640, 6), _normal(300, 640, 7, torch.float32)
    side, main = torch.cuda.Stream(), torch.cuda.Stream()
    main.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    mx.linear(mx.quantize(x, "fp8"), mx.quantize(m, "fp4"))
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=main):
        xq, w = mx.quantize(x, "fp8"), mx.quantize(m, "fp4")
        side.wait_stream(main)
        y = mx.linear(xq, w, stream=side)
        del xq, w
        # more temporaries of those sizes while the side stream still reads the first
        z = mx.linear(mx.quantize(x * 2, "fp8"), mx.quantize(m * 2, "fp4"))
        main.wait_stream(side)
    for seed in (8, 9, 10):
        x.copy_(_normal(70, 640, seed))
        graph.replay()
        torch.cuda.synchronize()
        xq, w = mx.quantize(x, "fp8"), mx.quantize(m, "fp4")
        assert torch.equal(y, mx.linear(xq, w)), seed
        assert torch.equal(z, mx.linear(mx.quantize(x * 2, "fp8"), mx.quantize(m * 2, "fp4"))), seed
        torch.cuda.synchronize()


def test_recording_empty_and_given_matrices():
    side = torch.cuda.Stream()
    mx.MXMatrix(0, 64, "fp8").record_stream(side)
    m = mx.quantize(_normal(5, 64, 11), "fp4")
    mx.MXMatrix(5, 64, "fp4", codes=m.codes, scales=m.scales).record_stream(side)
    m.record_stream(side)
    assert mx.linear(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), m, stream=side).shape == (0, 5)


def test_a_stream_of_another_device_is_refused():
    class Other:
        device = torch.device("cuda", torch.cuda.current_device() + 1)

    x = _normal(5, 64, 12)
    m = mx.quantize(x, "fp4")
    for call in (lambda s: mx.quantize(x, "fp8", stream=s), lambda s: mx.dequantize(m, stream=s),
                 lambda s: mx.linear(x, m, stream=s), lambda s: mx.act_forward("gelu", x, stream=s)):
        with pytest.raises(ValueError, match="the stream is on"):
            call(Other())
