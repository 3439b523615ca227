"""Bounds of the microscaled products' sizes: refused before any device work."""
import pytest

from bit_adamw_update_amd import api

SHAPE = 2
P = 0x10000000   # a plausible aligned address: refused before it is used
WIDE = 1 << 23


def M(rows, cols, fmt=api.MX_FP8):
    return api.Q4MXMatrix(fmt, 0, rows, cols, P, 2 * P)


def W(rows, cols):
    return M(rows, cols, api.MX_FP4)


def refused(text, fn, *args):
    with pytest.raises(api.Q4Error) as e:
        fn(*args)
    assert e.value.status == SHAPE and text in str(e.value), str(e.value)


def test_widths_of_products():
    lin = lambda x, w: api.q4mx_linear(x, w, P, api.MX_BF16, 64, P, 1 << 50, 0)  # noqa: E731
    refused("2^23", lin, M(40, WIDE), W(64, WIDE))
    b = lambda ld, t, w: api.q4mx_linear_bf16(P, ld, t, w, P, api.MX_BF16, 64, P, 1 << 50, 0)  # noqa: E731
    refused("2^23", b, WIDE, 40, W(64, WIDE))
    refused("2^23", b, WIDE, 40, W(64, 128))
    d = lambda ld, t, w: api.q4mx_dgrad(P, ld, t, w, P, api.MX_BF16, WIDE + 1, P, 1 << 50, 0)  # noqa: E731
    refused("2^23", d, 64, 40, W(64, WIDE))
    refused("2^23", d, WIDE, 40, W(64, 128))
    g = lambda ld, n, x: api.q4mx_wgrad(P, ld, n, x, P, api.MX_BF16, WIDE + 1, 0, P, 1 << 50, 0)  # noqa: E731
    refused("2^23", g, 64, 64, M(40, WIDE))
    refused("2^23", g, WIDE, 64, M(40, 128))


def test_sizes_of_results():
    lin = lambda t, o: api.q4mx_linear(M(t, 128), W(o, 128), P, api.MX_BF16, o, P, 1 << 50, 0)  # noqa: E731
    refused("2^38", lin, 1 << 19, 1 << 19)
    refused("2^38", lin, 1 << 12, 1 << 26)
    b = lambda t, o: api.q4mx_linear_bf16(P, 128, t, W(o, 128), P, api.MX_BF16, o, P, 1 << 50, 0)  # noqa: E731
    refused("2^38", b, 1 << 19, 1 << 19)
    d = lambda t, i: api.q4mx_dgrad(P, 64, t, W(64, i), P, api.MX_BF16, i, P, 1 << 50, 0)  # noqa: E731
    refused("2^38", d, 1 << 16, 1 << 22)
    refused("2^38", d, (1 << 31) - 1, 129)
    g = lambda n, i: api.q4mx_wgrad(P, n, n, M(40, i), P, api.MX_BF16, i, 0, P, 1 << 50, 0)  # noqa: E731
    refused("2^38", g, 1 << 19, 1 << 19)


def test_sizes_just_inside_ask_for_a_workspace():
    """One below the bounds passes them: what is missing is the workspace or its size."""
    big = api.q4mx_dgrad_workspace_bytes(P + 2, 1, (1 << 27) + 5, W(1, 1))
    assert big >= ((1 << 27) + 5) * 16
    with pytest.raises(api.Q4Error) as e:
        api.q4mx_dgrad(P + 2, 1, (1 << 27) + 5, W(1, 1), P, api.MX_BF16, 1, P, big - 1, 0)
    assert e.value.status == 7
