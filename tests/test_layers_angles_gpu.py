"""Angles of every 64-bit position: the head norms' rotation, forward and
backward, against the plain 64-bit implementations.  The tolerances are those
of near positions (layers_reference.py): an angle is one FP64 product on either
side, and its cosine and sine come from a remainder that is exact beyond FP32."""
import math

import pytest
import torch

import layers_reference as ref
from bit_adamw_update_amd import layers
from test_layers_gpu import DEV, F32, _check_back, _check_heads, _laid, _normal

pytestmark = pytest.mark.gpu

FAR = [0, -1, (1 << 40) - 1, 1 << 40, -(1 << 46) - 3, (1 << 51) + 1, (1 << 52) + 1, -(1 << 53) + 1, (1 << 56) + 12345,
       -(1 << 58) - 777, (1 << 60) + (1 << 20), (1 << 62) + (1 << 40), (1 << 63) - 1, -(1 << 63)]


def _case(frequencies, inter, seed):
    t = len(FAR)
    gains = (1 + 0.5 * _normal(64, seed=seed, dtype=F32), 1 + 0.5 * _normal(64, seed=seed + 1, dtype=F32))
    return (_laid(t, 3, 64, "split", seed + 2), _laid(t, 2, 64, "by head", seed + 3), *gains, torch.tensor(FAR),
            frequencies.to(DEV), {"eps": 1e-6, "interleaved": inter})


@pytest.mark.parametrize("inter", [False, True])
def test_every_position_turns_as_its_angle_says(inter):
    # frequencies of a rotation, and large ones: angles of up to 2^71.97
    large = torch.tensor([500.0, 3.25, 1.0, 0.1] + [1e-3] * 20, dtype=torch.float64)
    for f in (layers.rope_frequencies(64, device="cpu"), large):
        angle = ref.angles(torch.tensor(FAR), f)
        assert math.isclose(float(torch.cos(angle)[-1, 0]), math.cos(float(angle[-1, 0])), abs_tol=1e-15)
        case = _case(f, inter, 200)
        _check_heads(*case)
        t = len(FAR)
        _check_back(*case, _laid(t, 3, 64, "split", 210), _laid(t, 2, 64, "split", 211), dtype=F32)


@pytest.mark.parametrize("inter", [False, True])
def test_angles_out_of_range_are_not_a_number(inter):
    f = torch.tensor([math.inf, 1.0, 1024.0, 0.5], dtype=torch.float64)
    q, k, gq, gk, pos, f, how = _case(f, inter, 220)
    y, _ = layers.head_norm_rope(q, k, gq.to(DEV), gk.to(DEV), pos.to(DEV), f, **how)
    a, b = ref.pairs(64, 8, inter)
    nan = ~(ref.angles(pos, f).abs() < 2.0 ** 72)   # infinite ones (0 * inf is none), and those of the largest positions
    assert nan.sum(0).tolist() == [len(FAR), 0, 3, 0]
    for at in (a, b):
        same = torch.isnan(y[..., at]).cpu() == nan[:, None]
        assert bool(same.all())
    rest = [i for i in range(64) if i not in a.tolist() + b.tolist()]
    assert bool(torch.isfinite(y[..., rest]).all())
