"""Forms of embedding, head norms and dropout that test_layers_gpu.py's sizes do
not reach, with its tolerances."""
import pytest
import torch

from bit_adamw_update_amd import layers
from test_layers_gpu import DEV, _check_back, _heads_case, _laid

pytestmark = pytest.mark.gpu


# ---- head norms -----------------------------------------------------------------

@pytest.mark.parametrize("layout,batch", [("split", None), ("by head", 3), ("gaps", 3)])
def test_gradients_in_the_place_of_the_inputs(layout, batch):
    tokens = 601   # several rows to a lane
    q, k, gq, gk, pos, f, how = case = _heads_case(tokens, 4, 2, 64, 64, False, layout, 300, batch=batch)
    dq, dk = _laid(tokens, 4, 64, "split", 301, batch), _laid(tokens, 2, 64, layout, 302, batch)
    want = _check_back(*case, dq, dk)
    got = layers.head_norm_rope_backward(q, k, gq.to(DEV), gk.to(DEV), pos.to(DEV), f, dq, dk, out=(q, k), **how)
    assert got[0] is q and got[1] is k
    assert all(torch.equal(a, b) for a, b in zip(want, got))
