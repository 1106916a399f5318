"""moe_block_norm's sigmoid to the accuracy that its header states.  A residual of -1
times the sigmoid's fp32 value leaves what the kernel's differs from it."""
import numpy as np
import pytest
import torch

from gpu_util import load_binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    return load_binding()


def sigmoid64(g):
    return 1.0 / (1.0 + np.exp(-np.float64(g)))


@pytest.mark.parametrize("tokens,gate_rows", [(1, 1), (4, 4)])
def test_sigmoid(B, tokens, gate_rows):
    one = torch.ones(tokens, 64, dtype=torch.bfloat16, device="cuda")
    gates = torch.cat([torch.linspace(-87, 87, 120), torch.tensor([0.0, 1e-3, -1e-3, -0.5, 0.25])]).bfloat16()
    worst = 0.0
    for g in gates.tolist():
        want = sigmoid64(g)
        near = float(np.float32(want))
        out = B.block_norm(one, one, gate=torch.full((gate_rows, 64), g, device="cuda").bfloat16(),
                           gate_act="sigmoid", residual_scale=-near)
        left = out["residual_out"].double().cpu().numpy()      # the kernel's value less `near`, in bf16
        off = np.abs(left).max() * (1 + 2.0 ** -8) + abs(near - want)
        assert off <= want * (5e-7 + 1e-7 * abs(g)) + 2.0 ** -126, g
        worst = max(worst, off / want)
    assert worst > 1e-6         # more than a few units in the last place: the statement is not idle


def test_sigmoid_of_far_gates(B):
    one = torch.ones(3, 64, dtype=torch.bfloat16, device="cuda")
    for g, want in ((-100.0, 0.0), (-3e38, 0.0), (-float("inf"), 0.0), (100.0, 1.0), (float("inf"), 1.0)):
        out = B.block_norm(one, one, gate=torch.full((1, 64), g, device="cuda").bfloat16(), gate_act="sigmoid",
                           residual_scale=0.0)
        assert bool((out["residual_out"] == want).all()), g
    out = B.block_norm(one, one, gate=torch.full((1, 64), float("nan"), device="cuda").bfloat16(), gate_act="sigmoid")
    assert bool(torch.isnan(out["residual_out"]).all())
