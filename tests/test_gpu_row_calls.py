"""Calls of the row passes that a user may make by mistake or at the edge of
what is allowed, through the public entry points."""
import pytest
import torch

from input_adaptive_block_b200 import api

pytestmark = pytest.mark.gpu


def test_one_tensor_as_gradient_of_q_and_as_k():
    rope = api.rope_axes(64, (8, 12, 12))
    few, many = (torch.zeros(6, h, 64, dtype=torch.bfloat16, device="cuda") for h in (2, 5))
    for a, b in ((few, many), (many, few)):
        with pytest.raises(ValueError):
            api.qk_norm_rope_backward(a, b, a, a, rope, grid=(1, 2, 3), norm="head")


def test_modulation_per_row_of_no_rows():
    x = torch.empty(0, 64, device="cuda")
    m = torch.empty(0, 3, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    p = dict(gate=m[:, 0], scale=m[:, 1], shift=m[:, 2], weight=w)
    a, b = api.gate_residual_norm(x, x, **p)
    assert a.shape == b.shape == (0, 64)
    g = api.gate_residual_norm_backward(x, x, x, x, **p)
    assert g.x.shape == g.y.shape == g.gate.shape == g.scale.shape == g.shift.shape == (0, 64) and not g.weight.any()
    with pytest.raises(ValueError):
        api.norm_modulate(torch.empty(5, 64, device="cuda"), scale=m[:, 1])
