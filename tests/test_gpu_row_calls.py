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


@pytest.mark.parametrize("dim", [777, 1536, 5120, 8200, 16384])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("post", ["none", "rms"])
def test_results_over_inputs(dim, dtype, post):
    """Every place that the header allows a result in, the same bits as in a
    tensor of its own."""
    gen = torch.Generator(device="cuda").manual_seed(dim)
    x, y, a, b = (torch.randn(700, dim, generator=gen, device="cuda").to(dtype) for _ in range(4))
    p = {n: torch.randn(7, dim, generator=gen, device="cuda") * 0.3 for n in ("gate", "scale", "shift")}
    res = dict(gate=p["gate"], post_norm=post)
    pre = dict(scale=p["scale"], shift=p["shift"])

    def same(want, got):
        assert torch.equal(want, got)

    want = api.norm_modulate(x, **pre)
    t = x.clone()
    same(want, api.norm_modulate(t, **pre, out=t))
    want = api.gate_residual(x, y, **res)
    for i in (0, 1):
        t = [x.clone(), y.clone()]
        same(want, api.gate_residual(*t, **res, out=t[i]))
    want = api.norm_modulate_backward(b, x, **pre, dres=a)
    t = a.clone()
    got = api.norm_modulate_backward(b, x, **pre, dres=t, dx=t)
    same(want.x, t)
    same(want.scale, got.scale)
    want = api.gate_residual_backward(a, y, **res)
    t = y.clone()
    got = api.gate_residual_backward(a, t, **res, dy=t)
    same(want.y, t)
    same(want.gate, got.gate)
    want = api.gate_residual_norm_backward(a, b, x, y, **res, **pre)
    for i in (0, 1):
        d, t = a.clone(), [b.clone(), y.clone()]
        got = api.gate_residual_norm_backward(d, t[0], x, t[1], **res, **pre, dx=d, dy=t[i])
        same(want.x, d)
        same(want.y, t[i])
        for n in p:
            same(getattr(want, n), getattr(got, n))


@pytest.mark.parametrize("style", ["interleaved", "half"])
def test_bad_values_stay_in_their_pair(style):
    """Without a norm an infinity or NaN reaches its pair's two channels, also
    where the pair does not turn, and nothing else."""
    rope = api.rope_axes(64, (8, 12, 12), style=style)
    x = torch.randn(12, 2, 64, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    kw = dict(grid=(1, 2, 4), text_tokens=4)
    want = api.qk_norm_rope(x, None, rope, **kw)[0]
    assert torch.equal(want[8:], x[8:])
    for bad in (float("inf"), float("nan")):
        y = x.clone()
        y[3, 1, 9] = y[10, 0, 9] = bad
        got = api.qk_norm_rope(y, None, rope, **kw)[0]
        free = torch.ones_like(x, dtype=torch.bool)
        for c in (8, 9) if style == "interleaved" else (9, 9 + 32):
            free[3, 1, c] = free[10, 0, c] = False
        assert torch.equal(got[free], want[free])
        assert not got[10, 0, 9].isfinite()
