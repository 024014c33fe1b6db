"""Row passes around the attention on a machine without a GPU: the float64
definitions against differences, the rotation ladders, and every refusal of
the C ABI (with pointers that are never dereferenced: validation fails
first)."""
import ctypes

import numpy as np
import pytest
import torch

from input_adaptive_block_b200 import _lib, api
from input_adaptive_block_b200._lib import (SPADE_ERR_INVALID, SPADE_ERR_UNSUPPORTED, SPADE_ERR_WORKSPACE, SPADE_OK,
                                            SpadeQkDesc, SpadeRope, SpadeRowDesc, SpadeRowGrads, SpadeRowParams)
from oracle import row_oracle as R

BASE = 1 << 40


# ------------------------------------------- definitions, by differences --
def _slope(f, x, d, h=1e-5):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("style", ["interleaved", "half"])
@pytest.mark.parametrize("norm", ["none", "token", "head"])
def test_qk_gradient_is_the_slope(norm, style):
    rng = np.random.default_rng(5)
    rows, heads, d = 7, 3, 10
    axis, freq = R.rope_ladder((2, 1, 2), (10.0, 20.0, 30.0))
    cos, sin = R.rope_angles(R.grid_positions(rows, 2, 3, 2, 2), axis, freq, d, text_tokens=2)
    x, g = rng.normal(size=(rows, heads, d)), rng.normal(size=(rows, heads, d))
    w = None if norm == "none" else rng.normal(size=(heads if norm == "token" else 1, d))
    f = lambda x, w: (g * R.qk_norm_rope(x, w, cos, sin, norm, 1e-6, style)).sum()  # noqa: E731
    dx, dw = R.qk_norm_rope_backward(g, x, w, cos, sin, norm, 1e-6, style)
    t = rng.normal(size=x.shape)
    assert abs(_slope(lambda v: f(v, w), x, t) - (dx * t).sum()) < 1e-7 * (1 + np.abs(dx * t).sum())
    if norm != "none":
        t = rng.normal(size=w.shape)
        assert abs(_slope(lambda v: f(x, v), w, t) - (dw * t).sum()) < 1e-7 * (1 + np.abs(dw * t).sum())


PARAMS = ("gate", "post_weight", "weight", "bias", "scale", "shift")


@pytest.mark.parametrize("groups", [1, 3, 6])
@pytest.mark.parametrize("half", ["norm", "gate", "both"])
@pytest.mark.parametrize("norm,post", [("rms", "layer"), ("layer", "rms"), ("layer", "none")])
def test_row_gradient_is_the_slope(norm, post, half, groups):
    rng = np.random.default_rng(6)
    rows, dim = 6, 9
    v = {"x": rng.normal(size=(rows, dim)) + 1.0, "y": rng.normal(size=(rows, dim)) if half != "norm" else None}
    used = [n for n in PARAMS if (half == "both" or (n in ("gate", "post_weight")) == (half == "gate"))]
    if post == "none" and "post_weight" in used:
        used.remove("post_weight")
    for n in PARAMS:
        v[n] = rng.normal(size=(groups if n in ("gate", "scale", "shift") else 1, dim)) if n in used else None
    gx, gh = rng.normal(size=(rows, dim)), rng.normal(size=(rows, dim))
    kind = None if half == "gate" else norm

    def f(v):
        x, h = R.gate_residual_norm(v["x"], v["y"], v, kind, 1e-6, post, 1e-5, 0.7)
        return (gx * x).sum() + (0.0 if h is None else (gh * h).sum())

    grads = R.gate_residual_norm_backward(gx, gh, v["x"], v["y"], v, kind, 1e-6, post, 1e-5, 0.7, groups)
    for n in (["x"] if half != "gate" else []) + (["y"] if half != "norm" else []) + used:
        t = rng.normal(size=v[n].shape)
        want = (grads[n] * t).sum()
        got = _slope(lambda a: f({**v, n: a}), v[n], t)
        assert abs(got - want) < 1e-6 * (1 + np.abs(grads[n] * t).sum()), n


def test_rope_ladders():
    for pairs, theta, scale, shared in (((22, 21, 21), (1e4,) * 3, (1.0,) * 3, False),
                                        ((8, 28, 28), (256.0,) * 3, (1.0, 0.5, 2.0), False),
                                        ((3, 0, 5), (10.0, 1.0, 1e6), (1.0,) * 3, False),
                                        ((4, 4, 4), (1e4,) * 3, (1.0,) * 3, True), ((0, 0, 0), (1e4,) * 3, (1.0,) * 3, True)):
        rope = api.rope_axes(128, pairs, theta, scale, "half", shared)
        axis, freq = R.rope_ladder(pairs, theta, scale, shared)
        assert (rope.pairs, rope.style) == (sum(pairs), 1)
        assert list(rope.axis[: rope.pairs]) == axis.tolist()
        np.testing.assert_allclose(list(rope.freq[: rope.pairs]), freq, rtol=1e-14)
    with pytest.raises(ValueError):
        api.rope_axes(128, (64, 1, 0))
    with pytest.raises(ValueError):
        api.rope_axes(128, (64, 0))
    for bad in ({"theta": 0.0}, {"theta": float("nan")}, {"scale": float("inf")}, {"pairs": (-1, 1, 1)}):
        with pytest.raises(_lib.SpadeError):
            api.rope_axes(128, **{"pairs": (1, 1, 1), **bad})
    with pytest.raises(ValueError):
        api.rope_axes(128, (1, 1, 1), style="neox")


# ----------------------------------------------------------- Q/K refusals --
def _rope(pairs=64, style=0):
    r = SpadeRope(pairs=pairs, style=style)
    for i in range(pairs):
        r.axis[i], r.freq[i] = i % 3, 0.1
    return r


def _qk(rope=None, positions=None, q=BASE, k=2 * BASE, qw=None, kw=None, qo=3 * BASE, ko=4 * BASE, bwd=None, ws=None,
        ws_bytes=0, dqw=None, dkw=None, **over):
    desc = SpadeQkDesc(rows=1000, T=10, H=10, W=10, q_heads=4, k_heads=2, d=128, dt=1, weight_dt=0, norm=1, eps=1e-6)
    for n, v in over.items():
        setattr(desc, n, v)
    rope = _rope() if rope is None else rope
    lib = _lib.load()
    if bwd is None:
        return lib.spade_qk_norm_rope(ctypes.byref(desc), ctypes.byref(rope), positions, q, k, qw, kw, qo, ko, None)
    return lib.spade_qk_norm_rope_bwd(ctypes.byref(desc), ctypes.byref(rope), positions, bwd[0], bwd[1], q, k, qw, kw,
                                      qo, ko, dqw, dkw, ws, ws_bytes, None)


BIG = 1 << 33


@pytest.mark.parametrize("want,kw", [
    (SPADE_ERR_INVALID, {"rows": -1}), (SPADE_ERR_INVALID, {"text_tokens": 1001}), (SPADE_ERR_INVALID, {"text_tokens": -1}),
    (SPADE_ERR_INVALID, {"rows": 1001}), (SPADE_ERR_INVALID, {"token_offset": 1}), (SPADE_ERR_INVALID, {"token_offset": -1}),
    (SPADE_ERR_INVALID, {"H": 0}), (SPADE_ERR_UNSUPPORTED, {"T": 1 << 20, "H": 1 << 20, "W": 1 << 20}),
    (SPADE_ERR_INVALID, {"q_heads": 0, "k_heads": 0}), (SPADE_ERR_INVALID, {"q_heads": -1}),
    (SPADE_ERR_UNSUPPORTED, {"k_heads": 129}), (SPADE_ERR_UNSUPPORTED, {"d": 127}), (SPADE_ERR_UNSUPPORTED, {"d": 258}),
    (SPADE_ERR_UNSUPPORTED, {"d": 0}), (SPADE_ERR_INVALID, {"d": 64}), (SPADE_ERR_INVALID, {"dt": 2}),
    (SPADE_ERR_INVALID, {"weight_dt": -1}), (SPADE_ERR_INVALID, {"norm": 3}), (SPADE_ERR_INVALID, {"eps": -1.0}),
    (SPADE_ERR_INVALID, {"eps": float("nan")}), (SPADE_ERR_INVALID, {"eps": float("inf")}),
    (SPADE_ERR_INVALID, {"q_stride": 511}), (SPADE_ERR_INVALID, {"k_out_stride": -256}),
    (SPADE_ERR_INVALID, {"q_stride": 1 << 60}),
    (SPADE_ERR_INVALID, {"q": None}), (SPADE_ERR_INVALID, {"ko": None}), (SPADE_ERR_INVALID, {"q": BASE + 1}),
    (SPADE_ERR_INVALID, {"qw": BIG + 2}), (SPADE_ERR_INVALID, {"qw": BIG, "norm": 0}),
    (SPADE_ERR_INVALID, {"positions": BIG, "text_tokens": 5}), (SPADE_ERR_INVALID, {"positions": BIG + 2}),
    (SPADE_ERR_INVALID, {"ko": 3 * BASE}), (SPADE_ERR_INVALID, {"qo": BASE + 1024}), (SPADE_ERR_INVALID, {"qo": 2 * BASE}),
    (SPADE_ERR_INVALID, {"qo": BASE, "q_out_stride": 1024}), (SPADE_ERR_INVALID, {"qw": 3 * BASE}),
    (SPADE_ERR_INVALID, {"positions": 4 * BASE + 8}),
    (SPADE_ERR_INVALID, {"qw": 3 * BASE, "weight_dt": 1, "rows": 1}),       # written over its own weights
], ids=lambda v: str(v))
def test_qk_refusals(want, kw):
    assert _qk(**kw) == want
    assert _lib.load().spade_last_error_message()


def test_qk_refuses_bad_rotations():
    r = _rope()
    r.axis[3] = 3
    assert _qk(rope=r) == SPADE_ERR_INVALID
    r = _rope()
    r.freq[0] = float("inf")
    assert _qk(rope=r) == SPADE_ERR_INVALID
    assert _qk(rope=_rope(65)) == SPADE_ERR_INVALID
    assert _qk(rope=_rope(-1)) == SPADE_ERR_INVALID
    assert _qk(rope=_rope(64, style=2)) == SPADE_ERR_INVALID
    assert _qk(rope=_rope(63, style=1)) == SPADE_ERR_UNSUPPORTED
    lib = _lib.load()
    assert lib.spade_qk_norm_rope(None, ctypes.byref(_rope()), *[None] * 8) == SPADE_ERR_INVALID
    assert lib.spade_qk_norm_rope(ctypes.byref(SpadeQkDesc()), None, *[None] * 8) == SPADE_ERR_INVALID


def test_qk_backward_refusals():
    g = (5 * BASE, 6 * BASE)
    assert _qk(bwd=(None, 6 * BASE)) == SPADE_ERR_INVALID
    assert _qk(bwd=g, q=None) == SPADE_ERR_INVALID                       # the norm needs its input
    assert _qk(bwd=g, dqw=BIG) == SPADE_ERR_WORKSPACE
    assert _qk(bwd=g, dqw=BIG, ws=7 * BASE, ws_bytes=64) == SPADE_ERR_WORKSPACE
    assert _qk(bwd=g, dqw=BIG, ws=7 * BASE + 8, ws_bytes=BIG) == SPADE_ERR_INVALID
    assert _qk(bwd=g, dqw=BIG, ws=BASE, ws_bytes=BIG) == SPADE_ERR_INVALID   # scratch over q
    assert _qk(bwd=g, dqw=BIG, norm=0) == SPADE_ERR_INVALID
    assert _qk(bwd=g, dqw=BIG, qw=BIG, ws=7 * BASE, ws_bytes=BIG) == SPADE_ERR_INVALID   # gradient over its weight
    assert _qk(bwd=g, dkw=BIG, k=None, ko=None, k_heads=0, ws=7 * BASE, ws_bytes=BIG) == SPADE_ERR_INVALID
    assert _qk(bwd=g, q_dout_stride=100) == SPADE_ERR_INVALID


def test_qk_workspace():
    assert api.qk_norm_rope_workspace_bytes(0, 4, 4, 128, "token") == 0
    assert api.qk_norm_rope_workspace_bytes(1000, 4, 4, 128, "none") == 0
    assert api.qk_norm_rope_workspace_bytes(1000, 4, 2, 128, "token") % (6 * 128 * 4) == 0
    assert api.qk_norm_rope_workspace_bytes(1000, 4, 2, 128, "token") > 0
    assert api.qk_norm_rope_workspace_bytes(1000, 4, 200, 128, "head") == 0
    with pytest.raises(ValueError):
        api.qk_norm_rope_workspace_bytes(1000, 4, 2, 128, "layer")


# ----------------------------------------------------------- row refusals --
def _row(call="norm_modulate", p=None, g=None, ptrs=None, ws=9 * BASE, ws_bytes=BIG, **over):
    desc = SpadeRowDesc(rows=600, groups=6, dim=256, x_dt=0, branch_dt=1, param_dt=0, norm=2, post_norm=0, eps=1e-6,
                        post_eps=1e-6, residual_scale=1.0)
    for n, v in over.items():
        setattr(desc, n, v)
    params, grads = SpadeRowParams(**(p or {})), SpadeRowGrads(**(g or {}))
    names = {"norm_modulate": "xh", "gate_residual": "xyX", "gate_residual_norm": "xyXh", "norm_modulate_bwd": "Hrxd",
             "gate_residual_bwd": "Gye", "gate_residual_norm_bwd": "GHxyde"}[call]
    at = {n: (i + 1) * BASE for i, n in enumerate("xyXhHGde")}
    at["r"] = None
    at.update(ptrs or {})
    args = [ctypes.byref(desc), ctypes.byref(params)] + [at[n] for n in names]
    if call.endswith("bwd"):
        args += [ctypes.byref(grads), ws, ws_bytes]
    return getattr(_lib.load(), "spade_" + call)(*args, None)


W = 50 * BASE


@pytest.mark.parametrize("call", ["norm_modulate", "gate_residual", "gate_residual_norm", "norm_modulate_bwd",
                                  "gate_residual_bwd", "gate_residual_norm_bwd"])
def test_row_refusals_of_every_call(call):
    for want, kw in ((SPADE_ERR_INVALID, {"rows": -6}), (SPADE_ERR_INVALID, {"groups": 0}),
                     (SPADE_ERR_INVALID, {"groups": 7}), (SPADE_ERR_INVALID, {"dim": 0}),
                     (SPADE_ERR_UNSUPPORTED, {"dim": 16385}), (SPADE_ERR_INVALID, {"x_dt": 5}),
                     (SPADE_ERR_INVALID, {"param_dt": 5}), (SPADE_ERR_UNSUPPORTED, {"x_dt": 1, "branch_dt": 0}),
                     (SPADE_ERR_INVALID, {"norm": 3}), (SPADE_ERR_INVALID, {"post_norm": -1}),
                     (SPADE_ERR_INVALID, {"x_stride": 255}), (SPADE_ERR_INVALID, {"gate_stride": 1})):
        assert _row(call, **kw) == want, kw
        assert _lib.load().spade_last_error_message()
    for n in {"norm_modulate": "xh", "gate_residual": "xyX", "gate_residual_norm": "xyXh", "norm_modulate_bwd": "Hxd",
              "gate_residual_bwd": "Gye", "gate_residual_norm_bwd": "Hxyde"}[call]:
        assert _row(call, ptrs={n: None}) == SPADE_ERR_INVALID, n
        assert _row(call, ptrs={n: 20 * BASE + 1}) == SPADE_ERR_INVALID, n


def test_row_refusals():
    both = "gate_residual_norm"
    assert _row(norm=0) == SPADE_ERR_INVALID
    assert _row(eps=-1.0) == SPADE_ERR_INVALID
    assert _row(p={"gate": W}) == SPADE_ERR_INVALID
    assert _row(p={"weight": W + 2}) == SPADE_ERR_INVALID
    assert _row("gate_residual", p={"scale": W}) == SPADE_ERR_INVALID
    assert _row("gate_residual", p={"post_weight": W}) == SPADE_ERR_INVALID       # no post_norm
    assert _row(both, post_norm=1, post_eps=float("nan")) == SPADE_ERR_INVALID
    # overlaps: outputs with one another, with inputs not exactly theirs, with parameters
    assert _row(both, ptrs={"X": 4 * BASE}) == SPADE_ERR_INVALID
    assert _row(both, ptrs={"X": BASE + 1024}) == SPADE_ERR_INVALID
    assert _row(both, ptrs={"X": BASE}, x_out_stride=512) == SPADE_ERR_INVALID
    assert _row(both, ptrs={"h": BASE}) == SPADE_ERR_INVALID                       # other type than x
    assert _row(both, p={"scale": 4 * BASE + 64}) == SPADE_ERR_INVALID
    bwd = "gate_residual_norm_bwd"
    assert _row(bwd, g={"gate": W}, ws_bytes=16) == SPADE_ERR_WORKSPACE
    assert _row(bwd, g={"gate": W}, ws=None) == SPADE_ERR_WORKSPACE
    assert _row(bwd, g={"gate": W}, ws=9 * BASE + 4) == SPADE_ERR_INVALID
    assert _row(bwd, g={"gate": W}, ws=BASE) == SPADE_ERR_INVALID
    assert _row(bwd, g={"gate": W + 2}) == SPADE_ERR_INVALID
    assert _row(bwd, p={"gate": W}, g={"gate": W}) == SPADE_ERR_INVALID            # a gradient over its parameter
    assert _row(bwd, branch_dt=0, ptrs={"d": 2 * BASE}) == SPADE_ERR_INVALID       # dx over y, which is read later
    assert _row(bwd, g={"gate": W, "shift": W + 1024}) == SPADE_ERR_INVALID
    assert _row(bwd, g={"post_weight": W}) == SPADE_ERR_INVALID
    assert _row("norm_modulate_bwd", g={"gate": W}) == SPADE_ERR_INVALID
    assert _row("gate_residual_bwd", g={"weight": W}) == SPADE_ERR_INVALID
    assert _row(bwd, dy_stride=17) == SPADE_ERR_INVALID


def test_row_workspace():
    assert api.row_workspace_bytes(0, 256) == 0
    assert api.row_workspace_bytes(600, 256, 7) == 0
    assert api.row_workspace_bytes(600, 256, 6) > 0
    assert api.row_workspace_bytes(600, 20000) == 0


def test_no_rows_is_no_call():
    """No rows: nothing is launched, and operands may be null."""
    assert _row(rows=0, ptrs={"x": None, "h": None}) == SPADE_OK
    assert _qk(rows=0, q=None, k=None, qo=None, ko=None) == SPADE_OK


def test_host_tensors_are_refused():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        api.norm_modulate(x)
    with pytest.raises(ValueError):
        api.gate_residual(x, x)
    with pytest.raises(ValueError):
        api.qk_norm_rope(x.view(4, 1, 64), None, api.rope_axes(64, (8, 12, 12)), grid=(1, 2, 2))
