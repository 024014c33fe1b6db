"""The row passes around the attention on the GPU: norm and several-axis
rotation of Q and K, the modulated norm, the gated residual update, and their
gradients, against the float64 definitions within the error that float32 sums
and one rounding of the result allow (bounded.py)."""
import numpy as np
import pytest
import torch

import oracle as O
from bounded import Bounded, check, turned
from input_adaptive_block_b200 import api
from oracle import row_oracle as R
from spade_workloads import Scheme, Workload, make_qkv

from helpers import ATTN_MEAN_ABS_BF16, run_grouped, to_np

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
GUARD = 512


def _b(t):
    return Bounded(t.detach().double().cpu().numpy())


class Rows:
    """[rows, *inner] inside a larger buffer of a fill value: rows `gap`
    elements apart, the first `off` elements in.  The buffer around the rows
    must stay as it was."""

    def __init__(self, rows, inner, dtype, gap=0, off=0, gen=None, mean=0.0, std=1.0):
        self.n = int(np.prod(inner))
        self.stride = self.n + gap
        self.buf = torch.full((GUARD + off + rows * self.stride + GUARD,), 7.0, dtype=dtype, device="cuda")
        body = self.buf[GUARD + off: GUARD + off + rows * self.stride].view(rows, self.stride)
        self.t = body[:, : self.n].view(rows, *inner)
        if gen is not None:
            self.t.copy_(torch.randn(self.t.shape, generator=gen, device="cuda") * std + mean)

    def intact(self):
        mask = torch.ones_like(self.buf, dtype=torch.bool)
        start = self.t.storage_offset()
        idx = (start + torch.arange(self.t.shape[0], device="cuda")[:, None] * self.stride +
               torch.arange(self.n, device="cuda")[None])
        mask[idx.flatten()] = False
        return bool((self.buf[mask] == 7.0).all())


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------------- Q/K --
def _qk(rows, qh=3, kh=3, d=128, pairs=(22, 21, 21), style="interleaved", norm="token", dtype=BF, wdt=F32, grid=None,
        offset=0, text=0, positions=None, gap=0, off=0, theta=1e4, weights=True, shared=False, eps=1e-6):
    return dict(locals())


QK = {
    "one_token": _qk(1, positions="far"),
    "wan": _qk(2 * 5 * 7, qh=12, kh=12, grid=(2, 5, 7)),
    "text_rows": _qk(3 * 4 * 5 + 11, qh=4, kh=4, pairs=(8, 28, 28), norm="head", theta=256.0, grid=(3, 4, 5), text=11),
    "all_text": _qk(9, grid=(1, 1, 1), text=9, norm="head"),
    "offset": _qk(31, grid=(3, 4, 5), offset=29, norm="none"),
    "shared_keys": _qk(333, qh=40, kh=8, norm="head", grid=(9, 6, 7)),
    "one_key_head": _qk(257, qh=48, kh=1, norm="token", grid=(9, 6, 7)),
    "half": _qk(100, qh=2, kh=5, d=64, pairs=(10, 11, 11), style="half", norm="token", grid=(4, 5, 5)),
    "half_80": _qk(99, qh=14, kh=2, d=80, pairs=(16, 12, 12), style="half", norm="head", dtype=F32, positions="far"),
    "odd_pairs": _qk(65, qh=5, kh=2, d=34, pairs=(7, 5, 5), norm="token", grid=(5, 13, 1)),
    "odd_half": _qk(65, qh=5, kh=2, d=38, pairs=(7, 6, 6), style="half", norm="head", grid=(5, 13, 1)),
    "two_channels": _qk(40, qh=33, kh=1, d=2, pairs=(0, 0, 1), norm="head", dtype=F32, grid=(1, 5, 8)),
    "few_pairs": _qk(50, qh=2, kh=2, d=128, pairs=(9, 3, 0), norm="token", positions="far"),
    "no_pairs": _qk(50, qh=2, kh=2, d=96, pairs=(0, 0, 0), norm="head", grid=(50, 1, 1)),
    "widest": _qk(6, qh=128, kh=128, d=256, pairs=(44, 42, 42), norm="token", grid=(1, 2, 3)),
    "widest_odd": _qk(6, qh=128, kh=100, d=254, pairs=(43, 42, 42), norm="head", dtype=F32, grid=(1, 2, 3)),
    "many_lanes": _qk(70, qh=45, kh=20, d=192, pairs=(32, 32, 32), style="half", norm="head", grid=(2, 5, 7)),
    "f32_token": _qk(300, qh=7, kh=3, d=160, pairs=(30, 25, 25), dtype=F32, norm="token", grid=(4, 9, 9)),
    "apart": _qk(77, qh=4, kh=2, norm="token", gap=24, off=8, grid=(7, 11, 1), wdt=BF),
    "unaligned": _qk(77, qh=4, kh=2, norm="token", gap=3, off=1, grid=(7, 11, 1), wdt=BF),
    "unaligned_f32": _qk(77, qh=4, kh=2, d=64, pairs=(8, 12, 12), style="half", norm="head", dtype=F32, gap=5, off=3,
                         grid=(7, 11, 1)),
    "only_q": _qk(60, kh=0, norm="head", grid=(3, 4, 5)),
    "only_k": _qk(60, qh=0, norm="token", grid=(3, 4, 5)),
    "no_weights": _qk(60, norm="head", grid=(3, 4, 5), weights=False),
    "one_ladder": _qk(60, norm="none", grid=(3, 4, 5), shared=True, theta=1e6),
    "zero_eps": _qk(60, qh=5, kh=3, norm="head", grid=(3, 4, 5), eps=0.0),
    "f32_interleaved": _qk(400, qh=8, kh=8, d=128, dtype=F32, norm="token", grid=(4, 10, 10)),
    "f32_halves": _qk(400, qh=6, kh=2, d=64, pairs=(12, 10, 10), style="half", dtype=F32, norm="head", grid=(4, 10, 10)),
    "many_tokens": _qk(3001, qh=12, kh=12, norm="token", grid=(5, 30, 30)),
    "many_rows": _qk(4321, qh=2, kh=1, d=64, pairs=(8, 12, 12), norm="head", grid=(5, 30, 30)),
}


class QkCase:
    def __init__(self, c, seed=3):
        gen = _gen(seed)
        self.c = c
        mk = lambda h, std: Rows(c["rows"], (h, c["d"]), c["dtype"], c["gap"], c["off"], gen, 0.1, std) if h else None  # noqa: E731
        self.q, self.k = mk(c["qh"], 1.0), mk(c["kh"], 2.0)
        self.dq, self.dk = mk(c["qh"], 1.0), mk(c["kh"], 1.0)
        wn = lambda h: h * c["d"] if c["norm"] == "token" else c["d"]  # noqa: E731
        w = lambda h: ((torch.randn(wn(h), generator=gen, device="cuda") * 0.3 + 1.0).to(c["wdt"])  # noqa: E731
                       if h and c["weights"] and c["norm"] != "none" else None)
        self.qw, self.kw = w(c["qh"]), w(c["kh"])
        self.rope = api.rope_axes(c["d"], c["pairs"], theta=c["theta"], style=c["style"], shared_ladder=c["shared"])
        axis, freq = R.rope_ladder(c["pairs"], (c["theta"],) * 3, shared=c["shared"])
        self.pos = None
        if c["positions"]:
            hi = torch.tensor([2000000000, 128, 128], device="cuda")
            u = torch.rand(c["rows"], 3, generator=gen, device="cuda", dtype=torch.float64) * 2 - 1
            self.pos = (u * hi).to(torch.int32)
            p = self.pos.cpu().numpy().astype(np.int64)
        else:
            p = R.grid_positions(c["rows"], c["offset"], *c["grid"])
        cos, sin = R.rope_angles(p, axis, freq, c["d"], c["text"])
        self.cos, self.sin = turned(cos, sin, p, freq)

    def where(self):
        c = self.c
        kw = {"norm": c["norm"], "eps": c["eps"], "q_weight": self.qw, "k_weight": self.kw}
        return {**kw, "positions": self.pos} if self.pos is not None else \
            {**kw, "grid": c["grid"], "token_offset": c["offset"], "text_tokens": c["text"]}

    def weight(self, w, h):
        if w is None:
            return Bounded(np.ones((1, 1)))
        return _b(w).reshape(h if self.c["norm"] == "token" else 1, self.c["d"])

    def forward(self, x, w):
        return R.qk_norm_rope(_b(x), self.weight(w, x.shape[1]), self.cos, self.sin, self.c["norm"], self.c["eps"],
                              self.c["style"])

    def backward(self, g, x, w):
        return R.qk_norm_rope_backward(_b(g), _b(x), self.weight(w, x.shape[1]), self.cos, self.sin, self.c["norm"],
                                       self.c["eps"], self.c["style"])


def _t(r):
    return None if r is None else r.t


@pytest.mark.parametrize("name", QK)
def test_qk_forward(name):
    s = QkCase(QK[name])
    outs = [None if r is None else Rows(r.t.shape[0], r.t.shape[1:], r.t.dtype, s.c["gap"], s.c["off"]) for r in (s.q, s.k)]
    got = api.qk_norm_rope(_t(s.q), _t(s.k), s.rope, **s.where(), q_out=_t(outs[0]), k_out=_t(outs[1]))
    for x, w, o, g, what in ((s.q, s.qw, outs[0], got[0], "q"), (s.k, s.kw, outs[1], got[1], "k")):
        if x is None:
            assert g is None
            continue
        assert g is o.t and o.intact() and x.intact(), what
        check(o.t, s.forward(x.t, w), what)
    # written over its own input, the same bits as the same call into another tensor
    if s.q is not None:
        alone = {**s.where(), "k_weight": None}
        want = api.qk_norm_rope(s.q.t, None, s.rope, **alone)[0]
        check(want, s.forward(s.q.t, s.qw), "q alone")
        api.qk_norm_rope(s.q.t, None, s.rope, **alone, q_out=s.q.t)
        same = torch.equal(s.q.t, want)
        assert same and s.q.intact()


@pytest.mark.parametrize("name", QK)
def test_qk_backward(name):
    s = QkCase(QK[name])
    outs = [None if r is None else Rows(r.t.shape[0], r.t.shape[1:], r.t.dtype, s.c["gap"], s.c["off"]) for r in (s.q, s.k)]
    need = api.qk_norm_rope_workspace_bytes(s.c["rows"], s.c["qh"], s.c["kh"], s.c["d"], s.c["norm"])
    ws = torch.full((max(need, 16) + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    args = (_t(s.dq), _t(s.dk), _t(s.q), _t(s.k), s.rope)
    g = api.qk_norm_rope_backward(*args, **s.where(), dq=_t(outs[0]), dk=_t(outs[1]), workspace=ws[: max(need, 16)])
    assert bool((ws[max(need, 16):] == 0xA5).all())
    for x, gr, w, o, dx, dw, what in ((s.q, s.dq, s.qw, outs[0], g.q, g.q_weight, "q"),
                                      (s.k, s.dk, s.kw, outs[1], g.k, g.k_weight, "k")):
        if x is None:
            assert dx is None and dw is None
            continue
        assert dx is o.t and o.intact() and x.intact() and gr.intact(), what
        ref, refw = s.backward(gr.t, x.t, w)
        check(dx, ref, what)
        if w is None:
            assert dw is None
        else:
            check(dw, refw.reshape(-1), what + " weight")
    # the same bits on every run, and with gradients written over those that came in
    g2 = api.qk_norm_rope_backward(*args, **s.where(), dq=_t(s.dq), dk=_t(s.dk))
    for a, b in zip(g, g2):
        assert (a is None and b is None) or torch.equal(a, b)


def test_qk_norm_without_rows():
    e = torch.empty(0, 4, 64, dtype=BF, device="cuda")
    w = torch.ones(64, device="cuda")
    rope = api.rope_axes(64, (8, 12, 12))
    q, k = api.qk_norm_rope(e, e, rope, grid=(1, 1, 1), norm="head", q_weight=w, k_weight=w)
    assert q.shape == k.shape == e.shape
    g = api.qk_norm_rope_backward(e, e, e, e, rope, grid=(1, 1, 1), norm="head", q_weight=w, k_weight=w)
    assert not g.q_weight.any() and not g.k_weight.any()


def test_qk_of_one_projection_in_place():
    """Q and K slices of one QKV tensor, rotated where they lie; V untouched."""
    qkv = torch.randn(60, 3, 4, 128, generator=_gen(1), device="cuda").to(BF)
    before = qkv.clone()
    rope = api.rope_axes(128, (22, 21, 21))
    w = torch.rand(512, generator=_gen(2), device="cuda")
    kw = dict(grid=(3, 4, 5), norm="token", q_weight=w, k_weight=w)
    want = api.qk_norm_rope(before[:, 0], before[:, 1], rope, **kw)
    api.qk_norm_rope(qkv[:, 0], qkv[:, 1], rope, **kw, q_out=qkv[:, 0], k_out=qkv[:, 1])
    assert torch.equal(qkv[:, 0], want[0]) and torch.equal(qkv[:, 1], want[1]) and torch.equal(qkv[:, 2], before[:, 2])


def test_qk_bad_values_stay_in_their_row():
    x = torch.randn(40, 3, 128, generator=_gen(1), device="cuda")
    rope, w = api.rope_axes(128, (22, 21, 21)), torch.ones(384, device="cuda")
    kw = dict(grid=(2, 4, 5), norm="token", q_weight=w, k_weight=w)
    want = api.qk_norm_rope(x, x, rope, **kw)
    for bad in (float("nan"), float("inf"), -float("inf")):
        y = x.clone()
        y[7, 1, 5] = bad
        got = api.qk_norm_rope(y, x, rope, **kw)
        keep = torch.arange(40, device="cuda") != 7
        assert torch.equal(got[0][keep], want[0][keep]) and torch.equal(got[1], want[1])
        assert torch.isnan(got[0][7]).any()
    z = torch.zeros_like(x)              # rows of zeros: eps keeps them at zero
    assert not api.qk_norm_rope(z, z, rope, **kw)[0].any()


# ------------------------------------------------------------ row passes --
PARAMS = ("gate", "post_weight", "weight", "bias", "scale", "shift")


def _row(rows, dim, half="both", groups=1, x=BF, b=BF, p=F32, norm="layer", post="none", params=("gate", "scale", "shift"),
         gap=0, off=0, rs=1.0, mean=0.25, apart=0):
    return dict(locals())


ALL = PARAMS
ROW = {
    "one_row": _row(1, 5120, x=F32, norm="rms", params=("gate", "weight")),
    "one_value": _row(3, 1, x=F32, b=F32, norm="rms", params=("gate", "scale", "shift")),
    "two_values": _row(5, 2, x=F32, b=F32, norm="layer"),
    "small": _row(9, 8, params=("gate", "scale", "shift")),
    "wan": _row(130, 5120),
    "frames": _row(42, 1536, groups=21, x=F32, half="norm", params=("scale", "shift")),
    "per_row": _row(65, 320, groups=65, params=ALL, post="rms", norm="rms"),
    "many_groups": _row(2400, 64, groups=600, params=ALL, post="layer", x=F32, b=F32),
    "groups_of_chunks": _row(1900, 136, groups=19, params=ALL, post="rms", x=F32),
    "few_long_groups": _row(3000, 72, groups=2, params=ALL, post="layer", norm="rms"),
    "gate_only": _row(200, 1536, half="gate", groups=4, x=F32, post="rms", params=("gate", "post_weight")),
    "gate_plain": _row(200, 1024, half="gate", params=("gate",), rs=0.5),
    "no_params": _row(100, 640, params=()),
    "weights_only": _row(333, 640, half="norm", params=("weight", "bias")),
    "weights_bf16": _row(333, 640, params=("weight", "bias", "post_weight", "gate"), post="rms", p=BF),
    "odd": _row(251, 1111, x=F32, b=F32, half="gate", post="rms", params=("gate", "post_weight"), rs=0.75),
    "odd_all": _row(101, 1111, x=F32, groups=101, params=ALL, post="layer", norm="layer"),
    "odd_bf16": _row(60, 777, groups=3, params=ALL, post="rms", p=BF),
    "unaligned": _row(50, 256, gap=3, off=1, params=ALL, post="layer", groups=5, apart=1),
    "apart": _row(50, 256, gap=24, off=8, params=ALL, post="layer", groups=5, apart=8),
    "wide": _row(37, 8192, params=ALL, post="rms", x=F32),
    "wider": _row(20, 8200, params=ALL, post="layer", x=F32, b=F32),
    "widest": _row(12, 16384, groups=4, params=ALL, post="rms", norm="layer"),
    "widest_odd": _row(12, 16383, groups=2, params=ALL, post="layer", norm="rms", x=F32),
    "between": _row(40, 5128, params=("gate", "scale", "shift")),
    "many": _row(3001, 1536, params=ALL, post="rms", x=F32),
    "many_of_five": _row(3005, 512, groups=5, params=ALL, post="layer"),
    "long": _row(1207, 5120, params=("gate", "scale", "shift", "weight", "bias")),
    "long_frames": _row(1212, 3584, groups=4, x=F32, b=F32),
    "far_from_zero": _row(64, 2048, x=F32, b=F32, half="norm", params=("scale", "shift"), mean=300.0),
}


class RowCase:
    def __init__(self, c, seed=4):
        self.c, gen = c, _gen(seed)
        mk = lambda dt, mean=0.0, std=1.0: Rows(c["rows"], (c["dim"],), dt, c["gap"], c["off"], gen, mean, std)  # noqa: E731
        norm, gate = c["half"] != "gate", c["half"] != "norm"
        self.x = mk(c["x"], c["mean"])
        self.y = mk(c["b"], 0.1, 0.7) if gate else None
        self.dx, self.dh = mk(c["x"]), (mk(c["b"]) if norm else None)
        self.p = {}
        for n in PARAMS:
            if n not in c["params"]:
                continue
            mod = n in ("gate", "scale", "shift")
            r = Rows(c["groups"] if mod else 1, (c["dim"],), c["p"], c["apart"] if mod else 0, c["apart"] if mod else 0, gen,
                     1.0 if "weight" in n else 0.0, 0.3)
            self.p[n] = r.t if mod else r.t[0]
        self.ref = {n: (_b(self.p[n]).reshape(-1, c["dim"]) if n in self.p else None) for n in PARAMS}
        self.pre = {n: self.p.get(n) for n in ("weight", "bias", "scale", "shift")}
        self.pre.update(norm=c["norm"], eps=1e-6)
        self.post = {n: self.p.get(n) for n in ("gate", "post_weight")}
        self.post.update(post_norm=c["post"], post_eps=1e-5, residual_scale=c["rs"])

    def like(self, r):
        return Rows(r.t.shape[0], r.t.shape[1:], r.t.dtype, self.c["gap"], self.c["off"])

    def definition(self):
        c = self.c
        return R.gate_residual_norm(_b(self.x.t), _b(self.y.t) if self.y else None, self.ref,
                                    c["norm"] if c["half"] != "gate" else None, 1e-6, c["post"], 1e-5, c["rs"])

    def gradients(self, dx):
        c = self.c
        return R.gate_residual_norm_backward(None if dx is None else _b(dx), _b(self.dh.t) if self.dh else None,
                                             _b(self.x.t), _b(self.y.t) if self.y else None, self.ref,
                                             c["norm"] if c["half"] != "gate" else None, 1e-6, c["post"], 1e-5, c["rs"],
                                             c["groups"])

    def forward(self, xo, h):
        if self.c["half"] == "norm":
            return None, api.norm_modulate(self.x.t, out=h, **self.pre)
        if self.c["half"] == "gate":
            return api.gate_residual(self.x.t, self.y.t, out=xo, **self.post), None
        return api.gate_residual_norm(self.x.t, self.y.t, x_out=xo, out=h, **self.post, **self.pre)

    def backward(self, dxo, dx=None, dy=None, ws=None):
        if self.c["half"] == "norm":
            return api.norm_modulate_backward(self.dh.t, self.x.t, dres=dxo, dx=dx, workspace=ws, **self.pre)
        if self.c["half"] == "gate":
            return api.gate_residual_backward(dxo, self.y.t, dy=dy, workspace=ws, **self.post)
        return api.gate_residual_norm_backward(dxo, self.dh.t, self.x.t, self.y.t, dx=dx, dy=dy, workspace=ws, **self.post,
                                               **self.pre)


@pytest.mark.parametrize("name", ROW)
def test_row_forward(name):
    s = RowCase(ROW[name])
    xo = s.like(s.x) if s.y else None
    h = Rows(s.c["rows"], (s.c["dim"],), s.c["b"], s.c["gap"], s.c["off"]) if s.dh else None
    s.forward(_t(xo), _t(h))
    rx, rh = s.definition()
    assert all(r is None or r.intact() for r in (s.x, s.y, xo, h))
    if xo is not None:
        check(xo.t, rx, "x")
    if h is not None:
        check(h.t, rh, "h")
    if s.y is not None:                    # over its inputs, the same bits
        want = (xo.t.clone(), None if h is None else h.t.clone())
        s.forward(s.x.t, s.y.t)
        assert torch.equal(s.x.t, want[0]) and (h is None or torch.equal(s.y.t, want[1]))


@pytest.mark.parametrize("name", ROW)
def test_row_backward(name):
    s = RowCase(ROW[name])
    for with_dx in ((True, False) if s.c["half"] != "gate" else (True,)):
        dxo = s.dx.t if with_dx else None
        dx = s.like(s.x) if s.dh else None
        dy = s.like(s.y) if s.y else None
        need = api.row_workspace_bytes(s.c["rows"], s.c["dim"], s.c["groups"])
        ws = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device="cuda")
        g = s.backward(dxo, _t(dx), _t(dy), ws[:need])
        assert bool((ws[need:] == 0xA5).all())
        ref = s.gradients(dxo)
        assert all(r is None or r.intact() for r in (s.x, s.y, s.dx, s.dh, dx, dy))
        if dx is not None:
            check(dx.t, ref["x"], "x")
        if dy is not None:
            check(dy.t, ref["y"], "y")
        for n in PARAMS:
            got = getattr(g, n)
            if n not in s.p:
                assert got is None, n
            else:
                assert got.shape == s.p[n].shape
                check(got.reshape(-1, s.c["dim"]), ref[n], n)
    g2 = s.backward(dxo)                   # the same bits on every run
    for a, b in zip(g, g2):
        assert (a is None and b is None) or torch.equal(a, b)
    if s.c["half"] == "both":              # over the gradients that came in
        g3 = s.backward(s.dx.t)
        g4 = s.backward(s.dx.t, dx=s.dx.t, dy=s.dh.t)
        for a, b in zip(g3, g4):
            assert (a is None and b is None) or torch.equal(a, b)


def test_row_modulation_for_all_rows_as_a_vector():
    s = RowCase(_row(40, 256))
    a = s.forward(None, None)
    flat = {n: t[0] for n, t in s.p.items()}
    b = api.gate_residual_norm(s.x.t, s.y.t, **flat, norm="layer", post_eps=1e-5)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    g = api.gate_residual_norm_backward(s.dx.t, s.dh.t, s.x.t, s.y.t, **flat, norm="layer")
    assert g.gate.shape == (256,) and torch.equal(g.gate, s.backward(s.dx.t).gate[0])


def test_row_slices_of_one_modulation_table():
    """gate, scale and shift as rows of the table that a time embedding gives."""
    mod = torch.randn(6, 6, 128, generator=_gen(1), device="cuda")
    x, y = (torch.randn(60, 128, generator=_gen(i), device="cuda").to(BF) for i in (2, 3))
    a = api.gate_residual_norm(x, y, gate=mod[:, 2], scale=mod[:, 1], shift=mod[:, 0])
    b = api.gate_residual_norm(x, y, gate=mod[:, 2].contiguous(), scale=mod[:, 1].contiguous(), shift=mod[:, 0].contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_row_without_rows():
    e = torch.empty(0, 64, device="cuda")
    p = torch.ones(1, 64, device="cuda")
    x, h = api.gate_residual_norm(e, e, gate=p, scale=p, shift=p)
    assert x.shape == h.shape == (0, 64)
    g = api.gate_residual_norm_backward(e, e, e, e, gate=p, scale=p, shift=p, weight=p[0])
    assert not any(getattr(g, n).any() for n in ("gate", "scale", "shift", "weight"))


def test_row_bad_values_stay_in_their_row():
    s = RowCase(_row(50, 256, post="rms", params=ALL))
    want = [t.clone() for t in s.forward(None, None)]
    keep = torch.arange(50, device="cuda") != 11
    for bad in (float("nan"), float("inf"), -float("inf"), torch.finfo(BF).min):
        s.y.t[11, 3] = bad
        got = s.forward(None, None)
        assert torch.equal(got[0][keep], want[0][keep]) and torch.equal(got[1][keep], want[1][keep])


def test_row_constant_rows():
    """Layer norm of a constant row is zero, so h is the shift: no variance is
    made of rounding."""
    x = torch.full((5, 1000), 1234.5678, device="cuda")
    t = torch.randn(1, 1000, generator=_gen(1), device="cuda")
    h = api.norm_modulate(x, shift=t, eps=0.01)
    # the mean is off by at most 69 half steps of the value; over sqrt(eps) = 0.1
    assert (h - t).abs().max().item() <= 1234.5678 * 69 * 2.0 ** -24 * 10 * 1.01


# ----------------------------------------------- streams, graphs, devices --
def test_other_stream_and_two_at_once():
    s = RowCase(_row(700, 512, params=ALL, post="rms"))
    want = s.backward(s.dx.t)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for st in streams:
        for _ in range(3):
            got.append(api.gate_residual_norm_backward(s.dx.t, s.dh.t, s.x.t, s.y.t, **s.post, **s.pre, stream=st))
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(want, g):
            assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.parametrize("stride", [1_200_000_000, 2_200_000_000])
def test_offsets_past_32_bits(stride):
    """Rows so far apart that their offsets pass 32 bits, in elements and (the
    wider stride) in bytes of a single step."""
    def rows_of(shape, gen):
        n = int(np.prod(shape[1:]))
        buf = torch.empty(2 * stride + n, dtype=BF, device="cuda")
        t = buf.as_strided(shape, (stride, *(int(np.prod(shape[i + 1:])) for i in range(1, len(shape)))))
        t.copy_(torch.randn(shape, generator=gen, device="cuda"))
        return t

    gen = _gen(11)
    x = rows_of((3, 256), gen)
    y = torch.randn(3, 256, generator=gen, device="cuda").to(BF)
    near = x.contiguous()
    for a, b in zip(api.gate_residual_norm(x, y), api.gate_residual_norm(near, y)):
        assert torch.equal(a, b)
    for a, b in zip(api.gate_residual_norm_backward(x, y, x, y)[:2], api.gate_residual_norm_backward(near, y, near, y)[:2]):
        assert torch.equal(a, b)
    api.norm_modulate(near, out=x)
    assert torch.equal(x, api.norm_modulate(near))
    del x
    q = rows_of((3, 2, 128), gen)
    w, rope = torch.rand(256, generator=gen, device="cuda"), api.rope_axes(128, (22, 21, 21))
    kw = dict(grid=(1, 1, 3), norm="token", q_weight=w, k_weight=w)
    near = q.contiguous()
    k = torch.randn(3, 2, 128, generator=gen, device="cuda").to(BF)
    for a, b in zip(api.qk_norm_rope(q, k, rope, **kw), api.qk_norm_rope(near, k, rope, **kw)):
        assert torch.equal(a, b)
    far, want = api.qk_norm_rope_backward(q, k, q, k, rope, **kw), api.qk_norm_rope_backward(near, k, near, k, rope, **kw)
    half = 2.0 ** -8          # another split of the heads over threads: the sums' order, so a rounding, may differ
    for a, b in zip(far, want):
        assert (a.float() - b.float()).abs().max() <= 2.01 * half * b.float().abs().max()


def test_callers_on_several_host_threads():
    """Calls of one kernel with rings of different sizes from host threads at
    once, each on its own stream."""
    import threading
    cases = [RowCase(_row(rows, 5120, params=("scale", "shift"), half="norm")) for rows in (150, 700, 2400)]
    want = [s.forward(None, None)[1] for s in cases]
    torch.cuda.synchronize()
    got, errors = [[] for _ in cases], []

    def work(i):
        try:
            st = torch.cuda.Stream()
            for _ in range(50):
                got[i].append(api.norm_modulate(cases[i].x.t, **cases[i].pre, stream=st))
            st.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors, errors
    for w, g in zip(want, got):
        assert all(torch.equal(w, x) for x in g)


def test_no_parameter_gradients():
    x, y = (torch.randn(300, 512, generator=_gen(i), device="cuda") for i in (1, 2))
    ws = torch.full((api.row_workspace_bytes(300, 512),), 0xA5, dtype=torch.uint8, device="cuda")
    g = api.gate_residual_norm_backward(x, y, x, y, workspace=ws)
    assert bool((ws == 0xA5).all())
    assert g.x.shape == g.y.shape == x.shape and g.gate is None and g.weight is None
    ref = R.gate_residual_norm_backward(_b(x), _b(y), _b(x), _b(y), {n: None for n in PARAMS}, "layer", 1e-6, "none", 1e-6, 1.0)
    check(g.x, ref["x"], "x")
    check(g.y, ref["y"], "y")


def test_same_tensor_for_q_and_k():
    """One tensor as Q and as K, read twice, written to two outputs."""
    x = torch.randn(60, 4, 128, generator=_gen(1), device="cuda").to(BF)
    rope = api.rope_axes(128, (22, 21, 21))
    q, k = api.qk_norm_rope(x, x, rope, grid=(3, 4, 5))
    assert torch.equal(q, k)
    with pytest.raises(RuntimeError):
        api.qk_norm_rope(x, x, rope, grid=(3, 4, 5), q_out=x, k_out=x)
    with pytest.raises(RuntimeError):
        api.qk_norm_rope(x, x, rope, grid=(3, 4, 5), q_out=x)          # K would read what Q wrote


def test_captured_and_replayed():
    """Two graphs that share a workspace, replayed one after the other on new
    inputs."""
    s = RowCase(_row(700, 512, params=ALL, post="rms"))
    c = QkCase(QK["shared_keys"])
    ws = torch.empty(max(api.row_workspace_bytes(700, 512), api.qk_norm_rope_workspace_bytes(333, 40, 8, 128, "head")),
                     dtype=torch.uint8, device="cuda")

    def row():
        return s.backward(s.dx.t, ws=ws)

    def qk():
        return (*api.qk_norm_rope(c.q.t, c.k.t, c.rope, **c.where()),
                *api.qk_norm_rope_backward(c.dq.t, c.dk.t, c.q.t, c.k.t, c.rope, **c.where(), workspace=ws))

    row(), qk()
    graphs, outs = [], []
    for f in (row, qk):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f())
        graphs.append(g)
    for seed in (8, 9):
        s.y.t.copy_(torch.randn(s.y.t.shape, generator=_gen(seed), device="cuda"))
        c.k.t.copy_(torch.randn(c.k.t.shape, generator=_gen(seed), device="cuda"))
        for g in graphs:
            g.replay()
        got = [[t.clone() for t in o if t is not None] for o in outs]
        for f, o in zip((row, qk), got):
            for a, b in zip([t for t in f() if t is not None], o):
                assert torch.equal(a, b)
    torch.cuda.synchronize()


def test_refusals():
    x = torch.zeros(6, 64, device="cuda")
    rope = api.rope_axes(64, (8, 12, 12))
    q = x.view(6, 1, 64)
    cases = [
        (ValueError, lambda: api.norm_modulate(x, scale=torch.zeros(4, 64, device="cuda"))),       # 6 rows in 4 groups
        (ValueError, lambda: api.norm_modulate(x, scale=torch.zeros(2, 64, device="cuda"), shift=torch.zeros(3, 64, device="cuda"))),
        (ValueError, lambda: api.norm_modulate(x, weight=torch.zeros(63, device="cuda"))),
        (ValueError, lambda: api.norm_modulate(x, weight=torch.zeros(64))),
        (TypeError, lambda: api.norm_modulate(x, weight=torch.zeros(64, device="cuda"), bias=torch.zeros(64, device="cuda", dtype=BF))),
        (TypeError, lambda: api.norm_modulate(x.half())),
        (ValueError, lambda: api.norm_modulate(x, norm="group")),
        (ValueError, lambda: api.norm_modulate(x.t())),
        (ValueError, lambda: api.norm_modulate(x[:1].expand(6, 64))),
        (ValueError, lambda: api.norm_modulate(x[0])),
        (ValueError, lambda: api.gate_residual(x, x[:5])),
        (TypeError, lambda: api.gate_residual(x, x, out=x.to(BF))),
        (RuntimeError, lambda: api.gate_residual(x.to(BF), x)),
        (RuntimeError, lambda: api.gate_residual(x[:5], x[:5], out=x[1:])),
        (RuntimeError, lambda: api.norm_modulate_backward(x, x, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))),
        (ValueError, lambda: api.qk_norm_rope(q, q, rope)),
        (ValueError, lambda: api.qk_norm_rope(None, None, rope, grid=(1, 2, 3))),
        (ValueError, lambda: api.qk_norm_rope(q, q, rope, grid=(1, 2, 3), positions=torch.zeros(6, 3, dtype=torch.int32, device="cuda"))),
        (ValueError, lambda: api.qk_norm_rope(q, q, rope, positions=torch.zeros(6, 3, dtype=torch.int32))),
        (TypeError, lambda: api.qk_norm_rope(q, q, rope, positions=torch.zeros(6, 3, dtype=torch.int64, device="cuda"))),
        (ValueError, lambda: api.qk_norm_rope(q, q, rope, positions=torch.zeros(5, 3, dtype=torch.int32, device="cuda"))),
        (RuntimeError, lambda: api.qk_norm_rope(q, q, rope, grid=(1, 2, 2))),
        (ValueError, lambda: api.qk_norm_rope(q, q, rope, grid=(1, 2, 3), norm="token", q_weight=torch.ones(63, device="cuda"))),
        (RuntimeError, lambda: api.qk_norm_rope(q, q, rope, grid=(1, 2, 3), q_weight=torch.ones(64, device="cuda"))),
        (ValueError, lambda: api.qk_norm_rope(q, q.view(1, 6, 64), rope, grid=(1, 2, 3))),
        (RuntimeError, lambda: api.qk_norm_rope_backward(q, q, None, None, rope, grid=(1, 2, 3), norm="head")),
    ]
    for i, (error, call) in enumerate(cases):
        with pytest.raises(error):
            call()
            pytest.fail(f"case {i} was not refused")


# ------------------------------------------------------- together: a layer --
def test_layer_around_the_attention():
    """norm_modulate -> projection -> qk_norm_rope -> grouped attention ->
    projection -> gate_residual_norm, as a layer runs them, against the same
    chain in float64 on the attention's own kept lists."""
    wl = Workload("layer", 12, 4, 16, 16, 3, 128, "bf16", 0, (Scheme(4, 16, 16, 2, 8, 8),), (0,) * 3, (0.9,) * 3, (False,) * 3)
    n, dim, gen = wl.N, 3 * 128, _gen(7)
    x = torch.randn(n, dim, generator=gen, device="cuda")
    mod = torch.randn(6, dim, generator=gen, device="cuda") * 0.3
    wqkv = (torch.randn(3 * dim, dim, generator=gen, device="cuda") * dim ** -0.5).to(BF)
    wo = (torch.randn(dim, dim, generator=gen, device="cuda") * dim ** -0.5).to(BF)
    qw, kw = (torch.rand(dim, generator=gen, device="cuda") + 0.5 for _ in range(2))
    rope = api.rope_axes(128, (22, 21, 21))

    h = api.norm_modulate(x, scale=mod[1], shift=mod[0], out_dtype=BF)
    qkv = (h @ wqkv.t()).view(n, 3, 3, 128)
    q, k = api.qk_norm_rope(qkv[:, 0], qkv[:, 1], rope, grid=wl.schemes[0].as_tuple()[:3], norm="token", q_weight=qw,
                            k_weight=kw)
    v = qkv[:, 2].contiguous()
    o, _, kept = run_grouped(wl, q, k, v)
    y = o.view(n, dim) @ wo.t()
    x2, h2 = api.gate_residual_norm(x, y, gate=mod[2], scale=mod[4], shift=mod[3])

    p = {"gate": None, "post_weight": None, "weight": None, "bias": None, "scale": to_np(mod[1:2]), "shift": to_np(mod[:1])}
    _, rh = R.gate_residual_norm(to_np(x), None, p, "layer", 1e-6, "none", 0.0, 1.0)
    half = 2.0 ** -8
    assert np.abs(to_np(h) - rh).max() <= np.abs(rh).max() * (half + 2.0 ** -16)
    axis, freq = R.rope_ladder((22, 21, 21), (1e4,) * 3)
    cos, sin = R.rope_angles(R.grid_positions(n, 0, *wl.schemes[0].as_tuple()[:3]), axis, freq, 128)
    for got, src, w in ((q, qkv[:, 0], qw), (k, qkv[:, 1], kw)):
        ref = R.qk_norm_rope(to_np(src), to_np(w).reshape(3, 128), cos, sin, "token", 1e-6, "interleaved")
        assert np.abs(to_np(got) - ref).max() <= np.abs(ref).max() * (half + 2.0 ** -16)
    ro = O.block_sparse_attention(to_np(q), to_np(k), to_np(v), [wl.schemes[0].as_tuple()] * 3, [kept(i) for i in range(3)], 0)
    assert np.abs(to_np(o) - ro).mean() <= ATTN_MEAN_ABS_BF16
    p.update(gate=to_np(mod[2:3]), scale=to_np(mod[4:5]), shift=to_np(mod[3:4]))
    rx2, rh2 = R.gate_residual_norm(to_np(x), to_np(y), p, "layer", 1e-6, "none", 0.0, 1.0)
    assert np.abs(to_np(x2) - rx2).max() <= np.abs(rx2).max() * 2.0 ** -20
    assert np.abs(to_np(h2) - rh2).max() <= np.abs(rh2).max() * (half + 2.0 ** -16)
