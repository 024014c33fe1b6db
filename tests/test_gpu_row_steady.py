"""The row passes where a real size spends its time: blocks that refill their
ring of rows many times over, make angles again and again and cross from one
modulation group to the next, in every layout (pieces of 16, 8, 4 and 2 bytes,
one, two and four units or eights of columns a thread, even and uneven), against
the float64 definitions on the GPU within the bounds of bounded_gpu.py.

A ring holds at most 14 rows.  Rows are chosen so that the busiest layout, with
as many blocks of an SM as its registers allow, has more than 28 a block (or
more than twice the fewer that its ring holds)."""
import pytest
import torch

import bounded_gpu as G
from bounded_gpu import Bounded, check
from input_adaptive_block_b200 import api
from oracle import row_oracle as R
from test_gpu_row_passes import ALL, BF, F32, PARAMS, QkCase, RowCase, Rows, _qk, _row, _t

pytestmark = pytest.mark.gpu

CHUNK = 4_000_000        # elements of a chunk that goes through the definition


@pytest.fixture(autouse=True)
def row_steps(monkeypatch):
    """Additions of a column's sum over `rows` rows before it is kept in
    float64.  With resident blocks at least one to an SM, a block of a Q/K pass
    has at most rows / SMs + 1 rows and a unit of a row pass, or all of a block's
    units together, at most 2 rows / SMs + 8 (of the cuts that are tried, the
    one that fills the resident blocks eight times has no more, and the best is
    taken); the heads of a warp and the warps then add 5 and 32, and what else
    a single sum counts is in SUM_STEPS."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count

    def of(rows):
        monkeypatch.setattr(Bounded, "row_steps", 2 * (rows // sms + 1) + 8 + G.SUM_STEPS)

    return of


# ------------------------------------------------------------------- Q/K --
def _grid(rows, text=0, offset=0):
    return (-(-(rows - text + offset) // (30 * 31)), 30, 31)


def _many(rows, text=0, offset=0, **kw):
    if "positions" not in kw:
        kw["grid"] = _grid(rows, text, offset)
    return _qk(rows, text=text, offset=offset, **kw)


SIX = 148 * 6 * 30 + 37          # 30 tokens and more to a block, six blocks to an SM
FORTY = dict(qh=40, kh=40)
TWELVE = dict(qh=12, kh=12)
QK = {
    "token": _many(SIX, text=33, offset=7, **TWELVE),
    "token_40": _many(20001, **FORTY),
    "head_40": _many(8003, norm="head", positions="far", **FORTY),
    "none_40": _many(8001, norm="none", text=500, **FORTY),
    "uneven_half": _many(8003, qh=40, kh=33, style="half", norm="head", text=1),
    "uneven_token": _many(8002, qh=40, kh=33, positions="far"),
    "q_40": _many(9001, qh=40, kh=0),
    "k_side": _many(SIX, qh=10, kh=6, norm="token", wdt=BF),
    "f32": _many(20001, dtype=F32, **TWELVE),
    "f32_head": _many(20003, dtype=F32, norm="head", style="half", **TWELVE),
    "f32_40": _many(6001, dtype=F32, **FORTY),
    "f32_uneven_half": _many(6003, qh=40, kh=33, dtype=F32, norm="head", style="half"),
    "f32_none": _many(6003, norm="none", dtype=F32, style="half", **FORTY),
    "four_units": _many(3001, qh=45, kh=20, d=192, pairs=(32, 32, 32), style="half", norm="head"),
    "four_units_token": _many(3003, d=160, pairs=(30, 25, 25), **FORTY),
    "four_units_f32": _many(2003, d=160, pairs=(30, 25, 25), dtype=F32, **FORTY),
    "four_units_narrow": _many(2003, d=160, pairs=(30, 25, 25), gap=2, off=2, norm="head", **FORTY),
    "four_units_single": _many(2003, d=160, pairs=(30, 25, 25), style="half", gap=1, off=1, **FORTY),
    "pieces_of_two": _many(SIX, gap=2, off=2, **TWELVE),
    "pieces_of_two_half": _many(SIX, qh=14, kh=5, d=76, pairs=(14, 12, 12), style="half", norm="head", text=9),
    "pieces_of_two_40": _many(4003, gap=2, off=2, **FORTY),
    "pieces_of_two_half_40": _many(4003, gap=2, off=2, style="half", norm="head", **FORTY),
    "single": _many(20001, gap=3, off=1, **TWELVE),
    "single_half": _many(20001, gap=3, off=1, style="half", norm="head", **TWELVE),
    "single_40": _many(4003, gap=3, off=1, **FORTY),
    "single_half_40": _many(4003, gap=3, off=1, style="half", norm="head", **FORTY),
    "f32_single": _many(20001, qh=12, kh=5, d=80, pairs=(16, 12, 12), style="half", norm="head", dtype=F32, gap=1, off=1),
    "f32_single_40": _many(4001, gap=1, off=1, dtype=F32, **FORTY),
    "few_heads": _many(148 * 8 * 30 + 37, qh=2, kh=1, d=64, pairs=(8, 12, 12), norm="head", text=300),
    "few_heads_f32": _many(148 * 8 * 30 + 37, qh=1, kh=1, norm="token", dtype=F32),
    "odd_pairs": _many(40003, qh=5, kh=2, d=34, pairs=(7, 5, 5), norm="token"),
    "odd_half": _many(40003, qh=5, kh=2, d=38, pairs=(7, 6, 6), style="half", norm="head"),
    "few_pairs": _many(SIX, d=96, pairs=(9, 3, 0), norm="token", positions="far", **TWELVE),
}


def _pieces(rows, inner):
    step = max(1, CHUNK // inner)
    return [slice(i, min(i + step, rows)) for i in range(0, rows, step)]


class Definition:
    def __init__(self, s):
        self.s, self.cos, self.sin = s, Bounded.of(s.cos), Bounded.of(s.sin)

    def _given(self, w, x):
        if w is None:
            return Bounded.of(torch.ones(1, 1, dtype=torch.float64, device="cuda"))
        return Bounded.of(w).reshape(x.shape[1] if self.s.c["norm"] == "token" else 1, x.shape[2])

    def forward(self, x, w, at):
        c = self.s.c
        return R.qk_norm_rope(Bounded.of(x[at]), self._given(w, x), self.cos[at], self.sin[at], c["norm"], c["eps"], c["style"])

    def backward(self, g, x, w, at):
        c = self.s.c
        return R.qk_norm_rope_backward(Bounded.of(g[at]), Bounded.of(x[at]), self._given(w, x), self.cos[at], self.sin[at],
                                       c["norm"], c["eps"], c["style"])


def _outs(s):
    return [None if r is None else Rows(r.t.shape[0], r.t.shape[1:], r.t.dtype, s.c["gap"], s.c["off"]) for r in (s.q, s.k)]


@pytest.mark.parametrize("name", QK)
def test_qk_forward(name):
    s = QkCase(QK[name])
    outs, ref = _outs(s), Definition(s)
    api.qk_norm_rope(_t(s.q), _t(s.k), s.rope, **s.where(), q_out=_t(outs[0]), k_out=_t(outs[1]))
    for x, w, o, what in ((s.q, s.qw, outs[0], "q"), (s.k, s.kw, outs[1], "k")):
        if x is None:
            continue
        assert o.intact() and x.intact(), what
        for at in _pieces(s.c["rows"], x.n):
            check(o.t[at], ref.forward(x.t, w, at), (what, at))
    # over its own input, the same bits
    api.qk_norm_rope(_t(s.q), _t(s.k), s.rope, **s.where(), q_out=_t(s.q), k_out=_t(s.k))
    for x, o in ((s.q, outs[0]), (s.k, outs[1])):
        assert x is None or torch.equal(x.t, o.t)


@pytest.mark.parametrize("name", QK)
def test_qk_backward(name, row_steps):
    s = QkCase(QK[name])
    row_steps(s.c["rows"])
    outs, ref = _outs(s), Definition(s)
    args = (_t(s.dq), _t(s.dk), _t(s.q), _t(s.k), s.rope)
    g = api.qk_norm_rope_backward(*args, **s.where(), dq=_t(outs[0]), dk=_t(outs[1]))
    for x, gr, w, o, dw, what in ((s.q, s.dq, s.qw, outs[0], g.q_weight, "q"), (s.k, s.dk, s.kw, outs[1], g.k_weight, "k")):
        if x is None:
            continue
        assert o.intact() and x.intact() and gr.intact(), what
        total = None
        for at in _pieces(s.c["rows"], x.n):
            dx, part = ref.backward(gr.t, x.t, w, at)
            check(o.t[at], dx, (what, at))
            total = part if total is None or part is None else total.plus(part)
        if w is not None:
            check(dw, total.reshape(-1), what + " weight")
    g2 = api.qk_norm_rope_backward(*args, **s.where(), dq=_t(s.dq), dk=_t(s.dk))
    for a, b in zip(g, g2):
        assert (a is None and b is None) or torch.equal(a, b)


# ------------------------------------------------------------ row passes --
MOST = tuple(n for n in ALL if n != "post_weight")
ROWS = 148 * 3 * 30 + 37         # 30 rows and more to a block, three blocks to an SM
ROW = {
    "one_group": _row(ROWS, 1536),
    "one_group_norm": _row(ROWS, 1536, half="norm", params=("scale", "shift", "weight", "bias")),
    "groups": _row(20 * 670, 1536, groups=20),
    "groups_norm_f32_stream": _row(21 * 763, 1536, groups=21, x=F32, half="norm", params=("scale", "shift")),
    "groups_post": _row(21 * 763, 1536, groups=21, x=F32, params=ALL, post="rms", norm="rms"),
    "post": _row(ROWS, 1536, params=ALL, post="layer"),
    "f32": _row(ROWS, 1536, x=F32, b=F32, params=MOST),
    "f32_post": _row(ROWS, 1536, x=F32, b=F32, params=ALL, post="rms"),
    "gate": _row(ROWS, 1536, half="gate", params=("gate",)),
    "gate_post": _row(21 * 763, 1536, half="gate", groups=21, x=F32, params=("gate", "post_weight"), post="rms"),
    "gate_post_f32": _row(ROWS, 1536, half="gate", x=F32, b=F32, params=("gate", "post_weight"), post="layer", rs=0.5),
    "uneven": _row(ROWS, 1400, params=MOST),
    "wan": _row(8001, 5120),
    "wan_post": _row(20 * 200, 5120, groups=20, params=ALL, post="layer"),
    "wan_mixed": _row(4001, 5120, x=F32, params=ALL, post="rms"),
    "wan_f32": _row(4001, 5120, x=F32, b=F32, params=MOST),
    "wan_norm": _row(8003, 5120, half="norm", params=("scale", "shift")),
    "wan_gate_f32": _row(4003, 5120, half="gate", x=F32, b=F32, params=("gate", "post_weight"), post="rms"),
    "sixteen_uneven": _row(8003, 2568, params=MOST),
    "sixteen_mixed": _row(8003, 2564, x=F32, params=ALL, post="layer"),
    "pieces_of_two": _row(24003, 770, params=MOST),
    "pieces_of_four": _row(ROWS, 1108, params=ALL, post="rms"),
    "pieces_of_two_apart": _row(ROWS, 1536, gap=2, off=2, params=MOST, apart=2),
    "pieces_of_two_norm": _row(20 * 670, 1538, half="norm", groups=20, params=("scale", "shift", "weight", "bias")),
    "pieces_of_two_gate": _row(ROWS, 1538, half="gate", params=("gate", "post_weight"), post="layer"),
    "pieces_of_two_long": _row(4001, 5118, params=ALL, post="layer"),
    "single": _row(ROWS, 777, params=ALL, post="rms"),
    "single_norm": _row(ROWS, 777, half="norm", params=("scale", "shift")),
    "single_mixed": _row(ROWS, 1111, x=F32, params=MOST),
    "single_f32": _row(ROWS, 1111, x=F32, b=F32, params=ALL, post="layer"),
    "single_f32_even": _row(ROWS, 1110, x=F32, b=F32, params=MOST),
    "per_row": _row(45003, 320, groups=45003, params=ALL, post="rms"),
    "per_row_norm": _row(ROWS, 1536, groups=ROWS, half="norm", params=("scale", "shift")),
    "groups_of_five": _row(5 * 9001, 512, groups=9001, params=ALL, post="layer"),
    "groups_of_five_norm": _row(5 * 3001, 1536, groups=3001, x=F32, half="norm", params=("scale", "shift", "weight")),
    "long_rows": _row(2003, 8192, params=ALL, post="rms", x=F32),
    "long_rows_f32": _row(2003, 6144, params=MOST, x=F32, b=F32),
    "longer_rows": _row(2003, 8200, params=ALL, post="layer", x=F32, b=F32),
    "longest_rows": _row(2004, 16384, groups=4, params=MOST),
    "long_rows_single": _row(2003, 5121, params=ALL, post="rms"),
    "short_rows": _row(148 * 16 * 30 + 37, 8, params=MOST),
}


def _row_pieces(rows, dim, groups):
    """Pieces of whole groups, or of the rows of a single one."""
    per = rows // groups
    step = max(1, CHUNK // dim)
    if groups > 1:
        step = max(1, step // per) * per
    return [slice(i, min(i + step, rows)) for i in range(0, rows, step)]


class RowDefinition:
    def __init__(self, s):
        self.s, self.c = s, s.c
        self.per = s.c["rows"] // s.c["groups"]
        self.p = {n: None if s.p.get(n) is None else Bounded.of(s.p[n]).reshape(-1, s.c["dim"]) for n in PARAMS}

    def groups_at(self, at):
        """Modulation groups of the rows at `at`."""
        return slice(0, 1) if self.c["groups"] == 1 else slice(at.start // self.per, at.stop // self.per)

    def at(self, at):
        g = self.groups_at(at)
        return {n: p if p is None or n not in ("gate", "scale", "shift") else p[g] for n, p in self.p.items()}

    def _rows(self, r, at):
        return None if r is None else Bounded.of(r.t[at])

    def forward(self, at):
        s, c = self.s, self.c
        return R.gate_residual_norm(self._rows(s.x, at), self._rows(s.y, at), self.at(at),
                                    c["norm"] if c["half"] != "gate" else None, 1e-6, c["post"], 1e-5, c["rs"])

    def backward(self, dx, at):
        s, c, g = self.s, self.c, self.groups_at(at)
        return R.gate_residual_norm_backward(None if dx is None else Bounded.of(dx[at]), self._rows(s.dh, at),
                                             self._rows(s.x, at), self._rows(s.y, at), self.at(at),
                                             c["norm"] if c["half"] != "gate" else None, 1e-6, c["post"], 1e-5, c["rs"],
                                             g.stop - g.start)


@pytest.mark.parametrize("name", ROW)
def test_row_forward(name):
    s = RowCase(ROW[name])
    ref = RowDefinition(s)
    xo = s.like(s.x) if s.y else None
    h = Rows(s.c["rows"], (s.c["dim"],), s.c["b"], s.c["gap"], s.c["off"]) if s.dh else None
    s.forward(_t(xo), _t(h))
    assert all(r is None or r.intact() for r in (s.x, s.y, xo, h))
    for at in _row_pieces(s.c["rows"], s.c["dim"], s.c["groups"]):
        rx, rh = ref.forward(at)
        if xo is not None:
            check(xo.t[at], rx, ("x", at))
        if h is not None:
            check(h.t[at], rh, ("h", at))
    if s.y is not None:                    # over its inputs, the same bits
        s.forward(s.x.t, s.y.t)
        assert torch.equal(s.x.t, xo.t) and (h is None or torch.equal(s.y.t, h.t))


@pytest.mark.parametrize("name", ROW)
def test_row_backward(name, row_steps):
    s = RowCase(ROW[name])
    c = s.c
    row_steps(c["rows"])
    ref = RowDefinition(s)
    dx = s.like(s.x) if s.dh else None
    dy = s.like(s.y) if s.y else None
    g = s.backward(s.dx.t, _t(dx), _t(dy))
    assert all(r is None or r.intact() for r in (s.x, s.y, s.dx, s.dh, dx, dy))
    sums, mods = {}, {n: [] for n in PARAMS}
    for at in _row_pieces(c["rows"], c["dim"], c["groups"]):
        part = ref.backward(s.dx.t, at)
        if dx is not None:
            check(dx.t[at], part["x"], ("x", at))
        if dy is not None:
            check(dy.t[at], part["y"], ("y", at))
        for n in s.p:
            if n in ("gate", "scale", "shift") and c["groups"] > 1:
                mods[n].append((ref.groups_at(at), part[n]))
            else:
                sums[n] = part[n] if n not in sums else sums[n].plus(part[n])
    for n in s.p:
        got = getattr(g, n).reshape(-1, c["dim"])
        for at, part in mods[n]:
            check(got[at], part, (n, at))
        if n in sums:
            check(got, sums[n], n)
    g2 = s.backward(s.dx.t, dx=s.dx.t if s.dh else None, dy=s.dh.t if s.dh and s.y else None)      # over what came in
    for a, b in zip(g, g2):
        assert (a is None and b is None) or torch.equal(a, b)
