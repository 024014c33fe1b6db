"""What is measured of the row passes around the block-sparse attention of a
video-diffusion-transformer layer: the norm and several-axis rotation of Q and
K before it, and the modulated norms and gated residual updates on either side
of a block.  `run` computes them in plain torch, or, where `own` is true, by
the calls that a user makes of the framework."""
import functools
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # Q and K of one Wan-14B 720p layer as slices of one QKV projection: norm over the whole token, then rotation
        _qk("qk_14b", rows=75600, T=21, H=45, W=80, q_heads=40, k_heads=40, norm="token", fused=True),
        # the same norm and rotation in training, Wan-1.3B 480p
        _qk("qk_1.3b_bwd", rows=32760, T=21, H=30, W=52, q_heads=12, k_heads=12, norm="token", back=True),
        # a long clip with 256 text tokens behind it, norm per head, one frequency base of 256
        _qk("qk_text", rows=33 * 45 * 80 + 256, T=33, H=45, W=80, q_heads=20, k_heads=20, pairs=(8, 28, 28), theta=256.0,
            norm="head", text=256),
        # one new token far into a stream, fewer key heads
        _qk("qk_one", rows=1, q_heads=40, k_heads=8, norm="head", explicit=True),
        # image tokens of several sizes packed in one list, in training; 80 channels a head, halves paired, odd row count
        _qk("qk_packed_bwd", rows=4999, q_heads=14, k_heads=2, d=80, pairs=(16, 12, 12), norm="head", explicit=True,
            style="half", dtype="f32", back=True),
        # the norm that opens a block of Wan-14B at 720p: one modulation for the clip
        _row("norm_14b", "norm", rows=75600, dim=5120, scale=True, shift=True),
        # the same in training at Wan-1.3B 480p, the stream in 32 bits, one modulation for each latent frame
        _row("norm_frames_bwd", "norm", rows=32760, dim=1536, groups=21, x="f32", scale=True, shift=True, back=True),
        # the end of one block and the norm of the next, Wan-14B at 720p
        _row("gate_norm_14b", "gate_norm", rows=75600, dim=5120, gate=True, scale=True, shift=True),
        _row("gate_norm_14b_bwd", "gate_norm", rows=75600, dim=5120, gate=True, scale=True, shift=True, back=True),
        # one token between two blocks, with weights and no modulation
        _row("gate_norm_one", "gate_norm", rows=1, dim=5120, x="f32", norm="rms", weight=True, gate=True),
        # a block whose output is normalised before it joins the stream
        _row("gate_1.3b", "gate", rows=32760, dim=1536, x="f32", groups=21, gate=True, post="rms", post_weight=True),
        # the same in training: odd sizes, everything in 32 bits, a constant on the branch
        _row("gate_odd_bwd", "gate", rows=2501, dim=1111, x="f32", branch="f32", gate=True, post="rms", post_weight=True,
             residual_scale=0.75, back=True),
    ]


def _qk(name, rows, q_heads, k_heads, T=1, H=1, W=1, d=128, pairs=(22, 21, 21), theta=10000.0, style="interleaved",
        norm="none", dtype="bf16", text=0, offset=0, explicit=False, fused=False, back=False):
    return {"name": name, "op": "qk", "rows": rows, "T": T, "H": H, "W": W, "q_heads": q_heads, "k_heads": k_heads, "d": d,
            "pt": pairs[0], "py": pairs[1], "px": pairs[2], "theta": theta, "style": style, "norm": norm, "dtype": dtype,
            "text": text, "offset": offset, "explicit": explicit, "fused": fused, "back": back}


def _row(name, op, rows, dim, groups=1, x="bf16", branch="bf16", norm="layer", weight=False, bias=False, scale=False,
         shift=False, gate=False, post="none", post_weight=False, residual_scale=1.0, back=False):
    return {"name": name, "op": op, "rows": rows, "dim": dim, "groups": groups, "x": x, "branch": branch, "norm": norm,
            "weight": weight, "bias": bias, "scale": scale, "shift": shift, "gate": gate, "post": post,
            "post_weight": post_weight, "residual_scale": residual_scale, "back": back}


def _log_uniform(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def draw(rng):
    back = rng.random() < 0.5
    if rng.random() < 0.45:
        d = 2 * rng.randint(16, 80) if rng.random() < 0.3 else rng.choice([64, 80, 96, 128, 160, 256])
        style = rng.choice(["interleaved", "half"])
        py = px = (d // 2) // 3 if rng.random() < 0.6 else (d // 2) // 4
        pt = d // 2 - py - px
        k_heads = _log_uniform(rng, 1, 40)
        q_heads = min(48, k_heads * rng.choice([1, 1, 2, 5]))
        dtype = rng.choice(["bf16", "bf16", "f32"])
        most = 3.5e8 / (q_heads + k_heads) / d
        explicit = rng.random() < 0.35
        if explicit:
            T = H = W = 1
            text, offset, rows = 0, 0, _log_uniform(rng, 1, int(min(most, 80000)))
        else:
            T, H, W = rng.randint(1, 33), rng.randint(1, 45), rng.randint(1, 80)
            text = rng.choice([0, 0, 1, rng.randint(2, 300)])
            offset = rng.randint(0, T * H * W - 1) if rng.random() < 0.3 else 0
            rows = min(T * H * W - offset, max(1, int(most) - text)) + text
        return _qk("", rows, q_heads, k_heads, T, H, W, d, (pt, py, px), rng.choice([256.0, 10000.0, 1000000.0]), style,
                   rng.choice(["none", "token", "head"]), dtype, text, offset, explicit, rng.random() < 0.4 and q_heads == k_heads, back)
    op = rng.choice(["norm", "gate", "gate_norm"])
    dim = _log_uniform(rng, 64, 8192)
    dim = dim if rng.random() < 0.3 else max(64, dim // 64 * 64)
    kind = rng.random()
    rows = _log_uniform(rng, 1, int(min(80000, (0.5e8 if kind < 0.15 else 1.5e8) / dim)))
    groups = rows if kind < 0.15 else rng.randint(1, min(rows, 33)) if kind < 0.5 else 1
    rows = rows // groups * groups
    x, branch = rng.choice([("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
    weight = rng.random() < 0.4
    post = "none" if op == "norm" else rng.choice(["none", "none", "rms", "layer"])
    return _row("", op, rows, dim, groups, x, branch, rng.choice(["layer", "rms"]), weight, weight and rng.random() < 0.5,
                rng.random() < 0.7, rng.random() < 0.6, op != "norm" and rng.random() < 0.8, post,
                post != "none" and rng.random() < 0.7, rng.choice([1.0, 0.5]), back)


# ---------------------------------------------------------------- inputs --
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32, mean=0.0, std=1.0):
        t = torch.empty(shape, dtype=dtype, device="cuda")
        return t.normal_(mean, std, generator=gen)

    s = {"case": case}
    if case["op"] == "qk":
        rows, qh, kh, d, dt = case["rows"], case["q_heads"], case["k_heads"], case["d"], DTYPES[case["dtype"]]
        # projections of a normalised stream: unit size, some channels several times larger
        if case["fused"]:
            qkv = normal(rows, 3, qh, d, dtype=dt)
            qkv[..., 3::17] *= 4.0
            s["q"], s["k"] = qkv[:, 0], qkv[:, 1]
        else:
            s["q"], s["k"] = normal(rows, qh, d, dtype=dt), normal(rows, kh, d, dtype=dt, std=1.5)
            s["q"][..., 3::17] *= 4.0
        s["qw"] = s["kw"] = None
        if case["norm"] != "none":
            s["qw"] = normal(qh * d if case["norm"] == "token" else d, mean=1.0, std=0.2)
            s["kw"] = normal(kh * d if case["norm"] == "token" else d, mean=1.0, std=0.2)
        s["pos"] = None
        if case["explicit"]:  # a long stream's frames, and places within a frame
            s["pos"] = torch.stack([torch.randint(0, n, (rows,), generator=gen, device="cuda", dtype=torch.int32)
                                    for n in (200000, 128, 128)], dim=1)
        if case["back"]:
            s["dq"], s["dk"] = normal(rows, qh, d, dtype=dt), normal(rows, kh, d, dtype=dt)
        return s
    rows, dim, groups, xt, bt = case["rows"], case["dim"], case["groups"], DTYPES[case["x"]], DTYPES[case["branch"]]
    # a residual stream: off centre, a few channels far larger than the rest
    s["xs"] = normal(rows, dim, dtype=xt, mean=0.25, std=1.0)
    s["xs"][:, 7::251] *= 20.0
    s["ys"] = normal(rows, dim, dtype=bt, std=0.7) if case["op"] != "norm" else None
    s["w"] = normal(dim, mean=1.0, std=0.2) if case["weight"] else None
    s["b"] = normal(dim, std=0.2) if case["bias"] else None
    s["pw"] = normal(dim, mean=1.0, std=0.2) if case["post_weight"] else None
    mod = normal(groups, 6, dim, std=0.3)  # one table of six rows for a block, as its time embedding gives it
    s["t"] = mod[:, 0] if case["shift"] else None
    s["s"] = mod[:, 1] if case["scale"] else None
    s["g"] = mod[:, 2] if case["gate"] else None
    if case["back"]:
        s["dx"] = normal(rows, dim, dtype=xt) if case["op"] != "norm" else None
        s["dh"] = normal(rows, dim, dtype=bt) if case["op"] != "gate" else None
    return s


def work(case):
    if case["op"] == "qk":
        n = case["rows"] * (case["q_heads"] + case["k_heads"]) * case["d"]
        size = 2 if case["dtype"] == "bf16" else 4
        streams = 2 if not case["back"] or case["norm"] == "none" else 3
        extra = case["rows"] * 12 if case["explicit"] else 0
        return {"bytes": float(n * size * streams + extra), "flops": float(n * (20 if case["back"] else 10))}
    ex, eb = (2 if case[k] == "bf16" else 4 for k in ("x", "branch"))
    streams = {("norm", False): ex + eb, ("norm", True): 2 * ex + eb, ("gate", False): 2 * ex + eb, ("gate", True): ex + 2 * eb,
               ("gate_norm", False): 2 * ex + 2 * eb, ("gate_norm", True): 3 * ex + 3 * eb}[(case["op"], case["back"])]
    n = case["rows"] * case["dim"]
    mods = sum(case[k] for k in ("scale", "shift", "gate"))
    small = case["dim"] * 4 * (mods * case["groups"] + sum(case[k] for k in ("weight", "bias", "post_weight")))
    return {"bytes": float(n * streams + small * (2 if case["back"] else 1)), "flops": float(n * (40 if case["back"] else 15))}


# ------------------------------------------------------------ plain forms --
def _positions(c, pos):
    if pos is not None:
        return pos.double(), None
    tok = torch.arange(c["rows"], device="cuda") + c["offset"]
    p = torch.stack([tok // (c["H"] * c["W"]), tok // c["W"] % c["H"], tok % c["W"]], dim=1).double()
    return p, torch.arange(c["rows"], device="cuda") >= c["rows"] - c["text"]


def _cos_sin(c, pos):
    p, text = _positions(c, pos)
    ladder = [torch.arange(n, dtype=torch.float64, device="cuda") / max(n, 1) for n in (c["pt"], c["py"], c["px"])]
    freq = torch.pow(torch.tensor(c["theta"], dtype=torch.float64, device="cuda"), -torch.cat(ladder))
    axis = torch.repeat_interleave(torch.arange(3, device="cuda"), torch.tensor([c["pt"], c["py"], c["px"]], device="cuda"))
    a = p[:, axis] * freq
    if text is not None:
        a = torch.where(text[:, None], torch.zeros_like(a), a)
    return torch.cos(a).float()[:, None, :], torch.sin(a).float()[:, None, :]


def _split(x, style):
    return (x[..., 0::2], x[..., 1::2]) if style == "interleaved" else (x[..., : x.shape[-1] // 2], x[..., x.shape[-1] // 2:])


def _join(a, b, style):
    return torch.stack([a, b], dim=-1).flatten(-2) if style == "interleaved" else torch.cat([a, b], dim=-1)


def _qk_forward(c, x, w, cos, sin):
    n = x.float()
    if c["norm"] != "none":
        over = (1, 2) if c["norm"] == "token" else (2,)
        n = n * torch.rsqrt((n * n).mean(over, keepdim=True) + EPS) * w.view(-1, c["d"])
    a, b = _split(n, c["style"])
    return _join(a * cos - b * sin, a * sin + b * cos, c["style"]).to(x.dtype)


def _qk_backward(c, g, x, w, cos, sin):
    a, b = _split(g.float(), c["style"])
    u = _join(a * cos + b * sin, b * cos - a * sin, c["style"])
    if c["norm"] == "none":
        return u.to(g.dtype), None
    over = (1, 2) if c["norm"] == "token" else (2,)
    n = x.float()
    r = torch.rsqrt((n * n).mean(over, keepdim=True) + EPS)
    n = n * r
    dw = (u * n).sum((0,) if c["norm"] == "token" else (0, 1), dtype=torch.float64).float().flatten()
    u = u * w.view(-1, c["d"])
    return (r * (u - n * (u * n).mean(over, keepdim=True))).to(g.dtype), dw


def _hat(x, kind):
    """The normalised rows and what they were scaled by."""
    x = x - x.mean(1, keepdim=True) if kind == "layer" else x
    r = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    return x * r, r


def _hat_backward(u, hat, r, kind):
    u = u - hat * (u * hat).mean(1, keepdim=True)
    return r * (u - u.mean(1, keepdim=True)) if kind == "layer" else r * u


def _wide(m, c):
    return m if c["groups"] in (1, c["rows"]) else m.repeat_interleave(c["rows"] // c["groups"], dim=0)


def _by_group(x, c):
    return x.view(c["groups"], -1, c["dim"]).sum(1, dtype=torch.float64).float()


def _join_branch(s, c):
    y = s["ys"].float()
    y = _hat(y, c["post"])[0] if c["post"] != "none" else y
    y = y * s["pw"] if s["pw"] is not None else y
    y = y * _wide(s["g"], c) if s["g"] is not None else y
    return s["xs"].float() + c["residual_scale"] * y


def _norm_forward(s, c, x):
    h = _hat(x, c["norm"])[0]
    h = h * s["w"] if s["w"] is not None else h
    h = h + s["b"] if s["b"] is not None else h
    h = h * (1 + _wide(s["s"], c)) if s["s"] is not None else h
    return h + _wide(s["t"], c) if s["t"] is not None else h


def _norm_backward(s, c, x):
    hat, r = _hat(x, c["norm"])
    dh = s["dh"].float()
    affine = hat * s["w"] if s["w"] is not None else hat
    affine = affine + s["b"] if s["b"] is not None else affine
    ds = _by_group(dh * affine, c) if s["s"] is not None else None
    dt = _by_group(dh, c) if s["t"] is not None else None
    u = dh * (1 + _wide(s["s"], c)) if s["s"] is not None else dh
    dw = (u * hat).sum(0, dtype=torch.float64).float() if s["w"] is not None else None
    db = u.sum(0, dtype=torch.float64).float() if s["b"] is not None else None
    u = u * s["w"] if s["w"] is not None else u
    return _hat_backward(u, hat, r, c["norm"]), dw, db, ds, dt


def _gate_backward(s, c, dx):
    v = s["ys"].float()
    r = None
    if c["post"] != "none":
        v, r = _hat(v, c["post"])
    affine = v * s["pw"] if s["pw"] is not None else v
    u = dx * c["residual_scale"]
    dg = _by_group(u * affine, c) if s["g"] is not None else None
    u = u * _wide(s["g"], c) if s["g"] is not None else u
    dpw = (u * v).sum(0, dtype=torch.float64).float() if s["pw"] is not None else None
    u = u * s["pw"] if s["pw"] is not None else u
    return (_hat_backward(u, v, r, c["post"]) if r is not None else u), dg, dpw


def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "qk":
        cos, sin = _cos_sin(c, s["pos"])
        if not c["back"]:
            return _qk_forward(c, s["q"], s["qw"], cos, sin), _qk_forward(c, s["k"], s["kw"], cos, sin)
        dq, dqw = _qk_backward(c, s["dq"], s["q"], s["qw"], cos, sin)
        dk, dkw = _qk_backward(c, s["dk"], s["k"], s["kw"], cos, sin)
        return (dq, dk) if dqw is None else (dq, dk, dqw, dkw)
    xt, bt = s["xs"].dtype, DTYPES[c["branch"]]
    if c["op"] == "norm":
        if not c["back"]:
            return _norm_forward(s, c, s["xs"].float()).to(bt)
        dx, *small = _norm_backward(s, c, s["xs"].float())
        return _given(dx.to(xt), *small)
    if c["op"] == "gate":
        if not c["back"]:
            return _join_branch(s, c).to(xt)
        dy, *small = _gate_backward(s, c, s["dx"].float())
        return _given(dy.to(bt), *small)
    x = _join_branch(s, c)
    if not c["back"]:
        return x.to(xt), _norm_forward(s, c, x).to(bt)
    dx, *small = _norm_backward(s, c, x)
    dx = dx + s["dx"].float()
    dy, *more = _gate_backward(s, c, dx)
    return _given(dx.to(xt), dy.to(bt), *small, *more)


def _given(*outputs):
    return tuple(filter(lambda t: t is not None, outputs))


# --------------------------------------------------- the framework's calls --
@functools.lru_cache(maxsize=None)
def _rope(d, pairs, theta, style):
    from input_adaptive_block_b200 import api
    return api.rope_axes(d, pairs, theta=theta, style=style)


def _run_own(s, c):
    from input_adaptive_block_b200 import api
    if c["op"] == "qk":
        rope = _rope(c["d"], (c["pt"], c["py"], c["px"]), c["theta"], c["style"])
        where = {"positions": s["pos"]} if c["explicit"] else {"grid": (c["T"], c["H"], c["W"]), "token_offset": c["offset"],
                                                              "text_tokens": c["text"]}
        norm = {"norm": c["norm"], "q_weight": s["qw"], "k_weight": s["kw"], "eps": EPS}
        if not c["back"]:
            return api.qk_norm_rope(s["q"], s["k"], rope, **where, **norm)
        g = api.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], rope, **where, **norm)
        return _given(g.q, g.k, g.q_weight, g.k_weight)
    pre = {"norm": c["norm"], "eps": EPS, "weight": s["w"], "bias": s["b"], "scale": s["s"], "shift": s["t"]}
    post = {"gate": s["g"], "post_norm": c["post"], "post_weight": s["pw"], "post_eps": EPS, "residual_scale": c["residual_scale"]}
    if c["op"] == "norm":
        if not c["back"]:
            return api.norm_modulate(s["xs"], out_dtype=DTYPES[c["branch"]], **pre)
        g = api.norm_modulate_backward(s["dh"], s["xs"], **pre)
        return _given(g.x, g.weight, g.bias, g.scale, g.shift)
    if c["op"] == "gate":
        if not c["back"]:
            return api.gate_residual(s["xs"], s["ys"], **post)
        g = api.gate_residual_backward(s["dx"], s["ys"], **post)
        return _given(g.y, g.gate, g.post_weight)
    if not c["back"]:
        return api.gate_residual_norm(s["xs"], s["ys"], **post, **pre)
    g = api.gate_residual_norm_backward(s["dx"], s["dh"], s["xs"], s["ys"], **post, **pre)
    return _given(g.x, g.y, g.weight, g.bias, g.scale, g.shift, g.gate, g.post_weight)


# ------------------------------------------------- the definition, 64 bits --
def _exact_turn(c, first, n, pos):
    """Unit complex numbers [n, 1, d/2] of rows first .. first + n."""
    if pos is None:
        tok = torch.arange(first, first + n, device="cuda") + c["offset"]
        x = tok.remainder(c["W"])
        y = ((tok - x) // c["W"]).remainder(c["H"])
        t = (tok - x - y * c["W"]) // (c["W"] * c["H"])
        live = (torch.arange(first, first + n, device="cuda") < c["rows"] - c["text"]).double()
    else:
        t, y, x = pos[first:first + n].unbind(1)
        live = torch.ones(n, dtype=torch.float64, device="cuda")
    parts = []
    for p, m in ((t, c["pt"]), (y, c["py"]), (x, c["px"])):
        f = torch.tensor([math.exp(-math.log(c["theta"]) * i / m) for i in range(m)], dtype=torch.float64, device="cuda")
        parts.append(torch.outer(p.double() * live, f))
    a = torch.cat(parts, 1)
    return torch.polar(torch.ones_like(a), a)[:, None]


def _exact_qk(c, x, w, turn):
    if c["norm"] != "none":
        flat = x.flatten(1) if c["norm"] == "token" else x
        flat = flat / (flat.square().sum(-1, keepdim=True) / flat.shape[-1] + EPS).sqrt()
        x = (flat * w).view(x.shape)
    n = x.shape[-1] // 2
    z = torch.complex(x[..., 0::2], x[..., 1::2]) if c["style"] == "interleaved" else torch.complex(x[..., :n], x[..., n:])
    z = z * turn
    return torch.view_as_real(z).flatten(-2) if c["style"] == "interleaved" else torch.cat([z.real, z.imag], -1)


def _exact_normed(x, kind):
    if kind == "none":
        return x
    if kind == "layer":
        return (x - x.mean(-1, keepdim=True)) / (x.var(-1, correction=0, keepdim=True) + EPS).sqrt()
    return x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()


def _exact_block(c, x, y, p, group):
    """The stream after the branch has joined it, and the norm that follows; p holds the weights and this row's modulation."""
    pick = lambda m: m[group]  # noqa: E731
    if y is not None:
        b = _exact_normed(y, c["post"])
        for name, m in (("pw", None), ("g", pick)):
            if p[name] is not None:
                b = b * (m(p[name]) if m else p[name])
        x = x + c["residual_scale"] * b
    if c["op"] == "gate":
        return x, None
    h = _exact_normed(x, c["norm"])
    h = h * p["w"] if p["w"] is not None else h
    h = h + p["b"] if p["b"] is not None else h
    h = h + h * pick(p["s"]) if p["s"] is not None else h
    return x, (h + pick(p["t"]) if p["t"] is not None else h)


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    double = lambda t: None if t is None else t.double().requires_grad_(c["back"])  # noqa: E731
    grad = torch.enable_grad if c["back"] else torch.no_grad
    if c["op"] == "qk":
        width = (c["q_heads"] + c["k_heads"]) * c["d"]
        step = max(1, 40_000_000 // width)
        qw, kw = double(s["qw"]), double(s["kw"])
        out = ([], [])
        with grad():
            for first in range(0, c["rows"], step):
                n = min(step, c["rows"] - first)
                turn = _exact_turn(c, first, n, s["pos"])
                for i, (name, w) in enumerate((("q", qw), ("k", kw))):
                    x = double(s[name][first:first + n])
                    y = _exact_qk(c, x, w, turn)
                    if c["back"]:
                        y.backward(s["d" + name][first:first + n].double())
                        y = x.grad
                    out[i].append(y.detach())
        both = (torch.cat(out[0]), torch.cat(out[1]))
        return both + ((qw.grad, kw.grad) if c["back"] and qw is not None else ())
    p = {k: double(s[k]) for k in ("w", "b", "s", "t", "g", "pw")}
    step = max(1, 40_000_000 // c["dim"])
    per = c["rows"] // c["groups"]
    xs, ys, hs = [], [], []
    with grad():
        for first in range(0, c["rows"], step):
            last = min(first + step, c["rows"])
            x, y = double(s["xs"][first:last]), double(s["ys"][first:last]) if s["ys"] is not None else None
            group = torch.arange(first, last, device="cuda") // per
            nx, h = _exact_block(c, x, y, p, group)
            if c["back"]:
                loss = 0.0
                if s["dx"] is not None:
                    loss = loss + (nx * s["dx"][first:last].double()).sum()
                if s["dh"] is not None:
                    loss = loss + (h * s["dh"][first:last].double()).sum()
                loss.backward()
                xs.append(x.grad)
                ys.append(y.grad if y is not None else None)
            else:
                xs.append(nx.detach())
                hs.append(h.detach() if h is not None else None)
    whole = lambda parts: torch.cat(parts) if parts and parts[0] is not None else None  # noqa: E731
    if not c["back"]:
        return whole(hs) if c["op"] == "norm" else whole(xs) if c["op"] == "gate" else (whole(xs), whole(hs))
    small = [None if t is None else t.grad for t in (p["w"], p["b"], p["s"], p["t"])]
    more = [None if t is None else t.grad for t in (p["g"], p["pw"])]
    if c["op"] == "norm":
        return _given(whole(xs), *small)
    if c["op"] == "gate":
        return _given(whole(ys), *more)
    return _given(whole(xs), whole(ys), *small, *more)
