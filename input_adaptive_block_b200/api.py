"""PyTorch-facing binding of the C ABI (argument marshalling only).

Every function here hands device pointers of caller tensors and the current
CUDA stream to the matching `spade_*` entry point of libspade.so; all
arithmetic happens in its CUDA kernels.  PyTorch provides memory and streams.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Optional, Sequence, Tuple

import torch

from . import _lib
from ._lib import (NORM, QK_NORM, ROPE_STYLE, ROW_PARAMS, SpadeGeom, SpadeHeadScheme, SpadeQkDesc, SpadeRope,
                   SpadeRowDesc, SpadeRowGrads, SpadeRowParams, check)

__all__ = [
    "geom", "dtype_code", "tile3d", "summarize", "summarize_qk", "estimate", "estimate_scores", "select", "select_scores",
    "attn_workspace_bytes",
    "block_sparse_attn", "block_sparse_attn_noalloc", "grouped_workspace_bytes", "grouped_attn", "grouped_head_lists",
    "last_device_status", "selftest_bounded_wait", "num_blocks", "sics_workspace_bytes", "sics", "select_window",
    "grouped_attn_from_host", "grouped_host_workspace_bytes", "grouped_attn_lists",
    "rope_axes", "qk_norm_rope", "qk_norm_rope_backward", "qk_norm_rope_workspace_bytes", "QkGrads",
    "norm_modulate", "norm_modulate_backward", "gate_residual", "gate_residual_backward", "gate_residual_norm",
    "gate_residual_norm_backward", "row_workspace_bytes", "RowGrads",
]


def geom(g) -> SpadeGeom:
    """(T, H, W, bt, bh, bw) tuple, Scheme, or SpadeGeom -> SpadeGeom."""
    if isinstance(g, SpadeGeom):
        return g
    t = g.as_tuple() if hasattr(g, "as_tuple") else tuple(g)
    return SpadeGeom(*[int(v) for v in t])


def num_blocks(g) -> int:
    gg = geom(g)
    return -(-gg.T // gg.bt) * -(-gg.H // gg.bh) * -(-gg.W // gg.bw)


def dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float32:
        return _lib.SPADE_F32
    if dt == torch.bfloat16:
        return _lib.SPADE_BF16
    raise TypeError(f"unsupported dtype {dt}")


def _stream(stream: Optional[torch.cuda.Stream]) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _dev(t: torch.Tensor, name: str) -> int:
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    return t.data_ptr()


def tile3d(x: torch.Tensor, g, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    gg = geom(g)
    heads, d = x.shape[1], x.shape[2]
    nb, bs = num_blocks(gg), gg.bt * gg.bh * gg.bw
    if out is None:
        out = torch.empty(heads, nb, bs, d, dtype=x.dtype, device=x.device)
    check(_lib.load().spade_tile3d(_dev(x, "x"), _dev(out, "xt"), gg, heads, d, dtype_code(x.dtype),
                                   _stream(stream)), "spade_tile3d")
    return out


SUMMARY = {"mean": 0, "max": 1, "min": 2}


def summarize(x: torch.Tensor, g, out: Optional[torch.Tensor] = None, stream=None,
              mode: str = "mean") -> torch.Tensor:
    """Block summaries [heads, nb, d] float32: mean (default), max or min
    over each block's valid tokens."""
    gg = geom(g)
    heads, d = x.shape[1], x.shape[2]
    if out is None:
        out = torch.empty(heads, num_blocks(gg), d, dtype=torch.float32, device=x.device)
    if mode == "mean":
        check(_lib.load().spade_summarize(_dev(x, "x"), _dev(out, "xmean"), gg, heads, d, dtype_code(x.dtype),
                                          _stream(stream)), "spade_summarize")
    else:
        check(_lib.load().spade_summarize_mode(_dev(x, "x"), _dev(out, "out"), gg, heads, d, dtype_code(x.dtype),
                                               SUMMARY[mode], _stream(stream)), "spade_summarize_mode")
    return out


def summarize_qk(q: torch.Tensor, k: torch.Tensor, g, qout: Optional[torch.Tensor] = None,
                 kout: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Block means of Q and of K in one launch."""
    gg = geom(g)
    heads, d = q.shape[1], q.shape[2]
    if k.shape[1:] != q.shape[1:] or k.dtype != q.dtype:
        raise ValueError("q and k must have the same heads, d and dtype")
    nb = num_blocks(gg)
    if qout is None:
        qout = torch.empty(heads, nb, d, dtype=torch.float32, device=q.device)
    if kout is None:
        kout = torch.empty(heads, nb, d, dtype=torch.float32, device=q.device)
    check(_lib.load().spade_summarize_qk(_dev(q, "q"), _dev(k, "k"), _dev(qout, "qmean"), _dev(kout, "kmean"),
                                         gg, heads, d, dtype_code(q.dtype), _stream(stream)), "spade_summarize_qk")
    return qout, kout


def estimate(qmean: torch.Tensor, kmean: torch.Tensor, out: Optional[torch.Tensor] = None,
             stream=None) -> torch.Tensor:
    heads, nb, d = qmean.shape
    if out is None:
        out = torch.empty(heads, nb, nb, dtype=torch.float32, device=qmean.device)
    check(_lib.load().spade_estimate(_dev(qmean, "qmean"), _dev(kmean, "kmean"), _dev(out, "prob"),
                                     heads, nb, d, _stream(stream)), "spade_estimate")
    return out


def estimate_scores(qmean: torch.Tensor, kmean: torch.Tensor, out: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """The Estimator's pooled scores Qbar . Kbar^T / sqrt(d) (no softmax)."""
    heads, nb, d = qmean.shape
    if out is None:
        out = torch.empty(heads, nb, nb, dtype=torch.float32, device=qmean.device)
    check(_lib.load().spade_estimate_scores(_dev(qmean, "qmean"), _dev(kmean, "kmean"), _dev(out, "scores"),
                                            heads, nb, d, _stream(stream)), "spade_estimate_scores")
    return out


def _select(fn_name: str, x: torch.Tensor, taus: Sequence[float], cnt, idx, stream):
    heads, nb, _ = x.shape
    if cnt is None:
        cnt = torch.empty(heads, nb, dtype=torch.int32, device=x.device)
    if idx is None:
        idx = torch.full((heads, nb, nb), -1, dtype=torch.int32, device=x.device)
    tau_arr = (ctypes.c_float * heads)(*[float(t) for t in taus])
    check(getattr(_lib.load(), fn_name)(_dev(x, "input"), tau_arr, _dev(cnt, "cnt"), _dev(idx, "idx"),
                                        heads, nb, _stream(stream)), fn_name)
    return cnt, idx


def select(prob: torch.Tensor, taus: Sequence[float], cnt: Optional[torch.Tensor] = None,
           idx: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    return _select("spade_select", prob, taus, cnt, idx, stream)


def select_scores(scores: torch.Tensor, taus: Sequence[float], cnt: Optional[torch.Tensor] = None,
                  idx: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Softmax of each score row fused with the index search."""
    return _select("spade_select_scores", scores, taus, cnt, idx, stream)


def select_window(prob: torch.Tensor, taus: Sequence[float], radius, g, cnt: Optional[torch.Tensor] = None,
                  idx: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Selection with a static window per head: radius = (rt, ry, rx) for
    every head, or one such triple per head."""
    heads, nb, _ = prob.shape
    if cnt is None:
        cnt = torch.empty(heads, nb, dtype=torch.int32, device=prob.device)
    if idx is None:
        idx = torch.full((heads, nb, nb), -1, dtype=torch.int32, device=prob.device)
    rad = list(radius) if len(radius) == heads and hasattr(radius[0], "__len__") else [tuple(radius)] * heads
    rad_arr = (ctypes.c_int * (3 * heads))(*[int(r) for t in rad for r in t])
    tau_arr = (ctypes.c_float * heads)(*[float(t) for t in taus])
    check(_lib.load().spade_select_window(_dev(prob, "prob"), tau_arr, rad_arr, geom(g), _dev(cnt, "cnt"),
                                          _dev(idx, "idx"), heads, _stream(stream)), "spade_select_window")
    return cnt, idx


def attn_workspace_bytes(g, heads: int, d: int, text_tokens: int = 0) -> int:
    return int(_lib.load().spade_attn_workspace_bytes(geom(g), heads, d, text_tokens))


def block_sparse_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cnt: Optional[torch.Tensor],
                      idx: Optional[torch.Tensor], g, text_tokens: int = 0, out: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    gg = geom(g)
    heads, d = q.shape[1], q.shape[2]
    if out is None:
        out = torch.empty_like(q)
    need = attn_workspace_bytes(gg, heads, d, text_tokens)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    cp = _dev(cnt, "cnt") if cnt is not None else None
    ip = _dev(idx, "idx") if idx is not None else None
    check(_lib.load().spade_block_sparse_attn(
        _dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(out, "out"), cp, ip, gg, heads, d, text_tokens,
        dtype_code(q.dtype), _dev(workspace, "workspace"), workspace.numel(), _stream(stream)),
        "spade_block_sparse_attn")
    return out


def block_sparse_attn_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cnt: Optional[torch.Tensor],
                              idx: Optional[torch.Tensor], g, text_tokens: int = 0,
                              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """spade_block_sparse_attn without a workspace argument: the library keeps
    the scratch in a fixed device array of its own (see include/spade.h for
    the size limit and the rule that overlapping calls must be ordered)."""
    gg = geom(g)
    heads, d = q.shape[1], q.shape[2]
    if out is None:
        out = torch.empty_like(q)
    cp = _dev(cnt, "cnt") if cnt is not None else None
    ip = _dev(idx, "idx") if idx is not None else None
    check(_lib.load().spade_block_sparse_attn_noalloc(
        _dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(out, "out"), cp, ip, gg, heads, d, text_tokens,
        dtype_code(q.dtype), _stream(stream)), "spade_block_sparse_attn_noalloc")
    return out


def _tables(schemes, table):
    gs = (SpadeGeom * len(schemes))(*[geom(s) for s in schemes])
    rows = (SpadeHeadScheme * len(table))(*[SpadeHeadScheme(int(sc), float(tau), int(bool(dn)))
                                            for sc, tau, dn in table])
    return gs, rows


def grouped_workspace_bytes(schemes, table, d: int, text_tokens: int = 0) -> int:
    gs, rows = _tables(schemes, table)
    return int(_lib.load().spade_grouped_workspace_bytes(gs, len(schemes), rows, len(table), d, text_tokens))


def grouped_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, schemes, table, text_tokens: int = 0,
                 out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                 stream=None, summary=("mean", "mean"), window=None) -> torch.Tensor:
    """table: per head (scheme index, tau, dense); summary: the Q and K
    Summarizer reduces ("mean", "max" or "min"); window: optional static
    window block radii (rt, ry, rx) per head."""
    heads, d = q.shape[1], q.shape[2]
    gs, rows = _tables(schemes, table)
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        need = int(_lib.load().spade_grouped_workspace_bytes(gs, len(schemes), rows, heads, d, text_tokens))
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    if tuple(summary) == ("mean", "mean") and window is None:
        check(_lib.load().spade_grouped_attn(
            _dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(out, "out"), gs, len(schemes), rows, heads, d,
            text_tokens, dtype_code(q.dtype), _dev(workspace, "workspace"), workspace.numel(), _stream(stream)),
            "spade_grouped_attn")
    else:
        check(_lib.load().spade_grouped_attn_ex(
            _dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(out, "out"), gs, len(schemes), rows, heads, d,
            text_tokens, dtype_code(q.dtype), SUMMARY[summary[0]], SUMMARY[summary[1]],
            (ctypes.c_int * (3 * heads))(*[int(r) for t in window for r in t]) if window is not None else None,
            _dev(workspace, "workspace"), workspace.numel(), _stream(stream)), "spade_grouped_attn_ex")
    return out


def grouped_attn_lists(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, schemes, table, workspace: torch.Tensor,
                       text_tokens: int = 0, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Step 5 of a grouped layer under the kept lists an earlier grouped_attn
    call left in `workspace` (same schemes, table, d, text_tokens)."""
    heads, d = q.shape[1], q.shape[2]
    gs, rows = _tables(schemes, table)
    if out is None:
        out = torch.empty_like(q)
    check(_lib.load().spade_grouped_attn_lists(
        _dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(out, "out"), gs, len(schemes), rows, heads, d, text_tokens,
        dtype_code(q.dtype), _dev(workspace, "workspace"), workspace.numel(), _stream(stream)),
        "spade_grouped_attn_lists")
    return out


def grouped_host_workspace_bytes(schemes, table, d: int, text_tokens: int = 0, dtype=torch.bfloat16,
                                 head_chunk: int = 2) -> int:
    gs, rows = _tables(schemes, table)
    return int(_lib.load().spade_grouped_host_workspace_bytes(gs, len(schemes), rows, len(table), d, text_tokens,
                                                              dtype_code(dtype), head_chunk))


def grouped_attn_from_host(qh: torch.Tensor, kh: torch.Tensor, vh: torch.Tensor, out_h: torch.Tensor, schemes,
                           table, text_tokens: int = 0, head_chunk: int = 2,
                           workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One layer from host memory to host memory (spade_grouped_attn_host):
    qh, kh, vh, out_h are host tensors [N (+text), heads, d], pinned for the
    copies to overlap the compute; the library streams the layer through the
    GPU in groups of head_chunk heads.  workspace: a device uint8 tensor of
    grouped_host_workspace_bytes (allocated here when omitted).  Returns
    out_h once the work is enqueued; it is complete when the current stream
    (or `stream`) is."""
    for t, name in ((qh, "q"), (kh, "k"), (vh, "v"), (out_h, "out")):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous host tensor")
    heads, d = qh.shape[1], qh.shape[2]
    gs, rows = _tables(schemes, table)
    if workspace is None:
        need = grouped_host_workspace_bytes(schemes, table, d, text_tokens, qh.dtype, head_chunk)
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    check(_lib.load().spade_grouped_attn_host(
        qh.data_ptr(), kh.data_ptr(), vh.data_ptr(), out_h.data_ptr(), gs, len(schemes), rows, heads, d,
        text_tokens, dtype_code(qh.dtype), head_chunk, _dev(workspace, "workspace"), workspace.numel(),
        _stream(stream)), "spade_grouped_attn_host")
    return out_h


def grouped_head_lists(schemes, table, d: int, text_tokens: int, head: int) -> Tuple[int, int]:
    """Byte offsets of head's (cnt, idx) inside a grouped workspace; (-1, -1) for dense heads."""
    gs, rows = _tables(schemes, table)
    co, io = ctypes.c_int64(), ctypes.c_int64()
    check(_lib.load().spade_grouped_head_lists(gs, len(schemes), rows, len(table), d, text_tokens, head,
                                               ctypes.byref(co), ctypes.byref(io)), "spade_grouped_head_lists")
    return co.value, io.value


def sics_workspace_bytes(candidates, heads: int) -> int:
    gs = (SpadeGeom * len(candidates))(*[geom(c) for c in candidates])
    return int(_lib.load().spade_sics_workspace_bytes(gs, len(candidates), heads))


def sics(q: torch.Tensor, k: torch.Tensor, candidates, workspace: Optional[torch.Tensor] = None,
         stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Scheme generation: per head, the SICS of every candidate blocking
    scheme (Q plus K) and the index of the best one.  Returns (scores
    [heads, n_candidates] float32, choice [heads] int32), both on the device."""
    heads, d = q.shape[1], q.shape[2]
    gs = (SpadeGeom * len(candidates))(*[geom(c) for c in candidates])
    scores = torch.empty(heads, len(candidates), dtype=torch.float32, device=q.device)
    choice = torch.empty(heads, dtype=torch.int32, device=q.device)
    if workspace is None:
        need = int(_lib.load().spade_sics_workspace_bytes(gs, len(candidates), heads))
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    check(_lib.load().spade_sics(_dev(q, "q"), _dev(k, "k"), gs, len(candidates), heads, d, dtype_code(q.dtype),
                                 _dev(scores, "scores"), _dev(choice, "choice"), _dev(workspace, "workspace"),
                                 workspace.numel(), _stream(stream)), "spade_sics")
    return scores, choice


# ---- row passes around the attention ----------------------------------------
# Plain calls on plain tensors: autograd records none of them, the _backward
# calls are its counterpart.
def _fits(bits: int, *numbers: int) -> None:
    """ctypes cuts what a field cannot hold to its low bits without a word."""
    top = 1 << (bits - 1)
    for n in numbers:
        if not -top <= n < top:
            raise ValueError(f"{n} does not fit {bits} bits")


def rope_axes(d: int, pairs: Sequence[int], theta=10000.0, scale=1.0, style: str = "interleaved",
              shared_ladder: bool = False) -> SpadeRope:
    """The rotation of heads of d channels over the axes (t, y, x): pairs[a]
    pairs turn with axis a, at frequencies scale[a] * theta[a]^(-i / pairs[a])
    (theta, scale: one number or one per axis), or down one ladder over all
    pairs (shared_ladder).  style: "interleaved" pairs channels 2i, 2i + 1;
    "half" pairs i, i + d / 2.  A plan: make it once, pass it to every call."""
    per_axis = lambda v: [float(x) for x in v] if hasattr(v, "__len__") else [float(v)] * 3  # noqa: E731
    th, sc = per_axis(theta), per_axis(scale)
    if len(pairs) != 3 or len(th) != 3 or len(sc) != 3:
        raise ValueError("pairs, theta and scale have one entry per axis (t, y, x)")
    if 2 * sum(int(p) for p in pairs) > d:
        raise ValueError(f"{sum(pairs)} pairs in heads of {d} channels")
    _fits(32, *(int(p) for p in pairs))
    rope = SpadeRope()
    check(_lib.load().spade_rope_axes(ctypes.byref(rope), (ctypes.c_int32 * 3)(*[int(p) for p in pairs]),
                                      (ctypes.c_double * 3)(*th), (ctypes.c_double * 3)(*sc),
                                      _code(ROPE_STYLE, style, "style"),
                                      int(bool(shared_ladder))), "spade_rope_axes")
    return rope


class QkGrads(NamedTuple):
    """Gradients of qk_norm_rope: of its inputs, and of the weights given."""
    q: Optional[torch.Tensor]
    k: Optional[torch.Tensor]
    q_weight: Optional[torch.Tensor]
    k_weight: Optional[torch.Tensor]


class RowGrads(NamedTuple):
    """Gradients of a row pass: of its inputs, and of the parameters given."""
    x: Optional[torch.Tensor]
    y: Optional[torch.Tensor]
    weight: Optional[torch.Tensor]
    bias: Optional[torch.Tensor]
    scale: Optional[torch.Tensor]
    shift: Optional[torch.Tensor]
    gate: Optional[torch.Tensor]
    post_weight: Optional[torch.Tensor]


class _On:
    """Makes `like`'s device and, when given, `stream` current for a call, so
    that what it allocates belongs to the stream it runs on."""
    __slots__ = ("ctx", "device")

    def __init__(self, like: torch.Tensor, stream):
        self.ctx, self.device = None, like.get_device()
        if stream is not None:
            if stream.device != like.device:
                raise ValueError(f"stream of {stream.device} for tensors of {like.device}")
            self.ctx = torch.cuda.stream(stream)
        elif torch.cuda.current_device() != self.device:
            self.ctx = torch.cuda.device(self.device)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        return torch._C._cuda_getCurrentRawStream(self.device)

    def __exit__(self, *exc):
        return self.ctx.__exit__(*exc) if self.ctx is not None else None


def _on_gpu(t: torch.Tensor, name: str, like: torch.Tensor) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, not on {like.device}")


def _new(like: torch.Tensor, shape, dtype) -> torch.Tensor:
    """A packed tensor on like's device."""
    if like.dtype is dtype and like.shape == shape and like.is_contiguous():
        return torch.empty_like(like)
    return torch.empty(shape, dtype=dtype, device=like.device)


def _strided(t: Optional[torch.Tensor], name: str, like: torch.Tensor, shape, dtype) -> Tuple[Optional[int], int]:
    """(pointer, row stride) of a tensor of rows [rows, ...] whose rows are
    packed inside and may lie any distance apart."""
    if t is None:
        return None, 0
    if t.dtype is dtype and t.shape == shape and t.is_contiguous():
        if t is like or (t.is_cuda and t.get_device() == like.get_device()):      # like is on a GPU
            return t.data_ptr(), 0
    _on_gpu(t, name, like)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, not {dtype}")
    inner = 1
    for size, stride in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if size != 1 and stride != inner:
            raise ValueError(f"the rows of {name} must be contiguous")
        inner *= size
    if t.shape[0] <= 1 or inner == 0:
        return t.data_ptr(), 0
    if t.stride(0) < inner:
        raise ValueError(f"the rows of {name} overlap")
    return t.data_ptr(), t.stride(0)


def _output(t: Optional[torch.Tensor], name: str, like: torch.Tensor, shape, dtype):
    """(tensor, pointer, row stride) of an output: a new packed one where none
    is given."""
    if t is None:
        t = _new(like, shape, dtype)
        return t, t.data_ptr(), 0
    return (t, *_strided(t, name, like, shape, dtype))


def _vector(t: Optional[torch.Tensor], name: str, like: torch.Tensor, n: int, dtype) -> Optional[int]:
    if t is None:
        return None
    if t.dtype is dtype and t.is_contiguous() and t.numel() == n and t.is_cuda and t.get_device() == like.get_device():
        return t.data_ptr()
    _on_gpu(t, name, like)
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be {n} contiguous elements")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, not {dtype}")
    return t.data_ptr()


def _param_dtype(params) -> torch.dtype:
    dt = None
    for t in params:
        if t is not None and t.dtype is not dt:
            if dt is not None:
                raise TypeError(f"parameters of several dtypes: {dt}, {t.dtype}")
            dt = t.dtype
    return dt or torch.float32


def _scratch(workspace, need: int, like: torch.Tensor) -> Tuple[Optional[int], int, Optional[torch.Tensor]]:
    """(pointer, bytes, tensor) of the caller's workspace or of a new one."""
    if workspace is None:
        if not need:
            return None, 0, None
        workspace = torch.empty(need, dtype=torch.uint8, device=like.device)
        return workspace.data_ptr(), need, workspace
    _on_gpu(workspace, "workspace", like)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


@functools.lru_cache(maxsize=1024)
def _row_plan_bytes(device: int, rows: int, dim: int, groups: int) -> int:
    """Of sizes and the current device alone, which is `device`."""
    desc = SpadeRowDesc(rows=rows, groups=groups, dim=dim)
    return int(_lib.load().spade_row_bwd_workspace_bytes(ctypes.byref(desc)))


def _row_scratch_bytes(like: torch.Tensor, desc: SpadeRowDesc, given) -> int:
    """Of a backward row pass on like's device: none without a parameter."""
    for t in given.values():
        if t is not None:
            return _row_plan_bytes(like.get_device(), desc.rows, desc.dim, desc.groups)
    return 0


@functools.lru_cache(maxsize=1024)
def _qk_scratch_bytes(device: int, rows: int, q_heads: int, k_heads: int, d: int, norm: int) -> int:
    desc = SpadeQkDesc(rows=rows, q_heads=q_heads, k_heads=k_heads, d=d, norm=norm)
    return int(_lib.load().spade_qk_norm_rope_bwd_workspace_bytes(ctypes.byref(desc)))


def _code(table, key, name: str) -> int:
    if key not in table:
        raise ValueError(f"{name}={key!r} (one of {', '.join(table)})")
    return table[key]


def _qk_desc(q, k, q_weight, k_weight, grid, positions, token_offset, text_tokens, norm, eps):
    like = q if q is not None else k
    if like is None:
        raise ValueError("neither q nor k")
    _on_gpu(like, "q" if q is not None else "k", like)
    if like.dim() != 3 or (k is not None and (k.dim() != 3 or k.shape[0] != like.shape[0] or k.shape[2] != like.shape[2])):
        raise ValueError("q and k are [rows, heads, d]")
    rows, _, d = like.shape
    q_heads, k_heads = 0 if q is None else q.shape[1], 0 if k is None else k.shape[1]
    text_tokens, token_offset = int(text_tokens), int(token_offset)
    if (q_heads | k_heads | d) >> 31 or (text_tokens | token_offset) >> 63:
        _fits(32, q_heads, k_heads, d)
        _fits(64, text_tokens, token_offset)
    wdt = _param_dtype((q_weight, k_weight))
    desc = SpadeQkDesc(rows, text_tokens, token_offset, 0, 0, 0, q_heads, k_heads, d, dtype_code(like.dtype), dtype_code(wdt),
                       _code(QK_NORM, norm, "norm"), eps)
    pos = None
    if positions is not None:
        if grid is not None or token_offset:
            raise ValueError("positions and a grid")
        if positions.dtype != torch.int32:
            raise TypeError(f"positions has dtype {positions.dtype}, not torch.int32")
        if tuple(positions.shape) != (rows, 3) or not positions.is_contiguous():
            raise ValueError(f"positions must be contiguous [{rows}, 3]")
        _on_gpu(positions, "positions", like)
        pos = positions.data_ptr()
    elif grid is not None:
        g = grid if isinstance(grid, SpadeGeom) else None
        t = (g.T, g.H, g.W) if g is not None else (grid.as_tuple() if hasattr(grid, "as_tuple") else tuple(grid))
        T, H, W = int(t[0]), int(t[1]), int(t[2])
        if (T | H | W) >> 31:
            _fits(32, T, H, W)
        desc.T, desc.H, desc.W = T, H, W
    elif rows > text_tokens:
        raise ValueError("neither positions nor a grid")
    per = lambda t: 0 if t is None else (t.shape[1] * d if norm == "token" else d)  # noqa: E731
    weights = (_vector(q_weight, "q_weight", like, per(q), wdt), _vector(k_weight, "k_weight", like, per(k), wdt))
    return desc, like, pos, weights


def qk_norm_rope(q: Optional[torch.Tensor], k: Optional[torch.Tensor], rope: SpadeRope, grid=None,
                 positions: Optional[torch.Tensor] = None, token_offset: int = 0, text_tokens: int = 0,
                 norm: str = "none", q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, q_out: Optional[torch.Tensor] = None,
                 k_out: Optional[torch.Tensor] = None, stream=None):
    """Q and K ready for the attention, in one pass: rms norm (norm "token":
    over heads * d, "head": over d, "none") times weight, then the rotation.

    q [rows, q_heads, d], k [rows, k_heads, d] (either may be None); rows may
    lie apart, as in slices of one QKV projection.  Row r stands at token
    token_offset + r of grid (T, H, W) (a blocking scheme does too), its last
    text_tokens rows are text and not rotated; or at positions[r] (int32
    [rows, 3], t y x).  q_out / k_out: where the results go (q and k
    themselves are allowed), packed tensors by default.  Returns (q_out,
    k_out).  Plain results: autograd records nothing, whatever the inputs
    require; qk_norm_rope_backward gives the gradients."""
    desc, like, pos, (qw, kw) = _qk_desc(q, k, q_weight, k_weight, grid, positions, token_offset, text_tokens, norm, eps)
    with _On(like, stream) as s:
        dt, qo, ko = like.dtype, None, None
        qp, desc.q_stride = _strided(q, "q", like, None if q is None else q.shape, dt)
        kp, desc.k_stride = _strided(k, "k", like, None if k is None else k.shape, dt)
        if q is not None:
            q_out, qo, desc.q_out_stride = _output(q_out, "q_out", q, q.shape, dt)
        if k is not None:
            k_out, ko, desc.k_out_stride = _output(k_out, "k_out", k, k.shape, dt)
        check(_lib.load().spade_qk_norm_rope(ctypes.byref(desc), ctypes.byref(rope), pos, qp, kp, qw, kw, qo, ko, s),
              "spade_qk_norm_rope")
    return (q_out if q is not None else None), (k_out if k is not None else None)


def qk_norm_rope_workspace_bytes(rows: int, q_heads: int, k_heads: int, d: int, norm: str) -> int:
    """Scratch of qk_norm_rope_backward on the current device."""
    _fits(64, rows)
    _fits(32, q_heads, k_heads, d)
    desc = SpadeQkDesc(rows=rows, q_heads=q_heads, k_heads=k_heads, d=d, norm=_code(QK_NORM, norm, "norm"))
    return int(_lib.load().spade_qk_norm_rope_bwd_workspace_bytes(ctypes.byref(desc)))


def qk_norm_rope_backward(dq_out: Optional[torch.Tensor], dk_out: Optional[torch.Tensor], q: Optional[torch.Tensor],
                          k: Optional[torch.Tensor], rope: SpadeRope, grid=None,
                          positions: Optional[torch.Tensor] = None, token_offset: int = 0, text_tokens: int = 0,
                          norm: str = "none", q_weight: Optional[torch.Tensor] = None,
                          k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                          dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None) -> QkGrads:
    """Gradients of qk_norm_rope's inputs and of the weights given (float32),
    from those of its results.  q and k are that call's inputs (with norm
    "none" they may be None).  dq / dk: where the gradients go (dq_out and
    dk_out themselves are allowed)."""
    desc, like, pos, (qw, kw) = _qk_desc(dq_out, dk_out, q_weight, k_weight, grid, positions, token_offset, text_tokens,
                                         norm, eps)
    with _On(like, stream) as s:
        rows, d, dt = desc.rows, desc.d, like.dtype
        qs, ks = (rows, desc.q_heads, d), (rows, desc.k_heads, d)
        qo, ko = None, None
        gq, desc.q_dout_stride = _strided(dq_out, "dq_out", like, qs, dt)
        gk, desc.k_dout_stride = _strided(dk_out, "dk_out", like, ks, dt)
        normed = norm != "none"
        qp, desc.q_stride = _strided(q if normed and dq_out is not None else None, "q", like, qs, dt)
        kp, desc.k_stride = _strided(k if normed and dk_out is not None else None, "k", like, ks, dt)
        if dq_out is not None:
            dq, qo, desc.q_out_stride = _output(dq, "dq", dq_out, qs, dt)
        if dk_out is not None:
            dk, ko, desc.k_out_stride = _output(dk, "dk", dk_out, ks, dt)
        dqw, dkw = (None if w is None else _new(w, w.shape, torch.float32) for w in (q_weight, k_weight))
        lib = _lib.load()
        need = 0
        if dqw is not None or dkw is not None:
            need = _qk_scratch_bytes(like.get_device(), rows, desc.q_heads, desc.k_heads, d, desc.norm)
        wp, wn, workspace = _scratch(workspace, need, like)
        check(lib.spade_qk_norm_rope_bwd(ctypes.byref(desc), ctypes.byref(rope), pos, gq, gk, qp, kp, qw, kw, qo, ko,
                                         dqw.data_ptr() if dqw is not None else None,
                                         dkw.data_ptr() if dkw is not None else None, wp, wn, s),
              "spade_qk_norm_rope_bwd")
    return QkGrads(dq if dq_out is not None else None, dk if dk_out is not None else None, dqw, dkw)


_PER_GROUP = frozenset(("gate", "scale", "shift"))


def _row_call(like, x_dtype, branch_dtype, norm="none", eps=0.0, post_norm="none", post_eps=0.0, residual_scale=1.0,
              gate=None, post_weight=None, weight=None, bias=None, scale=None, shift=None):
    """Descriptor and parameters of a row pass over `like` [rows, dim]."""
    _on_gpu(like, "x", like)
    if like.dim() != 2:
        raise ValueError("rows are [rows, dim]")
    rows, dim = like.shape
    if dim >> 31:
        _fits(32, dim)
    params, strides, groups = SpadeRowParams(), None, None
    given = {"gate": gate, "post_weight": post_weight, "weight": weight, "bias": bias, "scale": scale, "shift": shift}
    pdt = _param_dtype(given.values())
    for name, t in given.items():
        if t is None:
            continue
        if name in _PER_GROUP:
            if t.dim() not in (1, 2) or t.shape[-1] != dim:
                raise ValueError(f"{name} must be [groups, {dim}] or [{dim}]")
            g = t.shape[0] if t.dim() == 2 else 1
            if groups is not None and groups != g:
                raise ValueError("gate, scale and shift must have one number of groups")
            groups = g
            p, stride = _strided(t if t.dim() == 2 else t.unsqueeze(0), name, like, (g, dim), pdt)
            if not g:
                p = None
            if stride:
                strides = strides or {}
                strides[name] = stride
        else:
            p = _vector(t, name, like, dim, pdt)
        setattr(params, name, p)
    if groups is None or groups == rows == 0:      # none, or one for each of no rows
        groups = 1
    if groups < 1 or rows % groups:
        raise ValueError(f"{rows} rows in {groups} groups")
    desc = SpadeRowDesc(rows, groups, dim, dtype_code(x_dtype), dtype_code(branch_dtype), dtype_code(pdt),
                        _code(NORM, norm, "norm"), _code(NORM, post_norm, "post_norm"), eps, post_eps, residual_scale)
    if strides:
        for name, stride in strides.items():
            setattr(desc, name + "_stride", stride)
    return desc, params, given


def _row_grads(given, like):
    """Float32 gradient tensors of the parameters given, and their table."""
    out, table = {}, SpadeRowGrads()
    for n in ROW_PARAMS:
        t = given[n]
        out[n] = t if t is None else _new(t, t.shape, torch.float32)
        if t is not None:
            setattr(table, n, out[n].data_ptr())
    return out, table


def row_workspace_bytes(rows: int, dim: int, groups: int = 1) -> int:
    """Scratch of norm_modulate_backward, gate_residual_backward and
    gate_residual_norm_backward on the current device."""
    _fits(64, rows, groups)
    _fits(32, dim)
    desc = SpadeRowDesc(rows=rows, groups=groups, dim=dim)
    return int(_lib.load().spade_row_bwd_workspace_bytes(ctypes.byref(desc)))


def norm_modulate(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                  scale: Optional[torch.Tensor] = None, shift: Optional[torch.Tensor] = None, norm: str = "layer",
                  eps: float = 1e-6, out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                  stream=None) -> torch.Tensor:
    """The norm that opens a block: (norm(x) * weight + bias) * (1 + scale) +
    shift, each parameter optional.  x [rows, dim]; weight, bias [dim]; scale,
    shift [groups, dim] (or [dim]): the rows fall into `groups` equal runs
    (frames, samples, or single tokens).  norm: "layer" or "rms".  The result
    is out, or a new tensor of out_dtype (x's by default).  Autograd records
    nothing, whatever the inputs require; norm_modulate_backward gives the
    gradients."""
    odt = out.dtype if out is not None else (out_dtype or x.dtype)
    desc, params, _ = _row_call(x, x.dtype, odt, norm, eps, weight=weight, bias=bias, scale=scale, shift=shift)
    with _On(x, stream) as s:
        xp, desc.x_stride = _strided(x, "x", x, x.shape, x.dtype)
        out, op, desc.h_stride = _output(out, "out", x, x.shape, odt)
        check(_lib.load().spade_norm_modulate(ctypes.byref(desc), ctypes.byref(params), xp, op, s), "spade_norm_modulate")
    return out


def norm_modulate_backward(dout: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                           bias: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                           shift: Optional[torch.Tensor] = None, norm: str = "layer", eps: float = 1e-6,
                           dres: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, stream=None) -> RowGrads:
    """Gradients of norm_modulate: of x (plus dres, a gradient that reaches x
    by another way) and of the parameters given (float32).  dx: where x's goes
    (dres itself is allowed)."""
    desc, params, given = _row_call(x, x.dtype, dout.dtype, norm, eps, weight=weight, bias=bias, scale=scale, shift=shift)
    with _On(x, stream) as s:
        xp, desc.x_stride = _strided(x, "x", x, x.shape, x.dtype)
        hp, desc.dh_stride = _strided(dout, "dout", x, x.shape, dout.dtype)
        rp, desc.dx_out_stride = _strided(dres, "dres", x, x.shape, x.dtype)
        dx, dp, desc.dx_stride = _output(dx, "dx", x, x.shape, x.dtype)
        out, grads = _row_grads(given, x)
        lib = _lib.load()
        wp, wn, workspace = _scratch(workspace, _row_scratch_bytes(x, desc, given), x)
        check(lib.spade_norm_modulate_bwd(ctypes.byref(desc), ctypes.byref(params), hp, rp, xp, dp, ctypes.byref(grads),
                                          wp, wn, s), "spade_norm_modulate_bwd")
    return RowGrads(x=dx, y=None, **out)


def gate_residual(x: torch.Tensor, y: torch.Tensor, gate: Optional[torch.Tensor] = None, post_norm: str = "none",
                  post_weight: Optional[torch.Tensor] = None, post_eps: float = 1e-6, residual_scale: float = 1.0,
                  out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The update that ends a block: x + residual_scale * gate *
    (post_norm(y) * post_weight).  x, y [rows, dim]; gate [groups, dim] or
    [dim].  out: where the sum goes (x itself is allowed).  Autograd records
    nothing, whatever the inputs require; gate_residual_backward gives the
    gradients."""
    desc, params, _ = _row_call(x, x.dtype, y.dtype, post_norm=post_norm, post_eps=post_eps,
                                residual_scale=residual_scale, gate=gate, post_weight=post_weight)
    with _On(x, stream) as s:
        xp, desc.x_stride = _strided(x, "x", x, x.shape, x.dtype)
        yp, desc.y_stride = _strided(y, "y", x, x.shape, y.dtype)
        out, op, desc.x_out_stride = _output(out, "out", x, x.shape, x.dtype)
        check(_lib.load().spade_gate_residual(ctypes.byref(desc), ctypes.byref(params), xp, yp, op, s),
              "spade_gate_residual")
    return out


def gate_residual_backward(dout: torch.Tensor, y: torch.Tensor, gate: Optional[torch.Tensor] = None,
                           post_norm: str = "none", post_weight: Optional[torch.Tensor] = None,
                           post_eps: float = 1e-6, residual_scale: float = 1.0, dy: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, stream=None) -> RowGrads:
    """Gradients of gate_residual: of y and of the parameters given (float32).
    x's gradient is dout (returned as x)."""
    desc, params, given = _row_call(dout, dout.dtype, y.dtype, post_norm=post_norm, post_eps=post_eps,
                                    residual_scale=residual_scale, gate=gate, post_weight=post_weight)
    with _On(dout, stream) as s:
        gp, desc.dx_out_stride = _strided(dout, "dout", dout, dout.shape, dout.dtype)
        yp, desc.y_stride = _strided(y, "y", dout, dout.shape, y.dtype)
        dy, dp, desc.dy_stride = _output(dy, "dy", y, dout.shape, y.dtype)
        out, grads = _row_grads(given, dout)
        lib = _lib.load()
        wp, wn, workspace = _scratch(workspace, _row_scratch_bytes(dout, desc, given), dout)
        check(lib.spade_gate_residual_bwd(ctypes.byref(desc), ctypes.byref(params), gp, yp, dp, ctypes.byref(grads), wp,
                                          wn, s), "spade_gate_residual_bwd")
    return RowGrads(x=dout, y=dy, **out)


def gate_residual_norm(x: torch.Tensor, y: torch.Tensor, gate: Optional[torch.Tensor] = None, post_norm: str = "none",
                       post_weight: Optional[torch.Tensor] = None, post_eps: float = 1e-6,
                       residual_scale: float = 1.0, weight: Optional[torch.Tensor] = None,
                       bias: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                       shift: Optional[torch.Tensor] = None, norm: str = "layer", eps: float = 1e-6,
                       x_out: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                       stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """gate_residual and the norm_modulate of the block that follows, in one
    pass: returns (x_out, out), out of y's dtype, taken of the sum before it
    is rounded to x's.  x_out may be x, out may be y.  gate, scale and shift
    have one number of groups.  Autograd records nothing, whatever the inputs
    require; gate_residual_norm_backward gives the gradients."""
    desc, params, _ = _row_call(x, x.dtype, y.dtype, norm, eps, post_norm, post_eps, residual_scale, gate, post_weight,
                                weight, bias, scale, shift)
    with _On(x, stream) as s:
        xp, desc.x_stride = _strided(x, "x", x, x.shape, x.dtype)
        yp, desc.y_stride = _strided(y, "y", x, x.shape, y.dtype)
        x_out, op, desc.x_out_stride = _output(x_out, "x_out", x, x.shape, x.dtype)
        out, hp, desc.h_stride = _output(out, "out", y, x.shape, y.dtype)
        check(_lib.load().spade_gate_residual_norm(ctypes.byref(desc), ctypes.byref(params), xp, yp, op, hp, s),
              "spade_gate_residual_norm")
    return x_out, out


def gate_residual_norm_backward(dx_out: Optional[torch.Tensor], dout: torch.Tensor, x: torch.Tensor, y: torch.Tensor,
                                gate: Optional[torch.Tensor] = None, post_norm: str = "none",
                                post_weight: Optional[torch.Tensor] = None, post_eps: float = 1e-6,
                                residual_scale: float = 1.0, weight: Optional[torch.Tensor] = None,
                                bias: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                                shift: Optional[torch.Tensor] = None, norm: str = "layer", eps: float = 1e-6,
                                dx: Optional[torch.Tensor] = None, dy: Optional[torch.Tensor] = None,
                                workspace: Optional[torch.Tensor] = None, stream=None) -> RowGrads:
    """Gradients of gate_residual_norm: of x and y (its inputs, given again)
    and of the parameters given (float32), from those of x_out (None: unused)
    and out.  dx may be dx_out; dy may be dout."""
    desc, params, given = _row_call(x, x.dtype, y.dtype, norm, eps, post_norm, post_eps, residual_scale, gate, post_weight,
                                    weight, bias, scale, shift)
    with _On(x, stream) as s:
        gp, desc.dx_out_stride = _strided(dx_out, "dx_out", x, x.shape, x.dtype)
        hp, desc.dh_stride = _strided(dout, "dout", x, x.shape, y.dtype)
        xp, desc.x_stride = _strided(x, "x", x, x.shape, x.dtype)
        yp, desc.y_stride = _strided(y, "y", x, x.shape, y.dtype)
        dx, dxp, desc.dx_stride = _output(dx, "dx", x, x.shape, x.dtype)
        dy, dyp, desc.dy_stride = _output(dy, "dy", y, x.shape, y.dtype)
        out, grads = _row_grads(given, x)
        lib = _lib.load()
        wp, wn, workspace = _scratch(workspace, _row_scratch_bytes(x, desc, given), x)
        check(lib.spade_gate_residual_norm_bwd(ctypes.byref(desc), ctypes.byref(params), gp, hp, xp, yp, dxp, dyp,
                                               ctypes.byref(grads), wp, wn, s), "spade_gate_residual_norm_bwd")
    return RowGrads(x=dx, y=dy, **out)


def last_device_status(stream=None) -> int:
    return int(_lib.load().spade_last_device_status(_stream(stream)))


def selftest_bounded_wait(timeout_ns: int, stream=None) -> None:
    check(_lib.load().spade_selftest_bounded_wait(int(timeout_ns), _stream(stream)),
          "spade_selftest_bounded_wait")
