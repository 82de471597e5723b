"""Rotary positions and attention over the key blocks that each query selects.

Binding of the operators beside the SparsePR call (include/sparsepr.h): argument marshalling
only, as in ``sparsepr.py``.  Tensors are [batch, heads, rows, d] CUDA tensors with
contiguous rows and any strides of whole 16-byte units (a transposed [batch, rows, heads, d]
buffer works); every call runs on the tensors' device and the current stream there.

    plan = spr.rotary_plan(128, device, base=1e4)
    q, k = spr.rotary(plan, positions, q, k)             # positions [batch, rows, 1] int32
    cfg = spr.SelectConfig(block=128, top=16, causal=True)
    out = spr.block_attention(q, k, v, cfg)              # means, selection and attention

or, call by call, with a workspace that the caller keeps:

    ws = spr.selected_workspace(q, k, cfg, backward=True)
    means = spr.key_means(k, cfg.block)
    sel = spr.select_blocks(q, means, k.shape[2], cfg, ws)
    rest = torch.empty(q.shape, dtype=q.dtype, device=q.device)   # bf16 training: what out's rounding leaves off
    out, lse = spr.selected_attn(q, k, v, sel, cfg, ws, rest=rest)
    dq, dk, dv = spr.selected_attn_backward(dout, q, k, v, out, lse, sel, cfg, ws, rest=rest)

Where a tensor needs a gradient, autograd records ``rotary``, ``selected_attn`` and
``block_attention`` (so ``block_attention(q, k, v, cfg).backward(dout)`` works); the calls for
gradients are for who keeps outputs and workspaces, and for steps captured into graphs.

For a cache, ``kv_len`` [batch] holds each sequence's length and ``q_start`` [batch] the key
position of its first query; after appending keys, ``key_means(..., kv_start=, max_new=,
out=means)`` renews the touched blocks' means.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
import math
import threading
from typing import NamedTuple, Optional, Sequence

import torch
from torch.autograd.function import once_differentiable

from . import sparsepr as _s

ROTARY_HALF, ROTARY_INTERLEAVED = 0, 1


class _CView(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride_b", ctypes.c_int64), ("stride_h", ctypes.c_int64),
                ("stride_n", ctypes.c_int64)]


class _CRotary(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("first", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("axes", ctypes.c_int32), ("pairs", ctypes.c_int32 * 4), ("inverse", ctypes.c_int32),
                ("factor", ctypes.c_float)]


class _CSelected(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("dtype", "Bt", "Hq", "Hkv", "Nq", "Nk", "d", "block", "top", "causal",
                                              "n_first", "n_local")] + \
               [("scale", ctypes.c_float), ("kv_len", ctypes.c_void_p), ("q_start", ctypes.c_void_p),
                ("out_rest", ctypes.c_void_p)]


def signatures():
    """ctypes result and argument types of these entry points."""
    vp, i32, i64, v = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.POINTER(_CView)
    p = ctypes.POINTER(_CSelected)
    return {
        "sparsepr_rotary": (ctypes.c_int, [ctypes.POINTER(_CRotary), vp, vp, i64, i64, ctypes.c_int, i32, i32, i32, i32, v,
                                           v, i32, v, v, vp]),
        "sparsepr_selected_workspace_size": (ctypes.c_size_t, [p, ctypes.c_int]),
        "sparsepr_key_means": (ctypes.c_int, [p, v, vp, i32, vp, vp]),
        "sparsepr_select_blocks": (ctypes.c_int, [p, v, vp, vp, vp, vp]),
        "sparsepr_selected_attn": (ctypes.c_int, [p, v, v, v, vp, v, vp, vp, vp]),
        "sparsepr_selected_attn_backward": (ctypes.c_int, [p, v, v, v, v, v, vp, vp, v, v, v, vp, vp]),
    }


def _view(t: Optional[torch.Tensor]) -> _CView:
    if t is None:
        return _CView(None, 0, 0, 0)
    n0, n1, n2, _ = t.shape
    s0, s1, s2, _ = t.stride()
    # a dimension of one row has no stride to speak of
    return _CView(t.data_ptr(), s0 if n0 > 1 else 0, s1 if n1 > 1 else 0, s2 if n2 > 1 else 0)


def _need_rows(name: str, t: torch.Tensor, shape=None, like: Optional[torch.Tensor] = None) -> None:
    """A [batch, heads, rows, d] CUDA tensor with contiguous rows (of the given shape, type and device)."""
    if not t.is_cuda:
        raise ValueError("SparsePR tensors must live on a CUDA device")
    if t.dim() != 4 or t.stride(3) != 1:
        raise ValueError(f"{name} must be [batch, heads, rows, d] with contiguous rows")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if like is None:
        _s._dtype_code(t)
    elif t.dtype != like.dtype or t.device != like.device:
        raise ValueError(f"{name} must have the type and device of the other tensors")


def _need_flat(name: str, t: Optional[torch.Tensor], shape, dtype, device) -> None:
    """A contiguous CUDA tensor of the given shape, type and device, or None."""
    if t is not None and (t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")


def _expanded(t: torch.Tensor) -> bool:
    return 0 in t.stride() and any(n > 1 and st == 0 for n, st in zip(t.shape, t.stride()))


def _need_out(name: str, t: torch.Tensor) -> None:
    """No two rows of an output in one place."""
    if _expanded(t):
        raise ValueError(f"{name} must not be an expanded tensor")


def _rows_like(t: torch.Tensor) -> torch.Tensor:
    """Empty tensor of t's shape and, unless it is expanded, memory order."""
    return torch.empty(t.shape, dtype=t.dtype, device=t.device) if _expanded(t) else torch.empty_like(t)


class _Call:
    """An entry point with its arguments checked and marshalled for one signature (shapes,
    strides, types, devices, options): a call fills in the pointers.  Kept per thread, because
    the structures are filled in place; nothing in it depends on an address or a value."""

    def __init__(self, name: str, device: torch.device):
        self.fn, self.name, self.device, self.index = getattr(_s.lib(), name), name, device, device.index

    def run(self, *args) -> None:
        stream = torch._C._cuda_getCurrentRawStream(self.index)
        if self.index == torch.cuda.current_device():
            rc = self.fn(*args, stream)
        else:
            with torch.cuda.device(self.index):
                rc = self.fn(*args, stream)
        if rc != _s.OK:
            raise _s.SparsePRError(rc, f"{self.name}: {_s.lib().sparsepr_last_error().decode(errors='replace')}")


_CALLS = threading.local()


def _signature(*tensors):
    return tuple([None if t is None else (t.shape, t.stride(), t.dtype, t.get_device()) for t in tensors])


def _prepared(key, make, *args):
    """The call of this signature, checked by ``make`` the first time."""
    calls = _CALLS.__dict__.setdefault("calls", {})
    call = calls.get(key)
    if call is None:
        call = make(*args)
        if len(calls) >= 512:
            calls.clear()
        calls[key] = call
    return call


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _written(*outs) -> None:
    """Given outputs count as changed in place, as by torch's own calls: a graph that kept one says so."""
    for t in outs:
        if t is not None and not t.is_inference():
            torch.autograd.graph.increment_version(t)


def _may_record(**outs) -> None:
    """Refusals of a call that autograd is to record: it makes its own outputs, and is not captured."""
    for name, t in outs.items():
        if t is not None:
            raise ValueError(f"{name} cannot be given where autograd records the call (it can under torch.no_grad())")
    if torch.cuda.is_current_stream_capturing():
        raise ValueError("a call that autograd records cannot be captured into a graph: capture it under torch.no_grad(), "
                         "with the calls for gradients")


def _plain_rows(g: torch.Tensor) -> torch.Tensor:
    """An incoming gradient as the calls take it: contiguous rows on 16-byte boundaries."""
    per = 16 // g.element_size()
    if g.stride(3) == 1 and g.data_ptr() % 16 == 0 and all(n == 1 or st % per == 0 for n, st in zip(g.shape[:3], g.stride())):
        return g
    return g.clone(memory_format=torch.contiguous_format)


# ------------------------------------------------------------------------------ rotary

class RotaryPlan(NamedTuple):
    """What a rotation needs besides the positions (made once by ``rotary_plan``)."""
    freqs: torch.Tensor   # [rot_dim / 2] float64: radians per step of the position
    d: int
    rot_dim: int
    first: int
    layout: int
    sections: tuple       # pairs of each position axis
    factor: float


def rotary_frequencies(sections: Sequence[int], base: float = 10000.0, scaling: str = "none", scaling_factor: float = 1.0,
                       trained_length: int = 0, slow: float = 1.0, fast: float = 32.0):
    """(frequencies, factor) of a rotation, in 64 bits on the host: for each axis with p pairs
    f_i = base^(-i/p), i < p, and for contexts ``scaling_factor`` s times the trained length

      "linear"  f_i / s (positions interpolated)
      "base"    the ladder of the base  base * s^(2p / (2p - 2)): the lowest frequency is divided by s
      "ramp"    by turns r_i = trained_length f_i / (2 pi) within the trained length: f_i / s where
                r_i <= slow, f_i where r_i >= fast, linear in r_i between; factor 0.1 ln s + 1
    """
    if scaling not in ("none", "linear", "base", "ramp"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if not (math.isfinite(base) and base > 0 and math.isfinite(scaling_factor) and scaling_factor > 0):
        raise ValueError("base and scaling_factor must be positive")
    if scaling == "ramp" and (trained_length < 1 or not fast > slow):
        raise ValueError("ramp scaling needs trained_length >= 1 and fast > slow")
    freqs = []
    for p in sections:
        if p < 0:
            raise ValueError("an axis cannot have a negative number of pairs")
        b = base
        if scaling == "base" and p > 1:
            b = base * scaling_factor ** (2 * p / (2 * p - 2))
        f = [b ** (-i / p) for i in range(p)]
        if scaling == "linear":
            f = [x / scaling_factor for x in f]
        elif scaling == "ramp":
            keep = [min(1.0, max(0.0, (trained_length * x / (2 * math.pi) - slow) / (fast - slow))) for x in f]
            f = [x * g + x / scaling_factor * (1.0 - g) for x, g in zip(f, keep)]
        freqs += f
    factor = 0.1 * math.log(scaling_factor) + 1.0 if scaling == "ramp" and scaling_factor > 1 else 1.0
    return freqs, factor


def rotary_plan(d: int, device, rot_dim: Optional[int] = None, first: int = 0, layout: int = ROTARY_HALF,
                sections: Optional[Sequence[int]] = None, freqs: Optional[torch.Tensor] = None,
                factor: Optional[float] = None, **ladder) -> RotaryPlan:
    """Plan for heads of d dims whose dims [first, first + rot_dim) rotate (default: all).
    ``sections``: pairs of each position axis, for example (24, 20, 20) for the t, y and x of a
    video grid at d = 128 (default: one axis).  Frequencies come from ``rotary_frequencies``
    (``ladder``: base, scaling, ...) or are given as ``freqs`` [rot_dim / 2], with ``factor``."""
    rot_dim = d - first if rot_dim is None else rot_dim
    if rot_dim < 2 or rot_dim % 2 or first < 0 or first + rot_dim > d:
        raise ValueError("the rotated part must be an even number of dims inside the head")
    if layout not in (ROTARY_HALF, ROTARY_INTERLEAVED):
        raise ValueError(f"unknown rotary layout {layout}")
    sections = (rot_dim // 2,) if sections is None else tuple(int(s) for s in sections)
    if not 1 <= len(sections) <= 4 or min(sections) < 0 or sum(sections) != rot_dim // 2:
        raise ValueError("sections: one to four axes whose pairs add up to rot_dim / 2")
    if freqs is None:
        f, scale = rotary_frequencies(sections, **ladder)
        freqs = torch.tensor(f, dtype=torch.float64, device=device)
    else:
        if ladder:
            raise ValueError("give frequencies or a ladder's parameters, not both")
        freqs, scale = torch.as_tensor(freqs, dtype=torch.float64, device=device).contiguous(), 1.0
        if tuple(freqs.shape) != (rot_dim // 2,):
            raise ValueError("freqs must hold rot_dim / 2 values")
    return RotaryPlan(freqs, d, rot_dim, first, layout, sections, float(scale if factor is None else factor))


def rotary(plan: RotaryPlan, positions: torch.Tensor, q: torch.Tensor, k: Optional[torch.Tensor] = None,
           inverse: bool = False, out=None):
    """q and k rotated by their positions, in one launch: a tensor, or a pair where k is given.

    positions: int32 [batch or 1, rows, axes] (axes may be left out where there is one), last
    dimension contiguous.  ``inverse`` rotates back: the gradient of the rotation (the factor
    is applied in both directions).  ``out``: the output tensor or pair, which may be the input
    itself or a strided view such as the new rows of a key cache.  Autograd records the call where
    q or k needs a gradient."""
    if (q.requires_grad or (k is not None and k.requires_grad)) and torch.is_grad_enabled():
        _may_record(out=out)
        return _Rotary.apply(plan, positions, bool(inverse), q, k)
    qo, ko = (None, None) if out is None else tuple(out) if k is not None else (out, None)
    key = ("rotary", plan[1:], bool(inverse), _signature(plan.freqs, positions, q, k, qo, ko))
    c = _prepared(key, _rotary_call, plan, positions, q, k, inverse, qo, ko)
    if out is not None:
        _written(qo, ko)
    qo = _rows_like(q) if qo is None else qo
    if k is not None:
        ko = _rows_like(k) if ko is None else ko
        c.k.data, c.ko.data = k.data_ptr(), ko.data_ptr()
    c.q.data, c.qo.data = q.data_ptr(), qo.data_ptr()
    c.run(c.par_ref, plan.freqs.data_ptr(), positions.data_ptr(), *c.sizes, c.q_ref, c.qo_ref, c.h2, c.k_ref, c.ko_ref)
    return qo if k is None else (qo, ko)


class _Rotary(torch.autograd.Function):
    """The gradient of a rotation is the rotation back."""

    @staticmethod
    def forward(ctx, plan, positions, inverse, q, k):
        ctx.save_for_backward(positions, plan.freqs)
        ctx.plan, ctx.inverse, ctx.both = plan, inverse, k is not None
        return rotary(plan, positions, q, k, inverse=inverse)

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        positions, freqs = ctx.saved_tensors
        gq, gk = (_plain_rows(g) for g in (grads if ctx.both else (grads[0], grads[0])))
        got = rotary(ctx.plan._replace(freqs=freqs), positions, gq, gk if ctx.both else None, inverse=not ctx.inverse)
        return (None, None, None) + (got if ctx.both else (got, None))


def _rotary_call(plan, positions, q, k, inverse, qo, ko) -> _Call:
    for name, t in (("q", q), ("k", k)):
        if t is not None:
            _need_rows(name, t, (q.shape[0], t.shape[1], q.shape[2], q.shape[3]), q)
    bt, h, n, d = q.shape
    if d != plan.d or plan.freqs.device != q.device:
        raise ValueError("the plan was made for another head dim or device")
    _need_flat("the plan's freqs", plan.freqs, (plan.rot_dim // 2,), torch.float64, q.device)
    axes = len(plan.sections)
    at = positions[..., None] if positions.dim() == 2 and axes == 1 else positions
    if at.dtype != torch.int32 or at.device != q.device or at.dim() != 3 or at.shape[0] not in (1, bt) or \
            tuple(at.shape[1:]) != (n, axes) or (axes > 1 and at.stride(2) != 1):
        raise ValueError(f"positions must be int32 [{bt} or 1, {n}, {axes}] on the tensors' device")
    for name, t, o in (("out of q", q, qo), ("out of k", k, ko)):
        if t is not None and o is not None:
            _need_rows(name, o, t.shape, t)
            _need_out(name, o)
    c = _Call("sparsepr_rotary", q.device)
    pairs = (ctypes.c_int32 * 4)(*(plan.sections + (0,) * (4 - axes)))
    c.par = _CRotary(plan.rot_dim, plan.first, plan.layout, axes, pairs, 1 if inverse else 0, plan.factor)
    c.q, c.k = _view(q), _view(k)
    # outputs that the call makes have the strides of _rows_like
    c.qo = _view(_rows_like(q) if qo is None else qo)
    c.ko = _view(None if k is None else _rows_like(k) if ko is None else ko)
    c.par_ref, c.q_ref, c.k_ref, c.qo_ref, c.ko_ref = (ctypes.byref(x) for x in (c.par, c.q, c.k, c.qo, c.ko))
    c.h2 = 0 if k is None else k.shape[1]
    c.sizes = (at.stride(0) if at.shape[0] > 1 else 0, at.stride(1), _s._dtype_code(q), bt, n, d, h)
    return c


# ------------------------------------------------------------- attention over selected blocks

@dataclasses.dataclass(frozen=True)
class SelectConfig:
    """Attention over selected key blocks: keys per block (64 or 128), blocks per query, causal
    masking, blocks that are always selected (the first ``n_first``; causal: the query's own
    block, unless ``n_first`` = ``top``, and the ``n_local`` - 1 before it) and the softmax scale
    (<= 0: 1/sqrt(d))."""
    block: int = 128
    top: int = 16
    causal: bool = False
    n_first: int = 0
    n_local: int = 0
    scale: float = 0.0


def _problem(dtype_of, bt, hq, hk, nq, nk, d, cfg: SelectConfig) -> _CSelected:
    return _CSelected(_s._dtype_code(dtype_of), bt, hq, hk, nq, nk, d, cfg.block, cfg.top, int(bool(cfg.causal)),
                      cfg.n_first, cfg.n_local, cfg.scale, None, None, None)


def _lengths(bt: int, device, kv_len, q_start) -> None:
    _need_flat("kv_len", kv_len, (bt,), torch.int32, device)
    _need_flat("q_start", q_start, (bt,), torch.int32, device)


def selected_workspace(q: torch.Tensor, k: torch.Tensor, cfg: SelectConfig, backward: bool = False) -> torch.Tensor:
    """Workspace of the calls below for tensors of these shapes (status header zeroed)."""
    _need_rows("q", q)
    _need_rows("k", k, (q.shape[0], k.shape[1], k.shape[2], q.shape[3]), q)
    p = _problem(q, q.shape[0], q.shape[1], k.shape[1], q.shape[2], k.shape[2], q.shape[3], cfg)
    size = int(_s.lib().sparsepr_selected_workspace_size(ctypes.byref(p), 1 if backward else 0))
    if size == 0:
        raise _s.SparsePRError(_s.ERR_INVALID_ARG,
                               f"selected_workspace: {_s.lib().sparsepr_last_error().decode(errors='replace')}")
    ws = torch.empty(size, dtype=torch.uint8, device=q.device)
    ws[:256].zero_()
    return ws


@functools.lru_cache(maxsize=256)
def _ws_size(dtype, bt, hq, hk, nq, nk, d, cfg: SelectConfig, backward: bool) -> int:
    """Workspace bytes of a problem: a function of its sizes alone."""
    p = _CSelected(dtype, bt, hq, hk, nq, nk, d, cfg.block, cfg.top, int(bool(cfg.causal)), cfg.n_first, cfg.n_local,
                   cfg.scale, None, None, None)
    return int(_s.lib().sparsepr_selected_workspace_size(ctypes.byref(p), 1 if backward else 0))


def _need_ws(ws: torch.Tensor, p: _CSelected, cfg: SelectConfig, device, backward: bool) -> None:
    size = _ws_size(p.dtype, p.Bt, p.Hq, p.Hkv, p.Nq, p.Nk, p.d, cfg, backward)
    if size and (ws.device != device or ws.dtype != torch.uint8 or not ws.is_contiguous() or ws.numel() < size):
        raise ValueError("the workspace is too small for these tensors or on another device")


def _need_aligned(ws: torch.Tensor) -> None:
    if ws.data_ptr() & 255:
        raise ValueError("the workspace must start on a 256-byte boundary")


def key_means(k: torch.Tensor, block: int, kv_len: Optional[torch.Tensor] = None,
              kv_start: Optional[torch.Tensor] = None, max_new: int = 0, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Mean key of every block of ``block`` keys: [batch, heads, ceil(rows / block), d] fp32.
    With ``kv_start`` [batch] int32 only the blocks holding keys [kv_start, kv_len) are renewed
    in ``out`` (at most ``max_new`` keys per sequence were appended).  For selections: carries no
    gradient."""
    c = _prepared(("means", block, _signature(k, kv_len, kv_start, out)), _means_call, k, block, kv_len, kv_start, out)
    means = torch.empty(c.shape, dtype=torch.float32, device=k.device) if out is None else out
    if out is not None:
        _written(out)
    c.k.data, c.p.kv_len = k.data_ptr(), _ptr(kv_len)
    c.run(c.p_ref, c.k_ref, _ptr(kv_start), max_new, means.data_ptr())
    return means


def _means_call(k, block, kv_len, kv_start, out) -> _Call:
    _need_rows("k", k)
    bt, h, n, d = k.shape
    _lengths(bt, k.device, kv_len, kv_start)
    if kv_start is not None and out is None:
        raise ValueError("kv_start renews blocks of an existing tensor: give out")
    c = _Call("sparsepr_key_means", k.device)
    c.shape = (bt, h, -(-n // block) if block > 0 else 0, d)
    _need_flat("out", out, c.shape, torch.float32, k.device)
    c.p, c.k = _problem(k, bt, h, h, 1, n, d, SelectConfig(block=block, top=1)), _view(k)
    c.p_ref, c.k_ref = ctypes.byref(c.p), ctypes.byref(c.k)
    return c


def select_blocks(q: torch.Tensor, means: torch.Tensor, keys: int, cfg: SelectConfig, ws: torch.Tensor,
                  kv_len: Optional[torch.Tensor] = None, q_start: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Blocks of the ``keys`` keys that each query attends to: [batch, key heads, rows, top]
    int32, ascending, then -1 (ties to the lower block; the scores are compared in 64 bits)."""
    key = ("select", keys, cfg, ws.numel(), _signature(q, means, ws, kv_len, q_start, out))
    c = _prepared(key, _select_call, q, means, keys, cfg, ws, kv_len, q_start, out)
    _need_aligned(ws)
    sel = torch.empty(c.shape, dtype=torch.int32, device=q.device) if out is None else out
    if out is not None:
        _written(out)
    c.q.data, c.p.kv_len, c.p.q_start = q.data_ptr(), _ptr(kv_len), _ptr(q_start)
    c.run(c.p_ref, c.q_ref, means.data_ptr(), sel.data_ptr(), ws.data_ptr())
    return sel


def _select_call(q, means, keys, cfg, ws, kv_len, q_start, out) -> _Call:
    _need_rows("q", q)
    bt, hq, n, d = q.shape
    hk = means.shape[1] if means.dim() == 4 else 0
    _need_flat("means", means, (bt, hk, -(-keys // cfg.block) if cfg.block > 0 else 0, d), torch.float32, q.device)
    _lengths(bt, q.device, kv_len, q_start)
    c = _Call("sparsepr_select_blocks", q.device)
    c.p, c.q, c.shape = _problem(q, bt, hq, hk, n, keys, d, cfg), _view(q), (bt, hk, n, cfg.top)
    _need_ws(ws, c.p, cfg, q.device, False)
    _need_flat("out", out, c.shape, torch.int32, q.device)
    c.p_ref, c.q_ref = ctypes.byref(c.p), ctypes.byref(c.q)
    return c


def _attention_call(name, backward, cfg, ws, sel, kv_len, q_start, lse, rest, q, k, v, others) -> _Call:
    """Checks of both attention calls; ``others``: (name, tensor or None where the call makes it,
    the tensor whose shape it has, whether it is an output)."""
    _need_rows("q", q)
    bt, hq, n, d = q.shape
    _need_rows("k", k, (bt, k.shape[1], k.shape[2], d), q)
    _need_rows("v", v, k.shape, q)
    _need_flat("sel", sel, (bt, k.shape[1], n, cfg.top), torch.int32, q.device)
    _need_flat("lse", lse, q.shape[:3], torch.float32, q.device)
    if rest is not None and q.dtype != torch.bfloat16:
        raise ValueError("rest goes with bf16 tensors")
    _need_flat("rest", rest, q.shape, torch.bfloat16, q.device)
    _lengths(bt, q.device, kv_len, q_start)
    c = _Call(name, q.device)
    c.p = _problem(q, bt, hq, k.shape[1], n, k.shape[2], d, cfg)
    _need_ws(ws, c.p, cfg, q.device, backward)
    c.views = [_view(q), _view(k), _view(v)]
    for what, t, like, is_out in others:
        if t is not None:
            _need_rows(what, t, like.shape, q)
            if is_out:
                _need_out(what, t)
        c.views.append(_view(_rows_like(like) if t is None else t))
    c.refs = [ctypes.byref(x) for x in c.views]
    c.p_ref, c.lse_shape = ctypes.byref(c.p), q.shape[:3]
    return c


def _fill(c: _Call, kv_len, q_start, rest, *tensors) -> None:
    c.p.kv_len, c.p.q_start, c.p.out_rest = _ptr(kv_len), _ptr(q_start), _ptr(rest)
    for view, t in zip(c.views, tensors):
        view.data = t.data_ptr()


def selected_attn(q, k, v, sel: torch.Tensor, cfg: SelectConfig, ws: torch.Tensor,
                  kv_len: Optional[torch.Tensor] = None, q_start: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                  rest: Optional[torch.Tensor] = None):
    """Softmax attention of every query over the keys of its selected blocks: (out, lse), out
    like q and lse [batch, heads, rows] fp32 (natural log; -inf and a zero row without keys).
    ``rest``: a contiguous bf16 tensor of q's shape that gets what the rounding of out left off,
    for the backward call.

    Autograd records the call where q, k or v needs a gradient (of out; lse carries none): it keeps
    the inputs, out, lse and, in bf16, a rest of its own, and its backward pass takes a workspace
    of its own, whose errors end up in ``ws``."""
    if (q.requires_grad or k.requires_grad or v.requires_grad) and torch.is_grad_enabled():
        _may_record(out=out, lse=lse, rest=rest)
        return _SelectedAttn.apply(cfg, ws, ws[:4].view(torch.int32), q, k, v, sel, kv_len, q_start)
    key = ("attn", cfg, _signature(q, k, v, sel, ws, kv_len, q_start, out, lse, rest))
    c = _prepared(key, _attention_call, "sparsepr_selected_attn", False, cfg, ws, sel, kv_len, q_start, lse, rest, q, k, v,
                  (("out", out, q, True),))
    _need_aligned(ws)
    if out is not None or lse is not None or rest is not None:
        _written(out, lse, rest)
    out = _rows_like(q) if out is None else out
    lse = torch.empty(c.lse_shape, dtype=torch.float32, device=q.device) if lse is None else lse
    _fill(c, kv_len, q_start, rest, q, k, v, out)
    r = c.refs
    c.run(c.p_ref, r[0], r[1], r[2], sel.data_ptr(), r[3], lse.data_ptr(), ws.data_ptr())
    return out, lse


def selected_attn_backward(dout, q, k, v, out, lse, sel: torch.Tensor, cfg: SelectConfig, ws: torch.Tensor,
                           kv_len: Optional[torch.Tensor] = None, q_start: Optional[torch.Tensor] = None, dq=None,
                           dk=None, dv=None, rest: Optional[torch.Tensor] = None):
    """(dq, dk, dv) of ``selected_attn`` for the gradient of its output; the selection is fixed.
    ``ws`` was made with ``backward=True``.  An expanded k or v gets the gradient of every repeated
    head (add them up); the heads of a group are added already.  The row sums of dout * out are
    formed from ``out`` as it is stored, so bf16 gradients carry its rounding (it is dq's largest
    error), unless ``rest`` of the forward call is given."""
    if lse is None:
        raise ValueError("lse of the forward call is needed")
    key = ("grad", cfg, _signature(dout, q, k, v, out, lse, sel, ws, kv_len, q_start, dq, dk, dv, rest))
    c = _prepared(key, _attention_call, "sparsepr_selected_attn_backward", True, cfg, ws, sel, kv_len, q_start, lse, rest,
                  q, k, v, (("dout", dout, q, False), ("out", out, q, False), ("dq", dq, q, True), ("dk", dk, k, True),
                            ("dv", dv, k, True)))
    _need_aligned(ws)
    if dq is not None or dk is not None or dv is not None:
        _written(dq, dk, dv)
    dq = _rows_like(q) if dq is None else dq
    dk = _rows_like(k) if dk is None else dk
    dv = _rows_like(k) if dv is None else dv
    _fill(c, kv_len, q_start, rest, q, k, v, dout, out, dq, dk, dv)
    r = c.refs
    c.run(c.p_ref, r[3], r[0], r[1], r[2], r[4], lse.data_ptr(), sel.data_ptr(), r[5], r[6], r[7], ws.data_ptr())
    return dq, dk, dv


class _SelectedAttn(torch.autograd.Function):
    """``selected_attn`` with ``selected_attn_backward``; ``status``: the status word of the caller's
    workspace (a view of it), or None."""

    @staticmethod
    def forward(ctx, cfg, ws, status, q, k, v, sel, kv_len, q_start):
        rest = torch.empty(q.shape, dtype=q.dtype, device=q.device) if q.dtype == torch.bfloat16 else None
        out, lse = selected_attn(q, k, v, sel, cfg, ws, kv_len=kv_len, q_start=q_start, rest=rest)
        ctx.save_for_backward(q, k, v, sel, kv_len, q_start, out, lse, rest)
        ctx.cfg, ctx.status = cfg, status
        ctx.mark_non_differentiable(lse)
        return out, lse

    @staticmethod
    @once_differentiable
    def backward(ctx, dout, _):
        q, k, v, sel, kv_len, q_start, out, lse, rest = ctx.saved_tensors
        ws = selected_workspace(q, k, ctx.cfg, backward=True)
        grads = selected_attn_backward(_plain_rows(dout), q, k, v, out, lse, sel, ctx.cfg, ws, kv_len=kv_len,
                                       q_start=q_start, rest=rest)
        if ctx.status is not None:
            torch.maximum(ctx.status, ws[:4].view(torch.int32), out=ctx.status)
        return (None, None, None) + grads + (None, None, None)


def block_attention(q, k, v, cfg: SelectConfig, ws: Optional[torch.Tensor] = None,
                    kv_len: Optional[torch.Tensor] = None, q_start: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Mean keys, selection and attention in one call: out like q.  Autograd records the call where
    q, k or v needs a gradient; the selection is fixed in it."""
    recorded = (q.requires_grad or k.requires_grad or v.requires_grad) and torch.is_grad_enabled()
    if recorded:
        _may_record(out=out)
    own = ws is None
    ws = selected_workspace(q, k, cfg) if own else ws
    means = key_means(k, cfg.block, kv_len=kv_len)
    sel = select_blocks(q, means, k.shape[2], cfg, ws, kv_len=kv_len, q_start=q_start)
    if recorded:  # (a view of a workspace made here would keep it until the backward pass)
        return _SelectedAttn.apply(cfg, ws, None if own else ws[:4].view(torch.int32), q, k, v, sel, kv_len, q_start)[0]
    return selected_attn(q, k, v, sel, cfg, ws, kv_len=kv_len, q_start=q_start, out=out)[0]
