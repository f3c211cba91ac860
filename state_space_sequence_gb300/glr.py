"""Thin Python binding over include/glr.h: the operators of a gated recurrent block.

* ``glr_scan`` / ``glr_scan_backward`` / ``glr_step``: the gated linear recurrence over a sequence
  (the diagonal recurrence with a decay that the token chooses), its gradients, one token;
* ``glr_join`` / ``glr_join_backward``: gate, norm, residual scale and add, and the next block's
  norm, with their gradients;
* ``glr_ckpt_pack`` / ``glr_ckpt_unpack``: activations kept in 8 bits, also written by
  ``glr_join(ckpt=True)`` and read by ``glr_join_backward(ckpt=...)``.

Like ``dlr.py`` this module passes pointers, sizes and the current torch CUDA stream, and turns
non-zero status codes into exceptions; there is no CPU fallback. Activations are float32,
bfloat16 or float16 with contiguous channels and otherwise any strides (so ``x``, ``r`` and ``i``
may be columns of one projection's output); parameters and states are contiguous float32. All are
on the current device. Memory allocated here for a call on ``stream`` belongs to that stream.
Gradients are calls of their own: nothing here is recorded for autograd.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import struct
from typing import NamedTuple, Optional

import torch

from . import dlr as _dlr

TYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
NORM = {"rms": 0, "layer": 1}
ACT = {"silu": 0, "sigmoid": 1, "none": 2}
STATE_STEPS = 8  # GLR_STATE_STEPS
CKPT_GROUP = 32   # GLR_CKPT_GROUP

_lib = None
# the argument structs of glr.h, every field 8 bytes wide
_SCAN = struct.Struct("4qd19q").pack
_SCAN_BACK = struct.Struct("4qd30q").pack
_STEP = struct.Struct("3qd16q").pack
_JOIN = struct.Struct("5qd22q").pack
_JOIN_BACK = struct.Struct("5qd36q").pack
_NONE3 = (0, 0, 0)


def _load():
    global _lib
    if _lib is None:
        lib = _dlr._load()
        P, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        for name in ("glr_scan", "glr_scan_backward", "glr_step", "glr_join", "glr_join_backward"):
            f = getattr(lib, name)
            f.argtypes, f.restype = [ctypes.c_char_p, P], i32
        for name, n in (("glr_scan_workspace_size", 3), ("glr_scan_backward_workspace_size", 3),
                        ("glr_join_backward_workspace_size", 2)):
            f = getattr(lib, name)
            f.argtypes, f.restype = [i64] * n, sz
        lib.glr_states.argtypes, lib.glr_states.restype = [i64], i64
        lib.glr_ckpt_pack.argtypes = [i64, i64, i64, P, i64, P, P, P]
        lib.glr_ckpt_pack.restype = i32
        lib.glr_ckpt_unpack.argtypes = [i64, i64, i64, P, P, P, i64, P]
        lib.glr_ckpt_unpack.restype = i32
        lib.glr_abi_version.restype = i32
        _lib = lib
    return _lib


def _ok(fn: str, status: int):
    if status:
        raise _dlr.DLRError(fn, status)


_current_device = torch._C._cuda_getDevice


def _stream(stream, dev: int):
    """The stream of a call whose tensors are on device ``dev``. The library launches on the current
    device, so that has to be the tensors' and the stream's: another device's pointers, or its
    stream's handle, would mean nothing there."""
    if dev != _current_device():
        raise ValueError(f"the tensors are on cuda:{dev}, but the current device is "
                         f"cuda:{_current_device()}: call within torch.cuda.device({dev})")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError(f"stream: on cuda:{stream.device_index}, the tensors on cuda:{dev}")
    return stream.cuda_stream


def _on(stream):
    """Allocations for a call on ``stream`` come from that stream's memory."""
    return _NOTHING if stream is None else torch.cuda.stream(stream)


_NOTHING = contextlib.nullcontext()


def _act_type(t) -> int:
    kind = TYPE.get(t.dtype)
    if kind is None or not t.is_cuda:
        raise TypeError("expected float32, bfloat16 or float16 CUDA tensors")
    return kind


def _wrong(t, like, shape, what: str):
    """Says what is wrong with a tensor that a check below turned down."""
    if t.dtype != like.dtype or t.device != like.device:
        raise TypeError(f"{what}: expected {like.dtype} on {like.device}")
    if t.shape != shape:
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{what}: channels must be contiguous")


def _views3(ts, like, dtype, dev, shape, what):
    """(pointer, stride_b, stride_t) of activations [B, L, H], one after the other."""
    out, H = [], shape[2]
    for t in ts:
        sb, st, sh = t.stride() if t.dtype is dtype and t.shape == shape and \
            t.get_device() == dev else (0, 0, -1)
        if sh != 1 and (H > 1 or sh < 0):
            _wrong(t, like, shape, what[len(out) // 3])
        out += (t.data_ptr(), sb, st)
    return out


def _strides3(t):
    """The same of a tensor that is known to fit."""
    sb, st, _ = t.stride()
    return t.data_ptr(), sb, st


def _views2(ts, like, dtype, dev, shape, what):
    """The same for rows [M, H]: (pointer, 0, stride_t), nothing for None."""
    out, H = [], shape[1]
    for t in ts:
        if t is None:
            out += _NONE3
            continue
        st, sh = t.stride() if t.dtype is dtype and t.shape == shape and \
            t.get_device() == dev else (0, -1)
        if sh != 1 and (H > 1 or sh < 0):
            _wrong(t, like, shape, what[len(out) // 3])
        out += (t.data_ptr(), 0, st)
    return out


def _new2(x, H: int, wanted: bool):
    """A tensor of rows for a result, and its (pointer, 0, stride_t); nothing when not wanted."""
    if not wanted:
        return None, _NONE3
    t = torch.empty_like(x, memory_format=torch.contiguous_format)
    return t, (t.data_ptr(), 0, H)


def _f32(t, shape, dev, what: str) -> int:
    if t is None:
        return 0
    if t.dtype is not torch.float32 or t.get_device() != dev or not t.is_contiguous():
        raise TypeError(f"{what}: expected a contiguous float32 tensor on cuda:{dev}")
    if t.shape != shape:
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _bytes(t, shape, dev, what: str) -> int:
    if t is None:
        return 0
    if t.dtype not in (torch.uint8, torch.bool) or t.get_device() != dev or \
            not t.is_contiguous():
        raise TypeError(f"{what}: expected a contiguous bool or uint8 tensor on cuda:{dev}")
    if t.shape != shape:
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


class _NoSpace:
    """Stands for a workspace of no bytes."""
    data_ptr = staticmethod(lambda: 0)
    numel = staticmethod(lambda: 0)


_NO_SPACE = _NoSpace()


def _workspace(workspace, need: int, x):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=x.device) if need else _NO_SPACE
    if workspace.dtype != torch.uint8 or workspace.device != x.device or \
            not workspace.is_contiguous():
        raise TypeError("workspace: expected a contiguous uint8 tensor on the same device")
    return workspace


# The sizes are pure functions of their arguments; asking the library costs 0.5 us a call.
@functools.lru_cache(maxsize=1024)
def glr_scan_workspace_size(B: int, L: int, H: int) -> int:
    """Bytes of device workspace glr_scan needs (0: none, or sizes out of range)."""
    return int(_load().glr_scan_workspace_size(B, L, H))


@functools.lru_cache(maxsize=1024)
def glr_scan_backward_workspace_size(B: int, L: int, H: int) -> int:
    """Bytes of device workspace glr_scan_backward needs (0 for sizes out of range)."""
    return int(_load().glr_scan_backward_workspace_size(B, L, H))


@functools.lru_cache(maxsize=1024)
def glr_join_backward_workspace_size(M: int, H: int) -> int:
    """Bytes of device workspace glr_join_backward needs (0 for sizes out of range)."""
    return int(_load().glr_join_backward_workspace_size(M, H))


def glr_scan(x, r, i, p, scale: float = 8.0, h0=None, reset=None, save_states: bool = False,
             out=None, workspace=None, stream=None):
    """The gated linear recurrence h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t with
    a_t = exp(-scale softplus(p) sigmoid(r_t)) over x, r, i [B, L, H]; p [H]; h0 [B, H] the state
    before the first step (None: zero); reset [B, L] (bool or uint8, None: none) marks steps that
    begin a new sequence. Returns (y [B, L, H], h_last [B, H]) and, with ``save_states``, the
    float32 states [B, ceil(L / 8), H] that glr_scan_backward takes."""
    lib, kind = _load(), _act_type(x)
    if x.dim() != 3:
        raise ValueError("x: expected [B, L, H]")
    shape, dtype, dev = x.shape, x.dtype, x.get_device()
    B, L, H = shape
    views = _views3((x, r, i), x, dtype, dev, shape, ("x", "r", "i"))
    with _on(stream):
        if out is None:
            out = torch.empty_like(x)
            y = _strides3(out)
        else:
            y = _views3((out,), x, dtype, dev, shape, ("out",))
        h_last = torch.empty((B, H), dtype=torch.float32, device=x.device)
        states = torch.empty((B, (L + STATE_STEPS - 1) // STATE_STEPS, H), dtype=torch.float32,
                             device=x.device) if save_states else None
        ws = _workspace(workspace, glr_scan_workspace_size(B, L, H), x)
    args = _SCAN(kind, B, L, H, scale, *views, _f32(p, (H,), dev, "p"),
                 _f32(h0, (B, H), dev, "h0"), _bytes(reset, (B, L), dev, "reset"), *y,
                 h_last.data_ptr(), 0 if states is None else states.data_ptr(), ws.data_ptr(),
                 ws.numel())
    _ok("glr_scan", lib.glr_scan(args, _stream(stream, dev)))
    return (out, h_last, states) if save_states else (out, h_last)


def glr_scan_backward(x, r, i, p, dy, states, scale: float = 8.0, h0=None, reset=None,
                      dh_last=None, out=None, workspace=None, stream=None):
    """Gradients of glr_scan for the gradients dy [B, L, H] of y and dh_last [B, H] (None: zero)
    of h_last; the other arguments as the forward call had them, ``states`` as it returned them.
    ``out``: (dx, dr, di) to write, e.g. the columns of one buffer. Returns (dx, dr, di, dp, dh0),
    dh0 None when h0 is."""
    lib, kind = _load(), _act_type(x)
    if x.dim() != 3:
        raise ValueError("x: expected [B, L, H]")
    shape, dtype, dev = x.shape, x.dtype, x.get_device()
    B, L, H = shape
    n = (L + STATE_STEPS - 1) // STATE_STEPS
    views = _views3((x, r, i, dy), x, dtype, dev, shape, ("x", "r", "i", "dy"))
    with _on(stream):
        if out is None:
            dx, dr, di = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
            outs = *_strides3(dx), *_strides3(dr), *_strides3(di)
        else:
            dx, dr, di = out
            outs = _views3(out, x, dtype, dev, shape, ("dx", "dr", "di"))
        dp = torch.empty((H,), dtype=torch.float32, device=x.device)
        dh0 = None if h0 is None else torch.empty_like(h0)
        ws = _workspace(workspace, glr_scan_backward_workspace_size(B, L, H), x)
    args = _SCAN_BACK(kind, B, L, H, scale, *views, _f32(p, (H,), dev, "p"),
                      _f32(h0, (B, H), dev, "h0"), _bytes(reset, (B, L), dev, "reset"),
                      _f32(states, (B, n, H), dev, "states"),
                      _f32(dh_last, (B, H), dev, "dh_last"), *outs, dp.data_ptr(),
                      0 if dh0 is None else dh0.data_ptr(), ws.data_ptr(), ws.numel())
    _ok("glr_scan_backward", lib.glr_scan_backward(args, _stream(stream, dev)))
    return dx, dr, di, dp, dh0


def glr_step(x, r, i, p, h, scale: float = 8.0, reset=None, h_out=None, out=None, stream=None):
    """One token of the gated linear recurrence: x, r, i [B, H], the state h [B, H] (float32),
    which becomes the next one in place unless ``h_out`` is given; reset [B] (bool or uint8)
    marks sequences that begin with this token. Returns y [B, H]."""
    lib, kind = _load(), _act_type(x)
    if x.dim() != 2:
        raise ValueError("x: expected [B, H]")
    shape, dtype, dev = x.shape, x.dtype, x.get_device()
    B, H = shape
    if out is None:
        with _on(stream):
            out = torch.empty_like(x, memory_format=torch.contiguous_format)
        yp, _, ys = out.data_ptr(), 0, H
    else:
        yp, _, ys = _views2((out,), x, dtype, dev, shape, ("out",))
    xp, _, xs, rp, _, rs, ip, _, is_ = _views2((x, r, i), x, dtype, dev, shape, ("x", "r", "i"))
    hp = _f32(h, shape, dev, "h")
    op = hp if h_out is None else _f32(h_out, shape, dev, "h_out")
    args = _STEP(kind, B, H, scale, xp, xs, 0, rp, rs, 0, ip, is_, 0, _f32(p, (H,), dev, "p"),
                 hp, _bytes(reset, (B,), dev, "reset"), yp, ys, 0, op)
    _ok("glr_step", lib.glr_step(args, _stream(stream, dev)))
    return out


class Ckpt8(NamedTuple):
    """An activation [M, H] in 8 bits: e4m3 codes [M, H] and, per group of 32 channels, the
    exponent of its power-of-two scale plus 127 [M, ceil(H / 32)] (both uint8)."""
    codes: torch.Tensor
    scales: torch.Tensor


def _new_ckpt(M, H, device) -> Ckpt8:
    return Ckpt8(torch.empty((M, H), dtype=torch.uint8, device=device),
                 torch.empty((M, (H + CKPT_GROUP - 1) // CKPT_GROUP), dtype=torch.uint8,
                             device=device))


def _ckpt_ptrs(c: Optional[Ckpt8], M, H, dev, what: str):
    if c is None:
        return 0, 0
    return (_bytes(c[0], (M, H), dev, what + " codes"),
            _bytes(c[1], (M, (H + CKPT_GROUP - 1) // CKPT_GROUP), dev, what + " scales"))


def glr_ckpt_pack(t, stream=None) -> Ckpt8:
    """t [M, H] (contiguous channels) as an 8-bit checkpoint."""
    lib, kind = _load(), _act_type(t)
    if t.dim() != 2:
        raise ValueError("t: expected [M, H]")
    dev = t.get_device()
    M, H = t.shape
    p, _, st = _views2((t,), t, t.dtype, dev, t.shape, ("t",))
    with _on(stream):
        c = _new_ckpt(M, H, t.device)
    _ok("glr_ckpt_pack", lib.glr_ckpt_pack(kind, M, H, p, st, c[0].data_ptr(), c[1].data_ptr(),
                                           _stream(stream, dev)))
    return c


def glr_ckpt_unpack(c: Ckpt8, dtype=torch.float32, out=None, stream=None):
    """The values [M, H] that an 8-bit checkpoint stands for, in ``dtype`` (or into ``out``)."""
    lib = _load()
    codes = c[0]
    if not codes.is_cuda or codes.dim() != 2:
        raise TypeError("codes: expected a CUDA tensor [M, H]")
    dev = codes.get_device()
    M, H = codes.shape
    if out is None:
        with _on(stream):
            out = torch.empty((M, H), dtype=dtype, device=codes.device)
    kind = _act_type(out)
    cp, sp = _ckpt_ptrs(c, M, H, dev, "c")
    p, _, st = _views2((out,), out, out.dtype, dev, codes.shape, ("out",))
    _ok("glr_ckpt_unpack", lib.glr_ckpt_unpack(kind, M, H, cp, sp, p, st, _stream(stream, dev)))
    return out


def glr_join(x, h, g, w, alpha, v, norm: str = "rms", act: str = "silu", eps: float = 1e-6,
             ckpt: bool = False, out=None, stream=None):
    """The end of a block and the norm that begins the next: y = x + alpha w norm(h act(g)),
    n = v norm(y), for rows x, h, g [M, H]; w, v [H] and alpha [1] float32. ``norm``: "rms" or
    "layer" (the mean taken off); ``act``: "silu", "sigmoid" or "none" (g None). v None: no next
    norm (n is None). h None: only n = v norm(x) (w, alpha, g None; y is None). ``out``: (y, n) to
    write; y may be x, and n may be h or g. Returns (y, n) and, with ``ckpt``, h and g as 8-bit
    checkpoints (Ckpt8 or None each) for glr_join_backward."""
    lib, kind = _load(), _act_type(x)
    if x.dim() != 2:
        raise ValueError("x: expected rows [M, H]")
    shape, dtype, dev = x.shape, x.dtype, x.get_device()
    M, H = shape
    if act == "none" and g is not None:
        raise ValueError('g: must be None with act="none"')
    if h is None and (g is not None or w is not None or alpha is not None or ckpt):
        raise ValueError("g, w, alpha and ckpt need h")
    views = _views2((x, h, g), x, dtype, dev, shape, ("x", "h", "g"))
    hc = gc = None
    with _on(stream):
        if out is not None:
            y, n = out
            yv, nv = _views2(out, x, dtype, dev, shape, ("y", "n")), ()
        else:
            y, yv = _new2(x, H, h is not None)
            n, nv = _new2(x, H, v is not None)
        if ckpt:
            hc = _new_ckpt(M, H, x.device)
            gc = None if g is None else _new_ckpt(M, H, x.device)
    args = _JOIN(kind, M, H, NORM[norm], ACT[act], eps, *views, _f32(w, (H,), dev, "w"),
                 _f32(alpha, (1,), dev, "alpha"), _f32(v, (H,), dev, "v"), *yv, *nv,
                 *_ckpt_ptrs(hc, M, H, dev, "h"), *_ckpt_ptrs(gc, M, H, dev, "g"))
    _ok("glr_join", lib.glr_join(args, _stream(stream, dev)))
    return (y, n, (hc, gc)) if ckpt else (y, n)


def glr_join_backward(dy, dn, x, h, g, w, alpha, v, norm: str = "rms", act: str = "silu",
                      eps: float = 1e-6, ckpt=None, out=None, workspace=None, stream=None):
    """Gradients of glr_join for the gradients dy (None: zero) of y and dn of n (given exactly
    when v is), the rest as the forward call had it. With ``ckpt`` (what glr_join returned) h and
    g come from their 8-bit checkpoints and are None here: the gradients are those at the values
    kept. ``out``: (dx, dh, dg) to write (those that exist); dx may be dy. Returns
    (dx, dh, dg, dw, dalpha, dv), None for what the call does not have."""
    lib, kind = _load(), _act_type(x)
    if x.dim() != 2:
        raise ValueError("x: expected rows [M, H]")
    shape, dtype, dev = x.shape, x.dtype, x.get_device()
    M, H = shape
    block = w is not None
    hc, gc = ckpt if ckpt is not None else (None, None)
    dw = dalpha = dv = None
    views = _views2((dy, dn, x, h, g), x, dtype, dev, shape, ("dy", "dn", "x", "h", "g"))
    with _on(stream):
        if out is not None:
            dx, dh, dg = out
            outs = _views2(out, x, dtype, dev, shape, ("dx", "dh", "dg"))
        else:
            dx, xv = _new2(x, H, True)
            dh, hv = _new2(x, H, block)
            dg, gv = _new2(x, H, block and act != "none")
            outs = *xv, *hv, *gv
        if block:
            dw = torch.empty((H,), dtype=torch.float32, device=x.device)
            dalpha = torch.empty((1,), dtype=torch.float32, device=x.device)
        if v is not None:
            dv = torch.empty((H,), dtype=torch.float32, device=x.device)
        ws = _workspace(workspace, glr_join_backward_workspace_size(M, H), x)
    args = _JOIN_BACK(kind, M, H, NORM[norm], ACT[act], eps, *views,
                      *_ckpt_ptrs(hc, M, H, dev, "h"), *_ckpt_ptrs(gc, M, H, dev, "g"),
                      _f32(w, (H,), dev, "w"), _f32(alpha, (1,), dev, "alpha"),
                      _f32(v, (H,), dev, "v"), *outs, 0 if dw is None else dw.data_ptr(),
                      0 if dalpha is None else dalpha.data_ptr(),
                      0 if dv is None else dv.data_ptr(), ws.data_ptr(), ws.numel())
    _ok("glr_join_backward", lib.glr_join_backward(args, _stream(stream, dev)))
    return dx, dh, dg, dw, dalpha, dv
