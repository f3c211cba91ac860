"""Thin Python binding over include/ssm.h: the operators of a selective state space block.

* ``ssm_conv`` / ``ssm_conv_backward`` / ``ssm_conv_step``: the short causal convolution before the
  scan over a sequence, its gradients, one token from the last inputs;
* ``ssm_scan`` / ``ssm_scan_backward`` / ``ssm_step``: the selective scan (N states to a channel; the
  step, the input map and the output map chosen by the token) over a sequence, its gradients, one
  token from a carried state.

Like ``glr.py`` this module passes pointers, sizes and the current torch CUDA stream, and turns
non-zero status codes into exceptions; there is no CPU fallback. Activations are float32, bfloat16
or float16 with contiguous channels and otherwise any strides (columns of one projection's output,
for example); parameters and scan states are contiguous float32, the convolution's carried inputs
contiguous activations. All are on the current device. Memory allocated here for a call on
``stream`` belongs to that stream. Gradients are calls of their own: nothing here is recorded for
autograd.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import NamedTuple, Optional

import torch

from . import dlr as _dlr
from .glr import (_NONE3, _act_type, _bytes, _f32, _ok, _on, _stream, _strides3, _views2, _views3,
                  _workspace, _wrong)

ACT = {"silu": 0, "none": 1}
STATE_STEPS = 16  # SSM_STATE_STEPS
MAX_TAPS = 8      # SSM_MAX_TAPS
MAX_STATES = 64   # SSM_MAX_STATES

_lib = None
# the argument structs of ssm.h, every field 8 bytes wide
_CONV = struct.Struct("17q").pack
_CONV_BACK = struct.Struct("25q").pack
_CONV_STEP = struct.Struct("16q").pack
_SCAN = struct.Struct("34q").pack
_SCAN_BACK = struct.Struct("53q").pack
_STEP = struct.Struct("30q").pack


def _load():
    global _lib
    if _lib is None:
        lib = _dlr._load()
        P, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        for name in ("ssm_conv", "ssm_conv_backward", "ssm_conv_step", "ssm_scan",
                     "ssm_scan_backward", "ssm_step"):
            f = getattr(lib, name)
            f.argtypes, f.restype = [ctypes.c_char_p, P], i32
        for name, n in (("ssm_conv_backward_workspace_size", 4), ("ssm_scan_workspace_size", 5),
                        ("ssm_scan_backward_workspace_size", 5)):
            f = getattr(lib, name)
            f.argtypes, f.restype = [i64] * n, sz
        lib.ssm_states.argtypes, lib.ssm_states.restype = [i64], i64
        lib.ssm_abi_version.restype = i32
        _lib = lib
    return _lib


@functools.lru_cache(maxsize=1024)
def ssm_conv_backward_workspace_size(B: int, L: int, H: int, K: int) -> int:
    """Bytes of device workspace ssm_conv_backward needs (0 for sizes out of range)."""
    return int(_load().ssm_conv_backward_workspace_size(B, L, H, K))


@functools.lru_cache(maxsize=1024)
def ssm_scan_workspace_size(B: int, L: int, H: int, N: int, G: int = 1) -> int:
    """Bytes of device workspace ssm_scan needs (0: none, or sizes out of range)."""
    return int(_load().ssm_scan_workspace_size(B, L, H, N, G))


@functools.lru_cache(maxsize=1024)
def ssm_scan_backward_workspace_size(B: int, L: int, H: int, N: int, G: int = 1) -> int:
    """Bytes of device workspace ssm_scan_backward needs (0 for sizes out of range)."""
    return int(_load().ssm_scan_backward_workspace_size(B, L, H, N, G))


def _rows(t, like, shape, what: str) -> int:
    """The pointer of a contiguous activation array, 0 for None."""
    if t is None:
        return 0
    if t.dtype != like.dtype or t.device != like.device or not t.is_contiguous():
        raise TypeError(f"{what}: expected a contiguous {like.dtype} tensor on {like.device}")
    if t.shape != shape:
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _taps(w, H: int, dev: int):
    """(pointer, K) of the taps [H, K]."""
    if w.dim() != 2:
        raise ValueError("w: expected [H, K]")
    K = w.shape[1]
    return _f32(w, (H, K), dev, "w"), K


def ssm_conv(x, w, bias=None, state=None, reset=None, act: str = "silu", out=None, stream=None):
    """The causal convolution p_t = bias + sum_j w_j x_{t-(K-1)+j} and y = act(p) over x [B, L, H]:
    w [H, K] (K <= 8) and bias [H] float32; state [B, K-1, H] the inputs before the first step (None:
    zero); reset [B, L] (bool or uint8, None: none) marks steps that begin a new sequence; ``act``
    "silu" or "none". Returns (y [B, L, H], last [B, K-1, H]), ``last`` the state that continues
    the sequence (None with K = 1)."""
    lib, kind = _load(), _act_type(x)
    if x.dim() != 3:
        raise ValueError("x: expected [B, L, H]")
    shape, dtype, dev = x.shape, x.dtype, x.get_device()
    B, L, H = shape
    wp, K = _taps(w, H, dev)
    view = _views3((x,), x, dtype, dev, shape, ("x",))
    rows = (B, K - 1, H)
    with _on(stream):
        if out is None:
            out = torch.empty((B, L, H), dtype=dtype, device=x.device)
            y = _strides3(out)
        else:
            y = _views3((out,), x, dtype, dev, shape, ("out",))
        last = torch.empty(rows, dtype=dtype, device=x.device) if K > 1 else None
    args = _CONV(kind, B, L, H, K, ACT[act], *view, wp, _f32(bias, (H,), dev, "bias"),
                 _rows(state, x, rows, "state"), _bytes(reset, (B, L), dev, "reset"), *y,
                 0 if last is None else last.data_ptr())
    _ok("ssm_conv", lib.ssm_conv(args, _stream(stream, dev)))
    return out, last


def ssm_conv_backward(x, w, dy, bias=None, state=None, reset=None, act: str = "silu", dlast=None,
                      out=None, workspace=None, stream=None):
    """Gradients of ssm_conv for the gradients dy [B, L, H] of y and dlast [B, K-1, H] (None: zero)
    of last; the other arguments as the forward call had them. ``out``: dx to write. Returns
    (dx, dw [H, K], dbias [H], dstate [B, K-1, H]), dbias and dstate None when bias and state are."""
    lib, kind = _load(), _act_type(x)
    if x.dim() != 3:
        raise ValueError("x: expected [B, L, H]")
    shape, dtype, dev = x.shape, x.dtype, x.get_device()
    B, L, H = shape
    wp, K = _taps(w, H, dev)
    views = _views3((x, dy), x, dtype, dev, shape, ("x", "dy"))
    rows = (B, K - 1, H)
    with _on(stream):
        if out is None:
            out = torch.empty((B, L, H), dtype=dtype, device=x.device)
            dx = _strides3(out)
        else:
            dx = _views3((out,), x, dtype, dev, shape, ("out",))
        dw = torch.empty_like(w)
        dbias = None if bias is None else torch.empty_like(bias)
        dstate = None if state is None else torch.empty_like(state)
        ws = _workspace(workspace, ssm_conv_backward_workspace_size(B, L, H, K), x)
    args = _CONV_BACK(kind, B, L, H, K, ACT[act], *views, wp, _f32(bias, (H,), dev, "bias"),
                      _rows(state, x, rows, "state"), _bytes(reset, (B, L), dev, "reset"),
                      _rows(dlast, x, rows, "dlast"), *dx, dw.data_ptr(),
                      0 if dbias is None else dbias.data_ptr(),
                      0 if dstate is None else dstate.data_ptr(), ws.data_ptr(), ws.numel())
    _ok("ssm_conv_backward", lib.ssm_conv_backward(args, _stream(stream, dev)))
    return out, dw, dbias, dstate


def ssm_conv_step(x, w, state, bias=None, reset=None, act: str = "silu", state_out=None, out=None,
                  stream=None):
    """One token of the causal convolution: x [B, H], the last inputs state [B, K-1, H] (None with
    K = 1), which become the next ones in place unless ``state_out`` is given; reset [B] (bool or
    uint8) marks sequences that begin with this token. Returns y [B, H]."""
    lib, kind = _load(), _act_type(x)
    if x.dim() != 2:
        raise ValueError("x: expected [B, H]")
    shape, dtype, dev = x.shape, x.dtype, x.get_device()
    B, H = shape
    wp, K = _taps(w, H, dev)
    if out is None:
        with _on(stream):
            out = torch.empty((B, H), dtype=dtype, device=x.device)
    xp, _, xs, yp, _, ys = _views2((x, out), x, dtype, dev, shape, ("x", "out"))
    rows = (B, K - 1, H)
    sp = _rows(state, x, rows, "state")
    op = sp if state_out is None else _rows(state_out, x, rows, "state_out")
    args = _CONV_STEP(kind, B, H, K, ACT[act], xp, xs, 0, wp, _f32(bias, (H,), dev, "bias"), sp,
                      _bytes(reset, (B,), dev, "reset"), yp, ys, 0, op)
    _ok("ssm_conv_step", lib.ssm_conv_step(args, _stream(stream, dev)))
    return out


def _maps(ts, like, B, L, H, dev, what):
    """(G, N) and the views (pointer, stride_b, stride_t) of maps [B, L, N] (one group) or
    [B, L, G, N], all of one shape."""
    shape = ts[0].shape
    if len(shape) not in (3, 4) or shape[0] != B or shape[1] != L:
        raise ValueError(f"{what[0]}: expected [{B}, {L}, N] or [{B}, {L}, G, N], got {tuple(shape)}")
    N, G = shape[-1], (1 if len(shape) == 3 else shape[2])
    if G < 1 or N < 1 or H % G:
        raise ValueError(f"{what[0]}: {G} groups of {N} states do not divide {H} channels")
    out = []
    for t, name in zip(ts, what):
        if t.dtype is not like.dtype or t.get_device() != dev or t.shape != shape:
            _wrong(t, like, shape, name)
        s = t.stride()
        if (s[-1] != 1 and N > 1) or (len(s) == 4 and G > 1 and s[2] != N):
            raise ValueError(f"{name}: groups and states must be contiguous")
        out += (t.data_ptr(), s[0], s[1])
    return G, N, out


def _maps_step(ts, like, B, H, dev, what):
    """The same for one token: [B, N] or [B, G, N]."""
    shape, dtype, out = ts[0].shape, like.dtype, []
    if len(shape) == 2:
        G, N = 1, shape[1]
    elif len(shape) == 3:
        G, N = shape[1], shape[2]
    else:
        raise ValueError(f"{what[0]}: expected [{B}, N] or [{B}, G, N], got {tuple(shape)}")
    if shape[0] != B or G < 1 or N < 1 or H % G:
        raise ValueError(f"{what[0]}: {tuple(shape)} for {B} entries of {H} channels")
    for t in ts:
        s = t.stride()
        if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or \
                (s[-1] != 1 and N > 1) or (G > 1 and s[1] != N):
            _wrong(t, like, shape, what[len(out) // 3])
        out += (t.data_ptr(), s[0], 0)
    return G, N, out


def ssm_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus: bool = True, h0=None,
             reset=None, save_states: bool = False, out=None, workspace=None, stream=None):
    """The selective scan over x and dt [batch, L, H]: with s = softplus(dt + dt_bias) (``softplus``
    False: dt + dt_bias), h_t = exp(s A) h_{t-1} + s x B_t and o = sum_n C_t h_t + D x, y = o silu(z).
    A [H, N] (N <= 64) and dt_bias, D [H] float32; B, C [batch, L, N] or [batch, L, G, N] for G
    groups of H / G channels; z [batch, L, H] (None: no gate); h0 [batch, H, N] the state before the
    first step (None: zero); reset [batch, L] (bool or uint8, None: none) marks steps that begin a new
    sequence. Returns (y, h_last [batch, H, N]) and, with ``save_states``, the float32 states
    [batch, ceil(L / 16), H, N] that ssm_scan_backward takes. The decays of 16-bit activations are off by up
    to 1.5 * 2^-24: states with a memory of thousands of steps by 1e-7 for each of them."""
    lib, kind = _load(), _act_type(x)
    if x.dim() != 3:
        raise ValueError("x: expected [batch, L, H]")
    shape, dtype, dev = x.shape, x.dtype, x.get_device()
    b, L, H = shape
    views = _views3((x, dt), x, dtype, dev, shape, ("x", "dt"))
    zv = _NONE3 if z is None else _views3((z,), x, dtype, dev, shape, ("z",))
    G, N, maps = _maps((B, C), x, b, L, H, dev, ("B", "C"))
    with _on(stream):
        if out is None:
            out = torch.empty((b, L, H), dtype=dtype, device=x.device)
            y = _strides3(out)
        else:
            y = _views3((out,), x, dtype, dev, shape, ("out",))
        h_last = torch.empty((b, H, N), dtype=torch.float32, device=x.device)
        states = torch.empty((b, (L + STATE_STEPS - 1) // STATE_STEPS, H, N), dtype=torch.float32,
                             device=x.device) if save_states else None
        ws = _workspace(workspace, ssm_scan_workspace_size(b, L, H, N, G), x)
    args = _SCAN(kind, b, L, H, N, G, bool(softplus), *views, *zv, *maps,
                 _f32(A, (H, N), dev, "A"), _f32(D, (H,), dev, "D"),
                 _f32(dt_bias, (H,), dev, "dt_bias"), _f32(h0, (b, H, N), dev, "h0"),
                 _bytes(reset, (b, L), dev, "reset"), *y, h_last.data_ptr(),
                 0 if states is None else states.data_ptr(), ws.data_ptr(), ws.numel())
    _ok("ssm_scan", lib.ssm_scan(args, _stream(stream, dev)))
    return (out, h_last, states) if save_states else (out, h_last)


class ScanGrads(NamedTuple):
    """What ssm_scan_backward returns; None for what the call does not have."""
    dx: torch.Tensor
    ddt: torch.Tensor
    dA: torch.Tensor
    dB: torch.Tensor
    dC: torch.Tensor
    dD: Optional[torch.Tensor]
    dz: Optional[torch.Tensor]
    ddt_bias: Optional[torch.Tensor]
    dh0: Optional[torch.Tensor]


def ssm_scan_backward(x, dt, A, B, C, dy, states, D=None, z=None, dt_bias=None,
                      softplus: bool = True, h0=None, reset=None, dh_last=None, out=None,
                      workspace=None, stream=None) -> ScanGrads:
    """Gradients of ssm_scan for the gradients dy [batch, L, H] of y and dh_last [batch, H, N] (None:
    zero) of h_last; the other arguments as the forward call had them, ``states`` as it returned
    them. ``out``: (dx, ddt, dB, dC, dz) to write (dz None without a gate), e.g. columns of the
    projections' gradients. dD, dz, ddt_bias and dh0 are None when D, z, dt_bias and h0 are."""
    lib, kind = _load(), _act_type(x)
    if x.dim() != 3:
        raise ValueError("x: expected [batch, L, H]")
    shape, dtype, dev = x.shape, x.dtype, x.get_device()
    b, L, H = shape
    views = _views3((x, dt), x, dtype, dev, shape, ("x", "dt"))
    zv = _NONE3 if z is None else _views3((z,), x, dtype, dev, shape, ("z",))
    yv = _views3((dy,), x, dtype, dev, shape, ("dy",))
    G, N, maps = _maps((B, C), x, b, L, H, dev, ("B", "C"))
    n = (L + STATE_STEPS - 1) // STATE_STEPS
    with _on(stream):
        if out is None:
            dx, ddt = (torch.empty((b, L, H), dtype=dtype, device=x.device) for _ in range(2))
            dz = None if z is None else torch.empty((b, L, H), dtype=dtype, device=x.device)
            dB, dC = (torch.empty(B.shape, dtype=dtype, device=x.device) for _ in range(2))
        else:
            dx, ddt, dB, dC, dz = out
        if (dz is None) != (z is None):
            raise ValueError("dz: given exactly when z is")
        outs = _views3((dx, ddt), x, dtype, dev, shape, ("dx", "ddt"))
        dzv = _NONE3 if dz is None else _views3((dz,), x, dtype, dev, shape, ("dz",))
        dmaps = _maps((dB, dC), x, b, L, H, dev, ("dB", "dC"))
        if dmaps[:2] != (G, N):
            raise ValueError(f"dB: expected the shape of B, {tuple(B.shape)}")
        dA = torch.empty_like(A)
        dD = None if D is None else torch.empty_like(D)
        dbias = None if dt_bias is None else torch.empty_like(dt_bias)
        dh0 = None if h0 is None else torch.empty_like(h0)
        ws = _workspace(workspace, ssm_scan_backward_workspace_size(b, L, H, N, G), x)
    at = lambda t: 0 if t is None else t.data_ptr()
    args = _SCAN_BACK(kind, b, L, H, N, G, bool(softplus), *views, *zv, *maps, *yv,
                      _f32(A, (H, N), dev, "A"), _f32(D, (H,), dev, "D"),
                      _f32(dt_bias, (H,), dev, "dt_bias"), _f32(h0, (b, H, N), dev, "h0"),
                      _bytes(reset, (b, L), dev, "reset"),
                      _f32(states, (b, n, H, N), dev, "states"),
                      _f32(dh_last, (b, H, N), dev, "dh_last"), *outs, *dzv, *dmaps[2],
                      dA.data_ptr(), at(dD), at(dbias), at(dh0), ws.data_ptr(), ws.numel())
    _ok("ssm_scan_backward", lib.ssm_scan_backward(args, _stream(stream, dev)))
    return ScanGrads(dx, ddt, dA, dB, dC, dD, dz, dbias, dh0)


def ssm_step(x, dt, A, B, C, h, D=None, z=None, dt_bias=None, softplus: bool = True, reset=None,
             h_out=None, out=None, stream=None):
    """One token of the selective scan: x, dt (and z) [batch, H], B, C [batch, N] or [batch, G, N],
    the state h [batch, H, N] (float32), which becomes the next one in place unless ``h_out`` is
    given; reset [batch] (bool or uint8) marks sequences that begin with this token. Returns
    y [batch, H]."""
    lib, kind = _load(), _act_type(x)
    if x.dim() != 2:
        raise ValueError("x: expected [batch, H]")
    shape, dtype, dev = x.shape, x.dtype, x.get_device()
    b, H = shape
    if out is None:
        with _on(stream):
            out = torch.empty((b, H), dtype=dtype, device=x.device)
    xp, _, xs, dp, _, ds, zp, _, zs, yp, _, ys = _views2((x, dt, z, out), x, dtype, dev, shape,
                                                         ("x", "dt", "z", "out"))
    G, N, maps = _maps_step((B, C), x, b, H, dev, ("B", "C"))
    hp = _f32(h, (b, H, N), dev, "h")
    op = hp if h_out is None else _f32(h_out, (b, H, N), dev, "h_out")
    args = _STEP(kind, b, H, N, G, bool(softplus), xp, xs, 0, dp, ds, 0, zp, zs, 0, *maps,
                 _f32(A, (H, N), dev, "A"), _f32(D, (H,), dev, "D"),
                 _f32(dt_bias, (H,), dev, "dt_bias"), hp, _bytes(reset, (b,), dev, "reset"), yp,
                 ys, 0, op)
    _ok("ssm_step", lib.ssm_step(args, _stream(stream, dev)))
    return out
