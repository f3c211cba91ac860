"""Thin Python binding over include/xent.h: the softmax cross entropy of a projection onto a
vocabulary, ``xent_loss``, and its gradients, ``xent_loss_backward``, without the logits ever being
held.

Like ``glr.py`` this module passes pointers, sizes and the current torch CUDA stream, and turns
non-zero status codes into exceptions; there is no CPU fallback. Rows and the vocabulary's weights are
float32, bfloat16 or float16 (one type) with contiguous channels, on the current device. Memory
allocated here for a call on ``stream`` belongs to that stream. Gradients are a call of their own:
nothing here is recorded for autograd.
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from . import dlr as _dlr
from .glr import _NONE3, _act_type, _f32, _ok, _on, _stream, _views2, _workspace

_lib = None
# the argument structs of xent.h, every field 8 bytes wide
_LOSS = struct.Struct("15q").pack
_BACK = struct.Struct("21q").pack
_IN_PLACE_H, _IN_PLACE_W = 16, 32  # XENT_H_IN_PLACE, XENT_W_IN_PLACE


def _load():
    global _lib
    if _lib is None:
        lib = _dlr._load()
        P, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        for name in ("xent_loss", "xent_loss_backward"):
            f = getattr(lib, name)
            f.argtypes, f.restype = [ctypes.c_char_p, P], i32
            f = getattr(lib, name + "_workspace_size")
            f.argtypes, f.restype = [i64] * 4, sz
        lib.xent_abi_version.restype = i32
        _lib = lib
    return _lib


@functools.lru_cache(maxsize=1024)
def _loss_space(kind: int, M: int, V: int, D: int) -> int:
    return int(_load().xent_loss_workspace_size(kind, M, V, D))


@functools.lru_cache(maxsize=1024)
def _back_space(kind: int, M: int, V: int, D: int) -> int:
    return int(_load().xent_loss_backward_workspace_size(kind, M, V, D))


def xent_loss_workspace_size(dtype, M: int, V: int, D: int, h=None, W=None) -> int:
    """Bytes of device workspace xent_loss needs (0: none, or sizes out of range), wherever its rows lie, or,
    with ``h`` or ``W``, for those rows: 16-bit ones that begin on 16 bytes and are a multiple of 8
    elements apart are read as they lie and need no room of their own."""
    return _loss_space(_act_kind(dtype) + _given(dtype, h, D) * _IN_PLACE_H +
                       _given(dtype, W, D) * _IN_PLACE_W, M, V, D)


def xent_loss_backward_workspace_size(dtype, M: int, V: int, D: int, W=None) -> int:
    """The same for xent_loss_backward, which always lays ``h`` out anew."""
    return _back_space(_act_kind(dtype) + _given(dtype, W, D) * _IN_PLACE_W, M, V, D)


def _given(dtype, t, D: int) -> bool:
    return t is not None and t.dtype == dtype and \
        _in_place(_act_kind(dtype), (t.data_ptr(), 0, t.stride(0)), t.shape[0], D)


def _act_kind(dtype) -> int:
    from .glr import TYPE
    if dtype not in TYPE:
        raise TypeError("expected float32, bfloat16 or float16")
    return TYPE[dtype]


def _rows(h, W):
    """(type, M, V, D, device, (pointer, 0, stride) of h and of W)."""
    kind = _act_type(h)
    if h.dim() != 2 or W.dim() != 2:
        raise ValueError("h, W: expected rows [M, D] and [V, D]")
    (M, D), V, dev = h.shape, W.shape[0], h.get_device()
    hv = _views2((h,), h, h.dtype, dev, h.shape, ("h",))
    wv = _views2((W,), h, h.dtype, dev, (V, D), ("W",))
    return kind, M, V, D, dev, hv, wv


def _in_place(kind: int, view, rows: int, D: int) -> bool:
    """Whether rows at a view (pointer, 0, stride) are read as they lie."""
    return kind != 0 and view[0] % 16 == 0 and (rows <= 1 or (view[2] % 8 == 0 and view[2] >= D))


def _target(t, M: int, dev: int) -> int:
    if t.dtype is not torch.int64 or t.get_device() != dev or not t.is_contiguous():
        raise TypeError(f"target: expected a contiguous int64 tensor on cuda:{dev}")
    if t.shape != (M,):
        raise ValueError(f"target: expected shape {(M,)}, got {tuple(t.shape)}")
    return t.data_ptr()


def xent_loss(h, W, target, workspace=None, stream=None):
    """The softmax cross entropy of the logits z = h W^T of rows h [M, D] over the vocabulary's rows
    W [V, D]: (loss [M], lse [M]), float32, with lse = log sum_v exp z and loss = lse - z[target].
    target: int64 [M]; a row whose target is outside 0 .. V-1 (-1 or -100, say) has the loss 0."""
    lib = _load()
    kind, M, V, D, dev, hv, wv = _rows(h, W)
    with _on(stream):
        loss = torch.empty((M,), dtype=torch.float32, device=h.device)
        lse = torch.empty((M,), dtype=torch.float32, device=h.device)
        space = kind + _in_place(kind, hv, M, D) * _IN_PLACE_H + _in_place(kind, wv, V, D) * _IN_PLACE_W
        ws = _workspace(workspace, _loss_space(space, M, V, D), h)
    args = _LOSS(kind, M, V, D, *hv, *wv, _target(target, M, dev), loss.data_ptr(),
                 lse.data_ptr(), ws.data_ptr(), ws.numel())
    _ok("xent_loss", lib.xent_loss(args, _stream(stream, dev)))
    return loss, lse


def xent_loss_backward(h, W, target, lse, dloss, wanted=(True, True), out=None, workspace=None,
                       stream=None):
    """Gradients (dh [M, D], dW [V, D]) of xent_loss for the gradients dloss [M] (float32) of its
    losses; h, W and target as the forward call had them, ``lse`` as it returned it. Rows without a
    target give and take nothing. ``wanted``: which of the two to form (None stands for the other);
    ``out``: (dh, dW) to write, None for one that is not wanted."""
    lib = _load()
    kind, M, V, D, dev, hv, wv = _rows(h, W)
    with _on(stream):
        if out is None:
            dh = torch.empty((M, D), dtype=h.dtype, device=h.device) if wanted[0] else None
            dW = torch.empty((V, D), dtype=h.dtype, device=h.device) if wanted[1] else None
        else:
            dh, dW = out
        space = kind + _in_place(kind, wv, V, D) * _IN_PLACE_W
        ws = _workspace(workspace, _back_space(space, M, V, D), h)
    dhv = _NONE3 if dh is None else _views2((dh,), h, h.dtype, dev, (M, D), ("dh",))
    dWv = _NONE3 if dW is None else _views2((dW,), h, h.dtype, dev, (V, D), ("dW",))
    args = _BACK(kind, M, V, D, *hv, *wv, _target(target, M, dev), _f32(lse, (M,), dev, "lse"),
                 _f32(dloss, (M,), dev, "dloss"), *dhv, *dWv, ws.data_ptr(), ws.numel())
    _ok("xent_loss_backward", lib.xent_loss_backward(args, _stream(stream, dev)))
    return dh, dW
