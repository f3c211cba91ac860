"""Float64 CPU definition of the softmax cross entropy over a vocabulary (include/xent.h), written from
the formula. Shares no code with the GPU path."""
import numpy as np

from .glr import _f


def loss(h, W, target):
    """(loss [M], lse [M], logits [M, V])."""
    h, W, target = _f(h), _f(W), np.asarray(target)
    z = h @ W.T
    top = z.max(1, keepdims=True)
    lse = (top + np.log(np.exp(z - top).sum(1, keepdims=True)))[:, 0]
    out = np.zeros(len(h))
    for m, t in enumerate(target):
        if 0 <= t < len(W):
            out[m] = lse[m] - z[m, t]
    return out, lse, z


def loss_backward(h, W, target, dloss):
    """(dh, dW)."""
    counts = [m for m, t in enumerate(np.asarray(target)) if 0 <= t < len(W)]
    dh, dW = np.zeros(np.shape(h)), np.zeros(np.shape(W))
    if not counts:
        return dh, dW
    hc, W, t = _f(h)[counts], _f(W), np.asarray(target)[counts]
    _, lse, z = loss(hc, W, t)
    d = np.exp(z - lse[:, None])
    d[np.arange(len(t)), t] -= 1.0
    d *= _f(dloss)[counts][:, None]
    dh[counts] = d @ W
    return dh, d.T @ hc
