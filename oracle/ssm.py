"""Float64 CPU definitions of the selective state space block's operators (include/ssm.h), written
from the formulas step by step. Shares no code with the GPU path."""
import numpy as np

from .glr import _f, sigmoid, softplus


def silu(p):
    return p * sigmoid(p)


def silu_slope(p):
    s = sigmoid(p)
    return s + p * s * (1 - s)


def _seen(reset, B, L, K):
    """[B, L]: how many of the K-1 inputs before a step it sees."""
    n = np.full((B, L), K - 1)
    if reset is not None:
        for t in range(L):
            before = n[:, t - 1] + 1 if t else K - 1
            n[:, t] = np.where(np.asarray(reset)[:, t] != 0, 0, np.minimum(before, K - 1))
    return n


def conv(x, w, bias=None, state=None, reset=None, act="silu"):
    """(y [B, L, H], last [B, K-1, H], p before the activation)."""
    x, w, bias, state = _f(x), _f(w), _f(bias), _f(state)
    B, L, H = x.shape
    K = w.shape[1]
    line = np.concatenate([np.zeros((B, K - 1, H)) if state is None else state, x], 1)
    seen = _seen(reset, B, L, K)
    p = np.zeros((B, L, H)) if bias is None else np.broadcast_to(bias, (B, L, H)).copy()
    for t in range(L):
        for j in range(K):  # the input j steps before, which may be infinite where it is not seen
            p[:, t] += np.where(j <= seen[:, t, None], w[:, K - 1 - j] * line[:, t + K - 1 - j], 0.0)
    last = line[:, L:].copy()
    for j in range(K - 1):  # j + 1 steps before the next one
        if L:
            last[:, K - 2 - j] = np.where(j <= seen[:, -1, None], last[:, K - 2 - j], 0.0)
    return (silu(p) if act == "silu" else p), last, p


def conv_backward(x, w, dy, bias=None, state=None, reset=None, act="silu", dlast=None):
    """(dx, dw, dbias, dstate)."""
    _, _, p = conv(x, w, bias, state, reset, act)
    x, w, dy, state, dlast = _f(x), _f(w), _f(dy), _f(state), _f(dlast)
    B, L, H = x.shape
    K = w.shape[1]
    line = np.concatenate([np.zeros((B, K - 1, H)) if state is None else state, x], 1)
    seen = _seen(reset, B, L, K)
    g = dy * (silu_slope(p) if act == "silu" else 1.0)
    d, dw = np.zeros_like(line), np.zeros_like(w)
    for t in range(L):
        for j in range(K):
            gj = np.where(j <= seen[:, t, None], g[:, t], 0.0)
            d[:, t + K - 1 - j] += w[:, K - 1 - j] * gj
            dw[:, K - 1 - j] += np.where(gj != 0, gj * line[:, t + K - 1 - j], 0.0).sum(0)
    if dlast is not None:
        for j in range(K - 1):
            ok = j <= seen[:, -1, None] if L else True
            d[:, L + K - 2 - j] += np.where(ok, dlast[:, K - 2 - j], 0.0)
    return d[:, K - 1:], dw, g.sum((0, 1)), d[:, :K - 1]


def _grouped(m, H):
    """Maps [B, L, N] or [B, L, G, N] for each channel: [B, L, H, N]."""
    m = _f(m)
    m = m[:, :, None] if m.ndim == 3 else m
    return np.repeat(m, H // m.shape[2], axis=2)


def scan(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, sp=True, h0=None, reset=None):
    """(y [B, L, H], every state before a step [B, L, H, N], the last one [B, H, N], o)."""
    x, dt, A, D, z, dt_bias, h0 = (_f(t) for t in (x, dt, A, D, z, dt_bias, h0))
    B, L, H = x.shape
    raw = dt if dt_bias is None else dt + dt_bias
    s = softplus(raw) if sp else raw
    Bm, Cm = _grouped(Bm, H), _grouped(Cm, H)
    h = np.zeros((B, H, A.shape[1])) if h0 is None else h0.copy()
    o, before = np.empty((B, L, H)), np.empty((B, L, H, A.shape[1]))
    for t in range(L):
        if reset is not None:
            h = np.where(np.asarray(reset)[:, t, None, None] != 0, 0.0, h)
        before[:, t] = h
        h = np.exp(s[:, t, :, None] * A) * h + (s[:, t] * x[:, t])[..., None] * Bm[:, t]
        o[:, t] = (Cm[:, t] * h).sum(-1)
    if D is not None:
        o = o + D * x
    return (o if z is None else o * silu(z)), before, h, o


def scan_backward(x, dt, A, Bm, Cm, dy, D=None, z=None, dt_bias=None, sp=True, h0=None, reset=None,
                  dh_last=None):
    """(dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dh0); dB and dC [B, L, G, N]."""
    _, before, _, o = scan(x, dt, A, Bm, Cm, D, z, dt_bias, sp, h0, reset)
    G = 1 if np.ndim(Bm) == 3 else np.shape(Bm)[2]
    x, dt, A, D, z, dt_bias, dy = (_f(t) for t in (x, dt, A, D, z, dt_bias, dy))
    B, L, H = x.shape
    N = A.shape[1]
    raw = dt if dt_bias is None else dt + dt_bias
    s, slope = (softplus(raw), sigmoid(raw)) if sp else (raw, 1.0)
    Bm, Cm = _grouped(Bm, H), _grouped(Cm, H)
    g = dy if z is None else dy * silu(z)
    carry = np.zeros((B, H, N)) if dh_last is None else _f(dh_last).copy()
    q, e, dA = np.empty((B, L, H)), np.empty((B, L, H)), np.zeros((H, N))
    dB, dC = np.empty((B, L, G, N)), np.empty((B, L, G, N))
    for t in range(L - 1, -1, -1):
        a, u = np.exp(s[:, t, :, None] * A), s[:, t] * x[:, t]
        h = a * before[:, t] + u[..., None] * Bm[:, t]
        dC[:, t] = (g[:, t, :, None] * h).reshape(B, G, H // G, N).sum(2)
        carry = carry + g[:, t, :, None] * Cm[:, t]
        dB[:, t] = (carry * u[..., None]).reshape(B, G, H // G, N).sum(2)
        q[:, t] = (carry * Bm[:, t]).sum(-1)
        carry = a * carry
        if reset is not None:
            carry = np.where(np.asarray(reset)[:, t, None, None] != 0, 0.0, carry)
        r = carry * before[:, t]
        e[:, t] = (r * A).sum(-1)
        dA += (r * s[:, t, :, None]).sum(0)
    ddt = (x * q + e) * slope
    dx = s * q + (0 if D is None else D * g)
    return (dx, ddt, dA, dB, dC, None if D is None else (g * x).sum((0, 1)),
            None if z is None else dy * o * silu_slope(z), ddt.sum((0, 1)), carry)
