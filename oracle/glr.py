"""Float64 CPU definitions of the gated recurrent block's operators (include/glr.h), written from
the formulas: the recurrence step by step, the join row by row, the 8-bit checkpoints value by
value. Shares no code with the GPU path."""
import numpy as np

GROUP = 32


def _f(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def softplus(v):
    return np.logaddexp(0.0, v)


def scan(x, r, i, p, c, h0=None, reset=None):
    """y [B, L, H] and every state before a step [B, L, H], and the last one [B, H]."""
    x, r, i, p, h0 = _f(x), _f(r), _f(i), _f(p), _f(h0)
    B, L, H = x.shape
    z = -c * softplus(p) * sigmoid(r)
    a, m = np.exp(z), np.sqrt(-np.expm1(2 * z))
    b = m * sigmoid(i) * x
    s = np.zeros((B, H)) if h0 is None else h0.copy()
    y, before = np.empty((B, L, H)), np.empty((B, L, H))
    for t in range(L):
        if reset is not None:
            s = np.where(np.asarray(reset)[:, t, None] != 0, 0.0, s)
        before[:, t] = s
        s = a[:, t] * s + b[:, t]
        y[:, t] = s
    return y, before, s


def scan_backward(x, r, i, p, c, dy, h0=None, reset=None, dh_last=None):
    """(dx, dr, di, dp, dh0)."""
    _, before, _ = scan(x, r, i, p, c, h0, reset)
    x, r, i, p, dy = _f(x), _f(r), _f(i), _f(p), _f(dy)
    B, L, H = x.shape
    k, sr, si = c * softplus(p), sigmoid(r), sigmoid(i)
    z = -k * sr
    a, m = np.exp(z), np.sqrt(-np.expm1(2 * z))
    G = np.zeros((B, H)) if dh_last is None else _f(dh_last).copy()
    dx, dr, di, dp = np.empty_like(x), np.empty_like(x), np.empty_like(x), np.zeros(H)
    for t in range(L - 1, -1, -1):
        G = G + dy[:, t]
        with np.errstate(divide="ignore", invalid="ignore"):
            # a^2 / m sigmoid(r): 0 in the limit sigmoid(r) -> 0
            q = np.where(m[:, t] > 0, a[:, t] ** 2 / m[:, t] * sr[:, t], 0.0)
        Es = G * (a[:, t] * before[:, t] * sr[:, t] - q * si[:, t] * x[:, t])
        dx[:, t] = G * m[:, t] * si[:, t]
        di[:, t] = G * m[:, t] * x[:, t] * si[:, t] * (1 - si[:, t])
        dr[:, t] = -k * Es * (1 - sr[:, t])
        dp += -c * sigmoid(p) * Es.sum(0)
        G = a[:, t] * G
        if reset is not None:
            G = np.where(np.asarray(reset)[:, t, None] != 0, 0.0, G)
    return dx, dr, di, dp, G


def norm(z, kind, eps):
    """(normalised rows, 1 / deviation)."""
    if kind == "layer":
        z = z - z.mean(1, keepdims=True)
    s = 1.0 / np.sqrt((z * z).mean(1, keepdims=True) + eps)
    return z * s, s


def act(g, kind):
    """(act(g), its derivative); (1, 0) without a gate."""
    if kind == "none":
        return 1.0, 0.0
    s = sigmoid(g)
    return (g * s, s + g * s * (1 - s)) if kind == "silu" else (s, s * (1 - s))


def join(x, h, g, w, alpha, v, kind="rms", gate="silu", eps=1e-6):
    """(y, n); y None without h, n None without v."""
    x, h, g, w, v = _f(x), _f(h), _f(g), _f(w), _f(v)
    y = x
    if h is not None:
        y = x + float(alpha) * w * norm(h * act(g, gate)[0], kind, eps)[0]
    return (None if h is None else y), (None if v is None else v * norm(y, kind, eps)[0])


def join_backward(dy, dn, x, h, g, w, alpha, v, kind="rms", gate="silu", eps=1e-6):
    """(dx, dh, dg, dw, dalpha, dv), None for what the call does not have."""
    x, h, g, w, v, dy, dn = _f(x), _f(h), _f(g), _f(w), _f(v), _f(dy), _f(dn)

    def behind(q, zh, s):
        d = q - zh * (q * zh).mean(1, keepdims=True)
        return s * (d - q.mean(1, keepdims=True) if kind == "layer" else d)
    y = x
    if h is not None:
        a, slope = act(g, gate)
        uh, us = norm(h * a, kind, eps)
        y = x + float(alpha) * w * uh
    D = np.zeros_like(x) if dy is None else dy
    dv = None
    if v is not None:
        yh, ys = norm(y, kind, eps)
        D = D + behind(v * dn, yh, ys)
        dv = (dn * yh).sum(0)
    if h is None:
        return D, None, None, None, None, dv
    du = behind(float(alpha) * w * D, uh, us)
    per = (D * uh).sum(0)
    return (D, du * a, None if gate == "none" else du * h * slope, float(alpha) * per,
            np.array([(w * per).sum()]), dv)


# the finite values of e4m3: 4 exponent bits (bias 7), 3 mantissa bits, subnormals below 2^-6
E4M3 = np.array([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7)
                 for e in range(16) for m in range(8)][:127])


def ckpt_pack(t):
    """(codes, scale bytes, values) of an 8-bit checkpoint, by search over e4m3's values."""
    t = _f(t)
    M, H = t.shape
    n = -(-H // GROUP)
    codes, scales, values = np.zeros((M, H), np.uint8), np.zeros((M, n), np.uint8), np.zeros((M, H))
    for j in range(n):
        s = slice(j * GROUP, min(H, (j + 1) * GROUP))
        z = t[:, s]
        top = np.max(np.where(np.isfinite(z), np.abs(z), 0.0), axis=1, keepdims=True)
        e = np.full(top.shape, -127)
        while (top > 448 * 2.0 ** e).any():
            e = np.where(top > 448 * 2.0 ** e, e + 1, e)
        q = np.abs(np.where(np.isfinite(z), z, 0.0)) / 2.0 ** e
        hi = np.clip(np.searchsorted(E4M3, q), 1, 126)
        lo = hi - 1
        dl, dh = q - E4M3[lo], E4M3[hi] - q
        k = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)  # ties to the even code
        k = np.where(np.isfinite(z), k, 127)
        neg = np.signbit(z) & np.isfinite(z)
        codes[:, s] = k + 128 * neg
        scales[:, j] = (e + 127)[:, 0]
        values[:, s] = np.where(np.isfinite(z), E4M3[np.minimum(k, 126)] * 2.0 ** e *
                                np.where(neg, -1, 1), np.nan)
    return codes, scales, values
