"""The recurrent block's operators: what is timed, their plain forms, and their definitions in 64 bits.

Three operators that stand together in a recurrent block of a language model:

* the gated linear recurrence over a sequence (forward, training step, and one token from a carried state),
* the block's join: gate, norm, residual scale and add, and the next block's norm (forward and training step),
* activation checkpoints in 8 bits (groups of 32 with a power-of-two scale), kept by the join's forward and read by its
  backward, or packed and unpacked alone.

`run` computes a case in elementary torch operations in 32 bits, or, where `own` is true, by the framework's calls.
"""
import math

import numpy as np
import torch

own = False

SCALE = 8.0   # c of a = exp(-c softplus(p) sigmoid(r))
EPS = 1e-6
GROUP = 32    # values that share a scale in an 8-bit checkpoint
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
MOST = 4 * 16384 * 2048  # elements of the largest training case


def listed():
    return [
        # one token of one stream: nothing but latency
        {"name": "step_one_stream", "op": "step", "B": 1, "H": 512, "type": "bf16"},
        # one token of each sequence of a full serving batch
        {"name": "step_batch", "op": "step", "B": 256, "H": 4096, "type": "bf16"},
        # a short prompt of odd length that continues a carried state
        {"name": "scan_prompt", "op": "scan", "B": 1, "L": 333, "H": 512, "type": "bf16", "h0": True, "docs": 0, "fused": True},
        # one very long sequence over few channels (the long bank's sizes)
        {"name": "scan_long", "op": "scan", "B": 1, "L": 65536, "H": 256, "type": "f32", "h0": False, "docs": 0, "fused": False},
        # a training step of the bank's sizes, several documents packed into each row
        {"name": "train_packed", "op": "train", "B": 8, "L": 4096, "H": 256, "type": "bf16", "h0": False, "docs": 5, "fused": True},
        # odd sizes in 32 bits, with a state carried in and its gradient
        {"name": "train_odd", "op": "train", "B": 3, "L": 1021, "H": 131, "type": "f32", "h0": True, "docs": 3, "fused": False},
        # a training step at a language model's width and a long context: the largest
        {"name": "train_wide", "op": "train", "B": 4, "L": 16384, "H": 2048, "type": "bf16", "h0": False, "docs": 0, "fused": True},
        # the join of a few decoded tokens
        {"name": "join_decode", "op": "join", "M": 16, "H": 2048, "type": "bf16", "norm": "rms", "act": "silu"},
        # its training step over a batch of long rows
        {"name": "join_train", "op": "join_train", "M": 32768, "H": 2048, "type": "bf16", "norm": "rms", "act": "silu"},
        # the same in 32 bits with mean-centred norms and a sigmoid gate, at an odd width
        {"name": "join_train_odd", "op": "join_train", "M": 8191, "H": 515, "type": "f32", "norm": "layer", "act": "sigmoid"},
        # a training step that keeps the gate's two inputs in 8 bits
        {"name": "ckpt_train", "op": "ckpt_train", "M": 65536, "H": 1024, "type": "bf16", "norm": "rms", "act": "silu"},
        # one activation of ragged width packed and read back
        {"name": "ckpt_pack", "op": "ckpt_pack", "M": 2041, "H": 1000, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "scan", "scan", "train", "train", "join", "join_train", "join_train", "ckpt_train", "ckpt_pack"])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    H = _log(rng, 16, 4096)
    if rng.random() < 0.7:
        H = max(16, H // 16 * 16)
    if op == "step":
        return {"op": op, "B": _log(rng, 1, 512), "H": H, "type": kind}
    if op in ("scan", "train"):
        B = _log(rng, 1, 16)
        L = _log(rng, 1, max(1, min(65536, MOST // (2 * B * H))))
        return {"op": op, "B": B, "L": L, "H": H, "type": kind, "h0": rng.random() < 0.5, "docs": rng.choice([0, 0, 3, 17]) if L > 64 else 0,
                "fused": rng.random() < 0.5}
    M = _log(rng, 1, min(131072, MOST // (2 * H)))
    c = {"op": op, "M": M, "H": H, "type": kind}
    if op != "ckpt_pack":
        c["norm"] = rng.choice(["rms", "layer"])
        c["act"] = rng.choice(["silu", "sigmoid"])
    elif kind == "f16":
        c["type"] = "bf16"  # a checkpoint's values span more than f16's range
    return c


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype, H = TYPES[case["type"]], case["H"]

    def normal(*shape, dtype=dtype):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)

    s = dict(case)
    if case["op"] in ("step", "scan", "train"):
        B, L = case["B"], case.get("L", 1)
        if case.get("fused"):  # the three are columns of one projection's output
            z = normal(B, L, 3 * H)
            s["x"], s["r"], s["i"] = z[..., :H], z[..., H:2 * H], z[..., 2 * H:]
        else:
            s["x"], s["r"], s["i"] = (normal(B, L, H) for _ in range(3))
        # decays spread over memories of some tens to some thousands of steps
        a0 = torch.rand(H, generator=gen, device="cuda") * (0.9995 - 0.9) + 0.9
        s["p"] = torch.log(torch.expm1(-torch.log(a0)))
        if case["op"] == "step":
            s["x"], s["r"], s["i"] = (s[n][:, 0] for n in "xri")
            s["h"] = normal(B, H, dtype=torch.float32)
            s["h_out"] = torch.empty_like(s["h"])
            return s
        s["h0"] = normal(B, H, dtype=torch.float32) if case["h0"] else None
        s["reset"] = None
        if case["docs"]:  # where documents begin in the packed rows
            at = torch.rand(B, case["docs"], generator=gen, device="cuda").mul(L).long()
            s["reset"] = torch.zeros(B, L, dtype=torch.bool, device="cuda")
            s["reset"].scatter_(1, at, True)
        if case["op"] == "train":
            s["dy"] = normal(B, L, H)
            s["dh_last"] = normal(B, H, dtype=torch.float32) if case["h0"] else None
        return s
    M = case["M"]
    if case["op"] == "ckpt_pack":
        # activations with a few channels far larger than the rest
        big = torch.exp(2.0 * torch.randn(H, generator=gen, device="cuda"))
        s["t"] = (normal(M, H, dtype=torch.float32) * big).to(dtype)
        return s
    for n in "xhg":
        s[n] = normal(M, H)
    for n in "wv":
        s[n] = 1.0 + 0.1 * normal(H, dtype=torch.float32)
    s["alpha"] = torch.full((1,), 0.4, device="cuda")
    if case["op"] != "join":
        s["dy"], s["dn"] = normal(M, H), normal(M, H)
    return s


# ---- the plain forms ---------------------------------------------------------------------------


def _sigmoid(t):
    return 1.0 / (1.0 + torch.exp(-t))


def _gates(s):
    x, sr, si = s["x"].float(), _sigmoid(s["r"].float()), _sigmoid(s["i"].float())
    k = SCALE * torch.log1p(torch.exp(s["p"]))
    log_a = -k * sr
    a, m = torch.exp(log_a), torch.sqrt(-torch.expm1(2.0 * log_a))
    return x, sr, si, k, a, m


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 1, by doubling the span that each entry covers."""
    d, L = 1, a.shape[1]
    while d < L:
        b = torch.cat([b[:, :d], b[:, d:] + a[:, d:] * b[:, :-d]], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return b


def _plain_scan(s):
    x, sr, si, k, a, m = _gates(s)
    abar = a if s["reset"] is None else torch.where(s["reset"][..., None], torch.zeros_like(a), a)
    b = m * si * x
    if s["h0"] is not None:
        b = torch.cat([b[:, :1] + abar[:, :1] * s["h0"][:, None], b[:, 1:]], 1)
    h = _scan(abar, b)
    y, h_last = h.to(s["x"].dtype), h[:, -1].clone()
    if s["op"] == "scan":
        return y, h_last
    first = torch.zeros_like(h[:, :1]) if s["h0"] is None else s["h0"][:, None]
    prev = torch.cat([first, h[:, :-1]], 1)
    g = s["dy"].float()
    if s["dh_last"] is not None:
        g = torch.cat([g[:, :-1], g[:, -1:] + s["dh_last"][:, None]], 1)
    after = torch.cat([abar[:, 1:], torch.zeros_like(a[:, :1])], 1)
    g = _scan(after.flip(1), g.flip(1)).flip(1)
    e = g * (abar * prev - a * a / m * (si * x))
    dx = g * (m * si)
    di = g * (m * x * si * (1.0 - si))
    dr = -k * e * sr * (1.0 - sr)
    dp = -SCALE * _sigmoid(s["p"]) * (e * sr).sum((0, 1))
    t = s["x"].dtype
    out = [y, h_last, dx.to(t), dr.to(t), di.to(t), dp]
    return out + [abar[:, 0] * g[:, 0]] if s["h0"] is not None else out


def _plain_step(s):
    x, sr, si, k, a, m = _gates(s)
    h = a * s["h"] + m * si * x
    return h.to(s["x"].dtype), h


def _act(kind, g):
    """The gate and its derivative."""
    sg = _sigmoid(g)
    return (g * sg, sg * (1.0 + g * (1.0 - sg))) if kind == "silu" else (sg, sg * (1.0 - sg))


def _norm(kind, z):
    if kind == "layer":
        z = z - z.mean(1, keepdim=True)
    rstd = torch.rsqrt((z * z).mean(1, keepdim=True) + EPS)
    return z * rstd, rstd


def _norm_grad(kind, q, z, rstd):
    d = q - z * (q * z).mean(1, keepdim=True)
    if kind == "layer":
        d = d - q.mean(1, keepdim=True)
    return rstd * d


def _plain_pack(t):
    """The values that t's 8-bit checkpoint stands for."""
    M, H = t.shape
    n = -(-H // GROUP)
    z = torch.zeros(M, n * GROUP, device=t.device)
    z[:, :H] = t.float()
    z = z.reshape(M, n, GROUP)
    mant, e = torch.frexp(z.abs().amax(2, keepdim=True))
    s = torch.where(mant <= 0.875, e - 9, e - 8).clamp(-127, 127)
    q = torch.ldexp(z, -s).to(torch.float8_e4m3fn).float()
    return torch.ldexp(q, s).reshape(M, n * GROUP)[:, :H]


def _plain_join(s):
    x, h, g, w, v, al = (s[n].float() for n in ("x", "h", "g", "w", "v", "alpha"))
    t = s["x"].dtype

    def forward(h, g):
        act, slope = _act(s["act"], g)
        un, ru = _norm(s["norm"], h * act)
        y = x + al * w * un
        yn, ry = _norm(s["norm"], y)
        return act, slope, un, ru, y, yn, ry

    act, slope, un, ru, y, yn, ry = forward(h, g)
    out = [y.to(t), (v * yn).to(t)]
    if s["op"] == "join":
        return out
    if s["op"] == "ckpt_train":  # the backward pass has the values that were kept
        h, g = _plain_pack(s["h"]), _plain_pack(s["g"])
        act, slope, un, ru, y, yn, ry = forward(h, g)
    dn = s["dn"].float()
    d = s["dy"].float() + _norm_grad(s["norm"], v * dn, yn, ry)
    du = _norm_grad(s["norm"], al * w * d, un, ru)
    per = (d * un).sum(0)
    return out + [d.to(t), (du * act).to(t), (du * h * slope).to(t), al * per, (w * per).sum().reshape(1), (dn * yn).sum(0)]


def _plain(s):
    if s["op"] == "step":
        return _plain_step(s)
    if s["op"] in ("scan", "train"):
        return _plain_scan(s)
    if s["op"] == "ckpt_pack":
        return _plain_pack(s["t"]).to(s["t"].dtype)
    return _plain_join(s)


def _own(s):
    from state_space_sequence_gb300 import glr
    op = s["op"]
    if op == "step":
        y = glr.glr_step(s["x"], s["r"], s["i"], s["p"], s["h"], scale=SCALE, h_out=s["h_out"])
        return y, s["h_out"]
    if op == "scan":
        return glr.glr_scan(s["x"], s["r"], s["i"], s["p"], scale=SCALE, h0=s["h0"], reset=s["reset"])
    if op == "train":
        y, h_last, states = glr.glr_scan(s["x"], s["r"], s["i"], s["p"], scale=SCALE, h0=s["h0"], reset=s["reset"], save_states=True)
        out = None
        if s["fused"]:  # the gradients of the projection's output, in its own layout
            B, L, H = s["x"].shape
            dz = torch.empty(B, L, 3 * H, dtype=s["x"].dtype, device="cuda")
            out = (dz[..., :H], dz[..., H:2 * H], dz[..., 2 * H:])
        dx, dr, di, dp, dh0 = glr.glr_scan_backward(s["x"], s["r"], s["i"], s["p"], s["dy"], states, scale=SCALE, h0=s["h0"],
                                                    reset=s["reset"], dh_last=s["dh_last"], out=out)
        return [y, h_last, dx, dr, di, dp] + ([dh0] if dh0 is not None else [])
    if op == "ckpt_pack":
        return glr.glr_ckpt_unpack(glr.glr_ckpt_pack(s["t"]), dtype=s["t"].dtype)
    args = (s["x"], s["h"], s["g"], s["w"], s["alpha"], s["v"])
    how = {"norm": s["norm"], "act": s["act"], "eps": EPS}
    if op == "join":
        return list(glr.glr_join(*args, **how))
    if op == "join_train":
        y, n = glr.glr_join(*args, **how)
        return [y, n, *glr.glr_join_backward(s["dy"], s["dn"], *args, **how)]
    y, n, kept = glr.glr_join(*args, ckpt=True, **how)
    return [y, n, *glr.glr_join_backward(s["dy"], s["dn"], s["x"], None, None, s["w"], s["alpha"], s["v"], ckpt=kept, **how)]


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    e, H, op = BYTES[case["type"]], case["H"], case["op"]
    if op == "step":
        n = case["B"] * H
        return {"bytes": 4 * e * n + 8 * n + 4 * H, "flops": 25 * n}
    if op in ("scan", "train"):
        B, n = case["B"], case["B"] * case["L"] * H
        mask = B * case["L"] if case["docs"] else 0
        got = {"bytes": 4 * e * n + 4 * H + (2 if case["h0"] else 1) * 4 * B * H + mask, "flops": 25 * n}
        if op == "train":
            got["bytes"] += 7 * e * n + 8 * H + (3 * 4 * B * H if case["h0"] else 0) + mask
            got["flops"] += 60 * n
        return got
    n = case["M"] * H
    kept = n + case["M"] * -(-H // GROUP)
    if op == "ckpt_pack":
        return {"bytes": 2 * e * n + 2 * kept, "flops": 6 * n}
    got = {"bytes": 5 * e * n + 8 * H, "flops": 20 * n}
    if op == "join_train":
        got = {"bytes": 13 * e * n + 24 * H, "flops": 65 * n}
    elif op == "ckpt_train":
        got = {"bytes": 11 * e * n + 4 * kept + 24 * H, "flops": 75 * n}
    return got


# ---- the definitions in 64 bits ------------------------------------------------------------------


def _exact_scan(s):
    f = {n: s[n].double().cpu().numpy() for n in ("x", "r", "i", "p")}
    one = s["op"] == "step"
    x, r, i = (f[n][:, None] if one else f[n] for n in "xri")
    B, L, H = x.shape
    si, sr = 1 / (1 + np.exp(-i)), 1 / (1 + np.exp(-r))
    k = SCALE * np.logaddexp(0.0, f["p"])
    a = np.exp(-k * sr)
    m = np.sqrt(-np.expm1(-2 * k * sr))
    start = s["h"] if one else s["h0"]
    keep = np.ones((B, L, 1)) if one or s["reset"] is None else 1.0 - s["reset"].double().cpu().numpy()[..., None]
    state = np.zeros((B, H)) if start is None else start.double().cpu().numpy()
    prev, y = np.empty_like(x), np.empty_like(x)
    for t in range(L):
        prev[:, t] = keep[:, t] * state
        state = a[:, t] * prev[:, t] + m[:, t] * si[:, t] * x[:, t]
        y[:, t] = state
    if one:
        return y[:, 0], state
    if s["op"] == "scan":
        return y, state
    dy = s["dy"].double().cpu().numpy()
    G = np.zeros((B, H)) if s["dh_last"] is None else s["dh_last"].double().cpu().numpy()
    dx, dr, di, dk = np.empty_like(x), np.empty_like(x), np.empty_like(x), np.zeros(H)
    for t in range(L - 1, -1, -1):
        G = G + dy[:, t]
        in_ = si[:, t] * x[:, t]
        da = G * (prev[:, t] - a[:, t] / m[:, t] * in_)
        dx[:, t] = G * m[:, t] * si[:, t]
        di[:, t] = G * m[:, t] * in_ * (1 - si[:, t])
        dlog = da * a[:, t]
        dr[:, t] = -dlog * k * sr[:, t] * (1 - sr[:, t])
        dk -= (dlog * sr[:, t]).sum(0)
        G = keep[:, t] * a[:, t] * G
    out = [y, state, dx, dr, di, dk * SCALE / (1 + np.exp(-f["p"]))]
    return out + [G] if s["h0"] is not None else out


def _exact_pack(t):
    z = t.double().cpu().numpy()
    out = np.zeros_like(z)
    for j in range(0, z.shape[1], GROUP):
        c = z[:, j:j + GROUP]
        top = np.abs(c).max(1, keepdims=True)
        with np.errstate(divide="ignore"):
            s = np.clip(np.where(top > 0, np.ceil(np.log2(top / 448.0)), -127), -127, 127)
        q = c / 2.0 ** s
        unit = 2.0 ** (np.maximum(np.frexp(q)[1] - 1, -6) - 3)  # the spacing of e4m3 at q
        out[:, j:j + GROUP] = np.rint(q / unit) * unit * 2.0 ** s
    return out


def _exact_join(s):
    names = ("x", "h", "g", "w", "alpha", "v")

    def forward(x, h, g, w, alpha, v):
        def norm(z):
            z = z - z.mean(1, keepdim=True) if s["norm"] == "layer" else z
            return z / ((z ** 2).mean(1, keepdim=True) + EPS) ** 0.5
        y = x + alpha * (norm(h * (g * torch.sigmoid(g) if s["act"] == "silu" else torch.sigmoid(g))) * w)
        return y, norm(y) * v

    t = {n: s[n].double().cpu() for n in names}
    y, n = forward(**t)
    if s["op"] == "join":
        return [y, n]
    if s["op"] == "ckpt_train":
        t["h"], t["g"] = torch.from_numpy(_exact_pack(s["h"])), torch.from_numpy(_exact_pack(s["g"]))
    for v in t.values():
        v.requires_grad_(True)
    y2, n2 = forward(**t)
    grads = torch.autograd.grad([y2, n2], list(t.values()), [s["dy"].double().cpu(), s["dn"].double().cpu()])
    return [y, n, *grads]


def exact(case, seed):
    size = case["H"] * (case["M"] if "M" in case else case["B"] * case.get("L", 1))
    if size > 17_000_000:
        return None
    s = prepare(case, seed)
    if case["op"] in ("step", "scan", "train"):
        return _exact_scan(s)
    return _exact_pack(s["t"]) if case["op"] == "ckpt_pack" else _exact_join(s)
