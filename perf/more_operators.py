"""A selective state space model's operators: what is timed, their plain forms, and their definitions in 64 bits.

Three operators that stand together in a language model of selective state space blocks:

* the short causal convolution before the scan (training step, and one token from the last inputs),
* the selective scan, N states to a channel (forward, training step, and one token from a carried state),
* the softmax cross entropy of a projection onto a vocabulary (loss, and loss with its gradients).

`run` computes a case in elementary torch operations in 32 bits, or, where `own` is true, by the framework's calls.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
SCAN_MOST = 4 * 4096 * 4096 * 16  # steps x channels x states of the largest training case
CONV_MOST = 4 * 16384 * 2048      # steps x channels of the largest convolution
HEAD_MOST = 8192 * 50257 * 2048   # rows x vocabulary x width of the largest loss


def listed():
    return [
        # one token of one stream: nothing but latency
        {"name": "step_one_stream", "op": "step", "B": 1, "H": 2048, "N": 16, "G": 1, "type": "bf16", "full": True},
        # one token of each sequence of a full serving batch
        {"name": "step_batch", "op": "step", "B": 256, "H": 4096, "N": 16, "G": 1, "type": "bf16", "full": True},
        # a short prompt of odd length that continues a carried state
        {"name": "scan_prompt", "op": "scan", "B": 1, "L": 333, "H": 1024, "N": 16, "G": 1, "type": "bf16", "full": True, "h0": True,
         "docs": 0, "fused": True},
        # one very long sequence over few channels with many states (the long bank's sizes), without gate and skip
        {"name": "scan_long", "op": "scan", "B": 1, "L": 65536, "H": 256, "N": 64, "G": 1, "type": "f32", "full": False, "h0": False,
         "docs": 0, "fused": False},
        # a training step of the bank's sizes, several documents packed into each row
        {"name": "train_packed", "op": "train", "B": 8, "L": 4096, "H": 256, "N": 16, "G": 1, "type": "bf16", "full": True, "h0": False,
         "docs": 5, "fused": True},
        # odd sizes in 32 bits, with a state carried in and its gradient
        {"name": "train_odd", "op": "train", "B": 3, "L": 1021, "H": 131, "N": 11, "G": 1, "type": "f32", "full": True, "h0": True,
         "docs": 3, "fused": False},
        # a training step at a language model's width: the largest scan
        {"name": "train_wide", "op": "train", "B": 4, "L": 4096, "H": 4096, "N": 16, "G": 1, "type": "bf16", "full": True, "h0": False,
         "docs": 0, "fused": True},
        # the convolution of a training step over long packed rows
        {"name": "conv_train", "op": "conv_train", "B": 4, "L": 16384, "H": 2048, "K": 4, "type": "bf16", "state": False, "docs": 17,
         "fused": True},
        # the convolution of one token of each sequence of a serving batch
        {"name": "conv_step", "op": "conv_step", "B": 256, "H": 4096, "K": 4, "type": "bf16"},
        # the log-likelihoods of a few tokens
        {"name": "head_score", "op": "head", "M": 16, "V": 50257, "D": 2048, "type": "bf16"},
        # a training step's loss with its gradients over a batch of tokens
        {"name": "head_train", "op": "head_train", "M": 8192, "V": 50257, "D": 2048, "type": "bf16"},
        # the same in 32 bits at odd sizes
        {"name": "head_train_odd", "op": "head_train", "M": 1021, "V": 4099, "D": 515, "type": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "scan", "scan", "train", "train", "train", "conv_step", "conv_train", "head", "head_train", "head_train"])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("head", "head_train"):
        D = _log(rng, 16, 4096)
        D = max(16, D // 16 * 16) if rng.random() < 0.7 else D
        V = _log(rng, 50, 131072)
        # a 32-bit product costs several of a 16-bit one
        most = HEAD_MOST // (8 if kind == "f32" else 1)
        M = _log(rng, 1, max(1, min(16384, most // (V * D), 2 ** 30 // V)))
        return {"op": op, "M": M, "V": V, "D": D, "type": kind}
    H = _log(rng, 16, 4096)
    H = max(16, H // 16 * 16) if rng.random() < 0.7 else H
    if op == "conv_step":
        return {"op": op, "B": _log(rng, 1, 512), "H": H, "K": rng.choice([2, 3, 4, 4]), "type": kind}
    if op == "conv_train":
        B = _log(rng, 1, 16)
        L = _log(rng, 1, max(1, min(65536, CONV_MOST // (B * H))))
        return {"op": op, "B": B, "L": L, "H": H, "K": rng.choice([2, 3, 4, 4]), "type": kind, "state": rng.random() < 0.5,
                "docs": rng.choice([0, 0, 3, 17]) if L > 64 else 0, "fused": rng.random() < 0.5}
    N = rng.choice([16, 16, 16, 8, 64, _log(rng, 1, 64)])
    G = rng.choice([1, 1, 1, 2, 4])
    H = -(-H // G) * G
    full = rng.random() < 0.75
    if op == "step":
        return {"op": op, "B": _log(rng, 1, 512), "H": H, "N": N, "G": G, "type": kind, "full": full}
    B = _log(rng, 1, 16)
    L = _log(rng, 1, max(1, min(65536, SCAN_MOST // (2 * B * H * N))))
    return {"op": op, "B": B, "L": L, "H": H, "N": N, "G": G, "type": kind, "full": full, "h0": rng.random() < 0.5,
            "docs": rng.choice([0, 0, 3, 17]) if L > 64 else 0, "fused": rng.random() < 0.5}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype, op = TYPES[case["type"]], case["op"]

    def normal(*shape, dtype=dtype, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    s = dict(case)
    if op in ("head", "head_train"):
        M, V, D = case["M"], case["V"], case["D"]
        s["W"] = normal(V, D, scale=1.0 / math.sqrt(D))
        s["target"] = uniform(M).mul(V).long().clamp(max=V - 1)
        # rows whose target a trained model finds, from hardly to almost surely
        sure = uniform(M, 1) * 16.0
        s["h"] = (normal(M, D, dtype=torch.float32) + sure * s["W"][s["target"]].float()).to(dtype)
        padded = uniform(M) < 0.05  # the ends of the batch's rows, which have no next token
        if M > 1:
            s["target"][padded] = -1
        if op == "head_train":
            # the mean over the rows that count, by a loss scale where the type's range is short
            count = (s["target"] >= 0).sum().clamp(min=1)
            s["dloss"] = torch.where(s["target"] >= 0, (4096.0 if case["type"] == "f16" else 1.0) / count, 0.0).float()
        return s
    B, L, H = case["B"], case.get("L", 1), case["H"]
    s["reset"] = None
    if case.get("docs"):  # where documents begin in the packed rows
        at = uniform(B, case["docs"]).mul(L).long()
        s["reset"] = torch.zeros(B, L, dtype=torch.bool, device="cuda")
        s["reset"].scatter_(1, at, True)
    if op in ("conv_step", "conv_train"):
        K = case["K"]
        s["w"] = normal(H, K, dtype=torch.float32, scale=1.0 / math.sqrt(K))
        s["bias"] = normal(H, dtype=torch.float32, scale=0.2)
        if op == "conv_step":
            s["x"], s["last"] = normal(B, H), normal(B, K - 1, H)
            s["last_out"] = torch.empty_like(s["last"])
            return s
        # the first half of a projection's columns, the gate behind it
        s["x"] = normal(B, L, 2 * H)[..., :H] if case["fused"] else normal(B, L, H)
        s["last"] = normal(B, K - 1, H) if case["state"] else None
        s["dy"] = normal(B, L, H)
        s["dlast"] = normal(B, K - 1, H) if case["state"] else None
        return s
    N, G = case["N"], case["G"]
    s["x"], s["dt"] = normal(B, L, H), normal(B, L, H, scale=0.5)
    if case.get("fused"):  # columns of one product: a low-rank step, then what the states take in and give out
        z = normal(B, L, 32 + 2 * G * N)
        s["Bm"], s["Cm"] = z[..., 32:32 + G * N].unflatten(-1, (G, N)), z[..., 32 + G * N:].unflatten(-1, (G, N))
        s["z"] = normal(B, L, 2 * H)[..., H:] if case["full"] else None
    else:
        s["Bm"], s["Cm"] = normal(B, L, G, N), normal(B, L, G, N)
        s["z"] = normal(B, L, H) if case["full"] else None
    # decay rates around 1 .. N, steps from 0.001 to 0.1
    s["A"] = -torch.exp(torch.log(torch.arange(1, N + 1, device="cuda").float()) + normal(H, N, dtype=torch.float32, scale=0.1))
    d = torch.exp(uniform(H) * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
    s["bias"] = torch.log(torch.expm1(d))
    s["D"] = 1.0 + normal(H, dtype=torch.float32, scale=0.1) if case["full"] else None
    if op == "step":
        for n in ("x", "dt", "z", "Bm", "Cm"):
            s[n] = s[n][:, 0] if s[n] is not None else None
        s["h"] = normal(B, H, N, dtype=torch.float32)
        s["h_out"] = torch.empty_like(s["h"])
        return s
    s["h0"] = normal(B, H, N, dtype=torch.float32) if case["h0"] else None
    if op == "train":
        s["dy"] = normal(B, L, H)
        s["dh_last"] = normal(B, H, N, dtype=torch.float32) if case["h0"] else None
    return s


# ---- the plain forms ---------------------------------------------------------------------------


def _sigmoid(t):
    return 1.0 / (1.0 + torch.exp(-t))


def _softplus(t):
    return t.clamp(min=0.0) + torch.log1p(torch.exp(-t.abs()))


def _documents(s, B, L):
    """The number of the document that each step belongs to."""
    if s["reset"] is None:
        return torch.zeros(B, L, dtype=torch.long, device="cuda")
    return s["reset"].long().cumsum(1)


def _plain_conv(s):
    x, w, t = s["x"], s["w"], s["x"].dtype
    B, L, H = x.shape
    K = w.shape[1]
    doc = torch.cat([torch.zeros(B, K - 1, dtype=torch.long, device="cuda"), _documents(s, B, L)], 1)
    before = torch.zeros(B, K - 1, H, device="cuda") if s["last"] is None else s["last"].float()
    xs = torch.cat([before, x.float()], 1)
    seen = [(doc[:, j:j + L] == doc[:, K - 1:])[..., None] for j in range(K)]
    pre = s["bias"].expand(B, L, H)
    for j in range(K):
        pre = pre + torch.where(seen[j], w[:, j] * xs[:, j:j + L], 0.0)
    sg = _sigmoid(pre)
    y = pre * sg
    last = torch.where((doc[:, L:] == doc[:, -1:])[..., None], xs[:, L:], 0.0).to(t)
    out = [y.to(t), last]
    g = s["dy"].float() * sg * (1.0 + pre * (1.0 - sg))
    dxs = torch.zeros_like(xs)
    if s["dlast"] is not None:
        dxs[:, L:] += torch.where((doc[:, L:] == doc[:, -1:])[..., None], s["dlast"].float(), 0.0)
    dw = []
    for j in range(K):
        gj = torch.where(seen[j], g, 0.0)
        dxs[:, j:j + L] += w[:, j] * gj
        dw.append((gj * xs[:, j:j + L]).sum((0, 1)))
    out += [dxs[:, K - 1:].to(t), torch.stack(dw, 1), g.sum((0, 1))]
    return out + [dxs[:, :K - 1].to(t)] if s["last"] is not None else out


def _plain_conv_step(s):
    xs = torch.cat([s["last"], s["x"][:, None]], 1)
    pre = s["bias"] + (xs.float() * s["w"].t()).sum(1)
    return (pre * _sigmoid(pre)).to(s["x"].dtype), xs[:, 1:].contiguous()


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 1, by doubling the span that each entry covers."""
    d, L = 1, a.shape[1]
    while d < L:
        b = torch.cat([b[:, :d], b[:, d:] + a[:, d:] * b[:, :-d]], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return b


def _wide(t, H):
    """What the groups share, for each channel: [..., G, N] -> [..., H, N] in 32 bits."""
    return t.float().repeat_interleave(H // t.shape[-2], -2)


def _plain_scan(s):
    x, H, t = s["x"].float(), s["H"], s["x"].dtype
    raw = s["dt"].float() + s["bias"]
    step = _softplus(raw)
    a = torch.exp(step[..., None] * s["A"])
    if s["reset"] is not None:
        a = torch.where(s["reset"][..., None, None], torch.zeros_like(a), a)
    Bm, Cm = _wide(s["Bm"], H), _wide(s["Cm"], H)
    b = (step * x)[..., None] * Bm
    if s["h0"] is not None:
        b[:, 0] += a[:, 0] * s["h0"]
    h = _scan(a, b)
    del b
    out = (h * Cm).sum(-1)
    if s["D"] is not None:
        out = out + s["D"] * x
    z = None if s["z"] is None else s["z"].float()
    sg = None if z is None else _sigmoid(z)
    got = [(out if z is None else out * z * sg).to(t), h[:, -1].clone()]
    if s["op"] == "scan":
        return got
    dy = s["dy"].float()
    g = dy if z is None else dy * z * sg
    grad = g[..., None] * Cm
    if s["dh_last"] is not None:
        grad[:, -1] += s["dh_last"]
    after = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    grad = _scan(after.flip(1), grad.flip(1)).flip(1)
    del after

    def shared(v):  # the sum over the channels of a group
        return v.unflatten(2, (s["G"], H // s["G"])).sum(3)

    dB, dC = shared(grad * (step * x)[..., None]), shared(g[..., None] * h)
    q = (grad * Bm).sum(-1)
    first = torch.zeros_like(h[:, :1]) if s["h0"] is None else s["h0"][:, None]
    grad *= a
    dh0 = grad[:, 0].clone()
    grad *= torch.cat([first, h[:, :-1]], 1)
    del h, a
    dstep = x * q + (grad * s["A"]).sum(-1)
    dA = (grad * step[..., None]).sum((0, 1))
    ddt = dstep * _sigmoid(raw)
    dx = step * q if s["D"] is None else step * q + s["D"] * g
    got += [dx.to(t), ddt.to(t), dA, dB.to(t), dC.to(t), ddt.sum((0, 1))]
    if z is not None:
        got += [(g * x).sum((0, 1)), (dy * out * sg * (1.0 + z * (1.0 - sg))).to(t)]
    return got + [dh0] if s["h0"] is not None else got


def _plain_step(s):
    x, H = s["x"].float(), s["H"]
    step = _softplus(s["dt"].float() + s["bias"])
    h = torch.exp(step[..., None] * s["A"]) * s["h"] + (step * x)[..., None] * _wide(s["Bm"], H)
    out = (h * _wide(s["Cm"], H)).sum(-1)
    if s["z"] is not None:
        z = s["z"].float()
        out = (out + s["D"] * x) * z * _sigmoid(z)
    return out.to(s["x"].dtype), h


def _plain_head(s):
    h, W, target = s["h"].float(), s["W"].float(), s["target"]
    valid = target >= 0
    at = target.clamp(min=0)[:, None]
    z = h @ W.t()
    top = z.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(z - top).sum(1, keepdim=True))
    loss = torch.where(valid, (lse - z.gather(1, at))[:, 0], 0.0)
    if s["op"] == "head":
        return loss, lse[:, 0]
    d = torch.exp(z - lse)
    d.scatter_add_(1, at, torch.full_like(lse, -1.0))
    d *= torch.where(valid, s["dloss"], 0.0)[:, None]
    return loss, lse[:, 0], (d @ W).to(s["h"].dtype), (d.t() @ h).to(s["W"].dtype)


def _plain(s):
    return {"step": _plain_step, "scan": _plain_scan, "train": _plain_scan, "conv_step": _plain_conv_step, "conv_train": _plain_conv,
            "head": _plain_head, "head_train": _plain_head}[s["op"]](s)


# ---- the framework's calls ---------------------------------------------------------------------


def _own(s):
    from state_space_sequence_gb300 import ssm, xent
    op = s["op"]
    if op == "conv_step":
        y = ssm.ssm_conv_step(s["x"], s["w"], s["last"], bias=s["bias"], state_out=s["last_out"])
        return y, s["last_out"]
    if op == "conv_train":
        y, last = ssm.ssm_conv(s["x"], s["w"], bias=s["bias"], state=s["last"], reset=s["reset"])
        dx, dw, dbias, dstate = ssm.ssm_conv_backward(s["x"], s["w"], s["dy"], bias=s["bias"], state=s["last"], reset=s["reset"],
                                                      dlast=s["dlast"])
        return [y, last, dx, dw, dbias] + ([dstate] if dstate is not None else [])
    if op == "head":
        return xent.xent_loss(s["h"], s["W"], s["target"])
    if op == "head_train":
        loss, lse = xent.xent_loss(s["h"], s["W"], s["target"])
        return loss, lse, *xent.xent_loss_backward(s["h"], s["W"], s["target"], lse, s["dloss"])
    args = (s["x"], s["dt"], s["A"], s["Bm"], s["Cm"])
    how = {"D": s["D"], "z": s["z"], "dt_bias": s["bias"]}
    if op == "step":
        y = ssm.ssm_step(*args, s["h"], h_out=s["h_out"], **how)
        return y, s["h_out"]
    how.update(h0=s["h0"], reset=s["reset"])
    if op == "scan":
        return list(ssm.ssm_scan(*args, **how))
    y, h_last, states = ssm.ssm_scan(*args, save_states=True, **how)
    g = ssm.ssm_scan_backward(*args, s["dy"], states, dh_last=s["dh_last"], **how)
    got = [y, h_last, g.dx, g.ddt, g.dA, g.dB, g.dC, g.ddt_bias]
    if s["z"] is not None:
        got += [g.dD, g.dz]
    return got + [g.dh0] if s["h0"] is not None else got


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    e, op = BYTES[case["type"]], case["op"]
    if op in ("head", "head_train"):
        M, V, D = case["M"], case["V"], case["D"]
        if op == "head":
            return {"bytes": e * (M + V) * D + 16 * M, "flops": 2 * M * V * D + 4 * M * V}
        return {"bytes": 2 * e * (M + V) * D + 20 * M, "flops": 6 * M * V * D + 8 * M * V}
    B, L, H = case["B"], case.get("L", 1), case["H"]
    n = B * L * H
    mask = B * L if case.get("docs") else 0
    if op in ("conv_step", "conv_train"):
        K = case["K"]
        rows, par = e * B * (K - 1) * H, 4 * H * (K + 1)
        if op == "conv_step":
            return {"bytes": 2 * e * n + 2 * rows + par, "flops": (2 * K + 5) * n}
        return {"bytes": 5 * e * n + (4 if case["state"] else 1) * rows + 2 * par + mask, "flops": (6 * K + 20) * n}
    N, G = case["N"], case["G"]
    full, shared, state, par = case["full"], e * B * L * G * N, 4 * B * H * N, 4 * H * (N + 2)
    if op == "step":
        return {"bytes": (4 if full else 3) * e * n + 2 * shared + 2 * state + par, "flops": (7 * N + 20) * n}
    got = {"bytes": (4 if full else 3) * e * n + 2 * shared + (2 if case["h0"] else 1) * state + par + mask, "flops": (7 * N + 20) * n}
    if op == "train":  # dy read, three or two gradients of activations and two of what the groups share written
        got["bytes"] += (4 if full else 3) * e * n + 2 * shared + par + (2 * state if case["h0"] else 0)
        got["flops"] += (16 * N + 40) * n
    return got


# ---- the definitions in 64 bits ------------------------------------------------------------------


def _exact_conv(s):
    f = {n: (None if s[n] is None else s[n].double()) for n in ("x", "w", "bias", "last")}
    one = s["op"] == "conv_step"
    leaves = {n: v.clone().requires_grad_(not one) for n, v in f.items() if v is not None}
    x = leaves["x"][:, None] if one else leaves["x"]
    w = leaves["w"]
    B, L, H = x.shape
    K = w.shape[1]
    seen = torch.zeros(B, L + K - 1, dtype=torch.long, device="cuda")  # how many documents have begun
    if s["reset"] is not None:
        seen[:, K - 1:] = torch.cumsum(s["reset"].long(), 1)
    first = leaves["last"] if "last" in leaves else torch.zeros(B, K - 1, H, dtype=torch.float64, device="cuda")
    line = torch.cat([first, x], 1)
    windows = line.unfold(1, K, 1)  # [B, L, H, K]
    same = (seen.unfold(1, K, 1) == seen[:, K - 1:, None])[:, :, None]
    pre = (torch.where(same, windows, torch.zeros((), dtype=torch.float64, device="cuda")) * w).sum(-1) + leaves["bias"]
    y = pre * torch.sigmoid(pre)
    last = line[:, L:] * (seen[:, L:] == seen[:, -1:])[..., None]
    if one:
        return y[:, 0], last
    loss = (y * s["dy"].double()).sum()
    if s["dlast"] is not None:
        loss = loss + (last * s["dlast"].double()).sum()
    order = ["x", "w", "bias"] + (["last"] if "last" in leaves else [])
    return [y.detach(), last.detach(), *torch.autograd.grad(loss, [leaves[n] for n in order])]


def _exact_scan(s):
    f = {n: (None if s[n] is None else s[n].double()) for n in ("x", "dt", "A", "Bm", "Cm", "D", "z", "bias")}
    one = s["op"] == "step"
    if one:
        for n in ("x", "dt", "Bm", "Cm", "z"):
            f[n] = None if f[n] is None else f[n][:, None]
    x, A, H, G = f["x"], f["A"], s["H"], s["G"]
    B, L, _ = x.shape
    raw = f["dt"] + f["bias"]
    step = torch.logaddexp(raw, torch.zeros_like(raw))
    group = torch.arange(H, device="cuda") // (H // G)
    start = s["h"] if one else s["h0"]
    h = torch.zeros(B, H, A.shape[1], dtype=torch.float64, device="cuda") if start is None else start.double()
    train = s["op"] == "train"
    prev, rates, out = [], [], torch.empty_like(x)
    for t in range(L):
        if s["reset"] is not None:
            h = torch.where(s["reset"][:, t, None, None], torch.zeros_like(h), h)
        a = torch.exp(step[:, t, :, None] * A)
        if train:
            prev.append(h)
            rates.append(a)
        h = a * h + (step[:, t] * x[:, t])[..., None] * f["Bm"][:, t, group]
        out[:, t] = torch.einsum("bhn,bhn->bh", h, f["Cm"][:, t, group])
    if f["D"] is not None:
        out = out + f["D"] * x
    y = out if f["z"] is None else out * (f["z"] * torch.sigmoid(f["z"]))
    if one:
        return y[:, 0], h
    if not train:
        return [y, h]
    dy = s["dy"].double()
    g = dy if f["z"] is None else dy * (f["z"] * torch.sigmoid(f["z"]))
    carry = torch.zeros_like(h) if s["dh_last"] is None else s["dh_last"].double()
    q, slope, dA = torch.empty_like(x), torch.empty_like(x), torch.zeros_like(A)
    dB, dC = torch.empty_like(f["Bm"]), torch.empty_like(f["Cm"])
    for t in range(L - 1, -1, -1):
        now = rates[t] * prev[t] + (step[:, t] * x[:, t])[..., None] * f["Bm"][:, t, group]
        dC[:, t] = (g[:, t, :, None] * now).unflatten(1, (G, H // G)).sum(2)
        carry = carry + g[:, t, :, None] * f["Cm"][:, t, group]
        dB[:, t] = (carry * (step[:, t] * x[:, t])[..., None]).unflatten(1, (G, H // G)).sum(2)
        q[:, t] = (carry * f["Bm"][:, t, group]).sum(-1)
        carry = carry * rates[t]
        through = carry * prev[t]
        slope[:, t] = (through * A).sum(-1)
        dA += (through * step[:, t, :, None]).sum(0)
        if s["reset"] is not None:
            carry = torch.where(s["reset"][:, t, None, None], torch.zeros_like(carry), carry)
    ddt = (x * q + slope) * torch.sigmoid(raw)
    dx = step * q + (0 if f["D"] is None else f["D"] * g)
    got = [y, h, dx, ddt, dA, dB, dC, ddt.sum((0, 1))]
    if f["z"] is not None:
        sg = torch.sigmoid(f["z"])
        got += [(g * x).sum((0, 1)), dy * out * (sg + f["z"] * sg * (1 - sg))]
    return got + [carry] if s["h0"] is not None else got


def _exact_head(s):
    h, W = s["h"].double(), s["W"].double()
    z = h @ W.t()
    lse = torch.logsumexp(z, 1)
    rows = torch.nonzero(s["target"] >= 0)[:, 0]
    loss = torch.zeros_like(lse)
    loss[rows] = lse[rows] - z[rows, s["target"][rows]]
    if s["op"] == "head":
        return loss, lse
    p = torch.exp(z.sub_(lse[:, None]))
    p[rows, s["target"][rows]] -= 1.0
    weight = torch.zeros_like(lse)
    weight[rows] = s["dloss"][rows].double()
    p *= weight[:, None]
    return loss, lse, p @ W, p.t() @ h


def exact(case, seed):
    op, L = case["op"], case.get("L", 1)
    if op in ("scan", "step", "train"):
        size = case["B"] * L * case["H"] * case["N"]
        # each step of a long row is some twenty launches
        if size > 2 ** 30 or (op == "train" and L > 20000):
            return None
    s = prepare(case, seed)
    if op in ("conv_step", "conv_train"):
        return _exact_conv(s)
    return _exact_head(s) if op.startswith("head") else _exact_scan(s)
