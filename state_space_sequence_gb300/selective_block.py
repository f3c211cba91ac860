"""A small selective state space block from the operators of :mod:`ssm`, as a program would use them,
trained with the loss of :mod:`xent`.

A stack keeps two arrays between blocks: the residual stream ``y`` and its norm ``n``. A block is

    x, z = n Wx, n Wz                        one product, of whose columns each is read as it lies
    u = causal convolution of x                                                     ssm_conv
    d, B, C = u Wp                           a low-rank step, and what the states take in and give out
    o = selective scan of (u, d Wdt, B, C), gated by z                              ssm_scan
    y, n = join of (y, o Wo)                 norm, scale, add, next norm             glr_join

``forward`` keeps what ``backward`` needs; ``step`` takes one token through the block from the last
inputs of its convolution and the state of its scan.

    python -m state_space_sequence_gb300.selective_block

trains a stack of two such blocks for some steps to repeat the last marked token of its sequence,
several documents to a row, and then decodes token by token from the states of a prompt.
"""
from __future__ import annotations

import math
from typing import NamedTuple, Optional

import torch

from . import glr, ssm, xent


class Params(NamedTuple):
    """Of one block of width H with E inner channels, N states, a step of rank R and K taps. The
    products' weights are of the activations' type, the others float32."""
    Wxz: torch.Tensor      # [H, 2E]
    taps: torch.Tensor     # [E, K]
    tap_bias: torch.Tensor  # [E]
    Wp: torch.Tensor       # [E, R + 2N]
    Wdt: torch.Tensor      # [R, E]
    dt_bias: torch.Tensor  # [E]
    A: torch.Tensor        # [E, N] the logarithms of the decay rates
    D: torch.Tensor        # [E]
    Wo: torch.Tensor       # [E, H]
    w: torch.Tensor        # [H] the inner norm's weights
    alpha: torch.Tensor    # [1] residual scale
    v: torch.Tensor        # [H] the next norm's weights


def make_params(H: int, E: Optional[int] = None, N: int = 16, R: int = 8, K: int = 4,
                dtype=torch.bfloat16, device="cuda", seed: int = 0) -> Params:
    gen = torch.Generator().manual_seed(seed)
    E = 2 * H if E is None else E
    mat = lambda a, b: (torch.randn(a, b, generator=gen) / a ** 0.5).to(dtype).to(device)
    step = torch.exp(torch.rand(E, generator=gen) * math.log(100.0) + math.log(0.001))
    return Params(mat(H, 2 * E), (torch.randn(E, K, generator=gen) / K ** 0.5).to(device),
                  torch.zeros(E, device=device), mat(E, R + 2 * N), mat(R, E),
                  torch.log(torch.expm1(step)).to(device),
                  torch.log(torch.arange(1, N + 1).float()).repeat(E, 1).to(device),
                  torch.ones(E, device=device), mat(E, H), torch.ones(H, device=device),
                  torch.full((1,), 0.5, device=device), torch.ones(H, device=device))


class State(NamedTuple):
    """What a sequence carries through a block: the convolution's last inputs [B, K-1, E] and the
    scan's states [B, E, N]."""
    inputs: torch.Tensor
    h: torch.Tensor


def start(par: Params, B: int) -> State:
    E, K = par.taps.shape
    return State(torch.zeros(B, K - 1, E, dtype=par.Wxz.dtype, device=par.Wxz.device),
                 torch.zeros(B, *par.A.shape, device=par.A.device))


class Saved(NamedTuple):
    y: torch.Tensor
    n: torch.Tensor
    xz: torch.Tensor
    u: torch.Tensor
    p: torch.Tensor
    dt: torch.Tensor
    states: torch.Tensor
    o: torch.Tensor
    out: torch.Tensor
    first: Optional[State]
    reset: Optional[torch.Tensor]


def _rows(t):
    return t.reshape(-1, t.shape[-1])


def _split(par: Params, p):
    """d, B and C among the columns of u Wp."""
    R, N = par.Wdt.shape[0], par.A.shape[1]
    return p[..., :R], p[..., R:R + N], p[..., R + N:]


def forward(par: Params, y, n, first: Optional[State] = None, reset=None):
    """y, n [B, L, H] -> (y, n, State, saved)."""
    E = par.taps.shape[0]
    xz = n @ par.Wxz
    x, z = xz[..., :E], xz[..., E:]
    before, h0 = (None, None) if first is None else first
    u, inputs = ssm.ssm_conv(x, par.taps, par.tap_bias, state=before, reset=reset)
    p = u @ par.Wp
    d, Bm, Cm = _split(par, p)
    dt = d @ par.Wdt
    o, h, states = ssm.ssm_scan(u, dt, -par.A.exp(), Bm, Cm, D=par.D, z=z, dt_bias=par.dt_bias, h0=h0,
                                reset=reset, save_states=True)
    out = o @ par.Wo
    y2, n2 = glr.glr_join(_rows(y), _rows(out), None, par.w, par.alpha, par.v, act="none")
    return (y2.view_as(y), n2.view_as(y), State(inputs, h),
            Saved(y, n, xz, u, p, dt, states, o, out, first, reset))


def backward(par: Params, s: Saved, dy, dn):
    """Gradients (dy, dn, Params of gradients) with respect to the block's inputs and parameters for
    those of its outputs."""
    E = par.taps.shape[0]
    x, z = s.xz[..., :E], s.xz[..., E:]
    before, h0 = (None, None) if s.first is None else s.first
    d, dout, _, dw, dalpha, dv = glr.glr_join_backward(
        _rows(dy), _rows(dn), _rows(s.y), _rows(s.out), None, par.w, par.alpha, par.v, act="none")
    do = (dout @ par.Wo.t()).view_as(s.o)
    # the gradients of the products' outputs, in their own layouts
    dxz, dp = torch.empty_like(s.xz), torch.empty_like(s.p)
    low, Bm, Cm = _split(par, s.p)
    dlow, dB, dC = _split(par, dp)
    du, ddt = torch.empty_like(s.u), torch.empty_like(s.dt)
    rate = -par.A.exp()
    g = ssm.ssm_scan_backward(s.u, s.dt, rate, Bm, Cm, do, s.states, D=par.D, z=z,
                              dt_bias=par.dt_bias, h0=h0, reset=s.reset,
                              out=(du, ddt, dB, dC, dxz[..., E:]))
    dlow.copy_((_rows(ddt) @ par.Wdt.t()).view_as(dlow))
    du += (_rows(dp) @ par.Wp.t()).view_as(du)
    _, dtaps, dtap_bias, _ = ssm.ssm_conv_backward(x, par.taps, du, par.tap_bias, state=before,
                                                   reset=s.reset, out=dxz[..., :E])
    t = lambda a, b: _rows(a).t() @ _rows(b)
    grads = Params(t(s.n, dxz), dtaps, dtap_bias, t(s.u, dp), t(low, ddt), g.ddt_bias, g.dA * rate,
                   g.dD, t(s.o, dout), dw, dalpha, dv)
    return d.view_as(dy), (_rows(dxz) @ par.Wxz.t()).view_as(dy), grads


def step(par: Params, y, n, state: State, reset=None):
    """One token: y, n [B, H] and the state, which becomes the next in place -> (y, n)."""
    E = par.taps.shape[0]
    xz = n @ par.Wxz
    u = ssm.ssm_conv_step(xz[:, :E], par.taps, state.inputs, par.tap_bias, reset=reset)
    d, Bm, Cm = _split(par, u @ par.Wp)
    o = ssm.ssm_step(u, d @ par.Wdt, -par.A.exp(), Bm, Cm, state.h, D=par.D, z=xz[:, E:],
                     dt_bias=par.dt_bias, reset=reset)
    return glr.glr_join(y, o @ par.Wo, None, par.w, par.alpha, par.v, act="none")


def stack(blocks, embed, first, tok, reset=None):
    """Tokens [B, L] looked up in embed [V, H] and normed (weights first [H]), then through the blocks:
    (n, each block's Saved)."""
    y = embed[tok].to(blocks[0].Wxz.dtype)
    n = glr.glr_join(_rows(y), None, None, None, None, first)[1].view_as(y)
    saved = []
    for b in blocks:
        y, n, _, s = forward(b, y, n, reset=reset)
        saved.append(s)
    return n, saved


def gradients(blocks, embed, first, tok, target, reset=None):
    """(losses [B L], each block's Params of gradients, embed's) of the mean loss over the tokens that have a
    target. The rows of embed [V, H] (float32) are looked up and are the vocabulary's: both count."""
    n, saved = stack(blocks, embed, first, tok, reset)
    rows, table = _rows(n), embed.to(n.dtype)
    losses, lse = xent.xent_loss(rows, table, target)
    weight = (1.0 / (target >= 0).sum()).expand(losses.shape).contiguous()
    dn, dtable = xent.xent_loss_backward(rows, table, target, lse, weight)
    dn, dy, grads = dn.view_as(n), torch.zeros_like(n), []
    for b, s in zip(blocks[::-1], saved[::-1]):
        dy, dn, g = backward(b, s, dy, dn)
        grads.insert(0, g)
    dx = glr.glr_join_backward(None, _rows(dn), _rows(saved[0].y), None, None, None, None, first)[0]
    dx = dx.float() + _rows(dy)  # the stack's first y is read by the norm and by the first block
    # a token's rows are added up in a fixed order
    return losses, grads, dtable.float().index_put_((tok.reshape(-1),), dx, accumulate=True)


def main(steps: int = 241) -> None:
    torch.manual_seed(0)
    B, L, H, V, lr = 16, 192, 128, 32, 3e-3
    dtype = torch.bfloat16
    blocks = [make_params(H, dtype=dtype, seed=k) for k in range(2)]
    embed = torch.randn(V, H, device="cuda")
    first = torch.ones(H, device="cuda")
    weights = [[t.float() for t in b] for b in blocks] + [[embed]]  # the masters, in float32
    moments = [[(torch.zeros_like(t), torch.zeros_like(t)) for t in b] for b in weights]

    def adam(k, ws, ms, grads):
        for t, (m, v), g in zip(ws, ms, grads):
            g = g.float()
            m.lerp_(g, 0.1)
            v.lerp_(g * g, 0.02)
            t.sub_(lr * (m / (1 - 0.9 ** (k + 1))) / ((v / (1 - 0.98 ** (k + 1))).sqrt() + 1e-8))

    def batch():
        """Tokens of which 1 marks the next one; at each step the last marked one is wanted, and
        nothing before the first."""
        tok = torch.randint(2, V, (B, L), device="cuda")
        tok[torch.rand(B, L, device="cuda") < 0.1] = 1
        reset = torch.zeros(B, L, dtype=torch.bool, device="cuda")
        reset[:, [0, 80, 131]] = True
        tok[reset] = 1
        want = torch.empty_like(tok)
        keep = torch.full((B,), -1, dtype=torch.long, device="cuda")
        for t in range(L):
            if t:
                keep = torch.where(tok[:, t - 1] == 1, tok[:, t], keep)
            keep = torch.where(reset[:, t], torch.full_like(keep, -1), keep)
            want[:, t] = keep
        return tok, reset, want.reshape(-1)

    for k in range(steps):
        tok, reset, want = batch()
        losses, grads, de = gradients(blocks, embed, first, tok, want, reset)
        if k % 60 == 0:
            print(f"step {k:3d}  loss {(losses.sum() / (want >= 0).sum()).item():.4f}")
        for j in (1, 0):
            adam(k, weights[j], moments[j], grads[j])
            blocks[j] = Params(*(w.to(t.dtype) for w, t in zip(weights[j], blocks[j])))
        adam(k, weights[2], moments[2], [de])

    # the same rows token by token: a state a block, begun anew where a document begins
    tok, reset, _ = batch()
    n = stack(blocks, embed, first, tok, reset)[0]
    states = [start(b, B) for b in blocks]
    worst = 0.0
    for t in range(L):
        yt = embed[tok[:, t]].to(dtype)
        nt = glr.glr_join(yt, None, None, None, None, first)[1]
        for b, s in zip(blocks, states):
            yt, nt = step(b, yt, nt, s, reset=reset[:, t].contiguous())
        worst = max(worst, (nt.float() - n[:, t].float()).abs().max().item())
    print(f"decoded {L} tokens of {B} rows; largest difference from the scan {worst:.4f}")


if __name__ == "__main__":
    main()
