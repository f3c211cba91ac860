"""A small gated recurrent block from the operators of :mod:`glr`, as a program would use them.

A stack keeps two arrays between blocks: the residual stream ``y`` and its norm ``n``. A block is

    x, r, i, g = n Wx, n Wr, n Wi, n Wg      one product for x, r, i, whose columns the scan reads
    h = gated linear recurrence of (x, r, i)                                       glr_scan
    y, n = join of (y, h, g)                 gate, norm, scale, add, next norm     glr_join

``forward`` keeps what ``backward`` needs: the scan's inputs and kept states, and h and g as 8-bit
checkpoints or as they are. ``step`` takes one token through the block from a carried state.

    python -m state_space_sequence_gb300.gated_block

trains a stack of two such blocks for a few steps to repeat the last marked token of its sequence,
several documents to a row, and then decodes token by token from the states of a prompt.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import glr


class Params(NamedTuple):
    """Of one block of width H. The products' weights are of the activations' type, the others
    float32."""
    Wxri: torch.Tensor    # [H, 3H]
    Wg: torch.Tensor      # [H, H]
    p: torch.Tensor       # [H] decay parameters
    w: torch.Tensor       # [H] the inner norm's weights
    alpha: torch.Tensor   # [1] residual scale
    v: torch.Tensor       # [H] the next norm's weights


def make_params(H: int, dtype=torch.bfloat16, device="cuda", seed: int = 0) -> Params:
    gen = torch.Generator().manual_seed(seed)
    a0 = torch.rand(H, generator=gen) * 0.099 + 0.9
    return Params((torch.randn(H, 3 * H, generator=gen) / H ** 0.5).to(dtype).to(device),
                  (torch.randn(H, H, generator=gen) / H ** 0.5).to(dtype).to(device),
                  torch.log(torch.expm1(-torch.log(a0))).to(device),
                  torch.ones(H, device=device), torch.full((1,), 0.5, device=device),
                  torch.ones(H, device=device))


class Saved(NamedTuple):
    y: torch.Tensor
    n: torch.Tensor
    xri: torch.Tensor
    states: torch.Tensor
    h: Optional[torch.Tensor]
    g: Optional[torch.Tensor]
    kept: Optional[tuple]
    reset: Optional[torch.Tensor]


def _rows(t):
    return t.reshape(-1, t.shape[-1])


def _columns(xri, H):
    return xri[..., :H], xri[..., H:2 * H], xri[..., 2 * H:]


def forward(par: Params, y, n, h0=None, reset=None, ckpt: bool = True):
    """y, n [B, L, H] -> (y, n, h_last [B, H], saved)."""
    H = y.shape[-1]
    xri, g = n @ par.Wxri, _rows(n @ par.Wg)
    h, h_last, states = glr.glr_scan(*_columns(xri, H), par.p, h0=h0, reset=reset,
                                     save_states=True)
    out = glr.glr_join(_rows(y), _rows(h), g, par.w, par.alpha, par.v, ckpt=ckpt)
    saved = Saved(y, n, xri, states, None if ckpt else h, None if ckpt else g,
                  out[2] if ckpt else None, reset)
    return out[0].view_as(y), out[1].view_as(y), h_last, saved


def backward(par: Params, saved: Saved, dy, dn, h0=None):
    """Gradients (dy, dn, Params of gradients) with respect to the block's inputs and parameters
    for those of its outputs."""
    H = dy.shape[-1]
    h, g = (None, None) if saved.kept is not None else (_rows(saved.h), saved.g)
    d, dh, dg, dw, dalpha, dv = glr.glr_join_backward(_rows(dy), _rows(dn), _rows(saved.y), h, g,
                                                      par.w, par.alpha, par.v, ckpt=saved.kept)
    dxri = torch.empty_like(saved.xri)
    _, _, _, dp, _ = glr.glr_scan_backward(*_columns(saved.xri, H), par.p, dh.view_as(dy),
                                           saved.states, h0=h0, reset=saved.reset,
                                           out=_columns(dxri, H))
    n = _rows(saved.n)
    grads = Params(n.t() @ _rows(dxri), n.t() @ dg, dp, dw, dalpha, dv)
    return d.view_as(dy), (_rows(dxri) @ par.Wxri.t() + dg @ par.Wg.t()).view_as(dy), grads


def step(par: Params, y, n, h, reset=None):
    """One token: y, n [B, H] and the state h [B, H] (float32, becomes the next) -> (y, n)."""
    o = glr.glr_step(*_columns(n @ par.Wxri, y.shape[-1]), par.p, h, reset=reset)
    return glr.glr_join(y, o, n @ par.Wg, par.w, par.alpha, par.v)


def main() -> None:
    torch.manual_seed(0)
    B, L, H, V, lr = 16, 192, 128, 32, 3e-3
    dtype = torch.bfloat16
    blocks = [make_params(H, dtype, seed=k) for k in range(2)]
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
        tok = torch.randint(2, V, (B, L), device="cuda")
        mark = torch.rand(B, L, device="cuda") < 0.1  # the next token is to be remembered
        tok[mark] = 1
        reset = torch.zeros(B, L, dtype=torch.bool, device="cuda")
        reset[:, [0, 80, 131]] = True
        tok[reset] = 1
        want = torch.zeros_like(tok)
        keep = torch.zeros(B, dtype=torch.long, device="cuda")
        for t in range(L):
            if t:
                keep = torch.where(tok[:, t - 1] == 1, tok[:, t], keep)
            keep = torch.where(reset[:, t], torch.zeros_like(keep), keep)
            want[:, t] = keep
        return tok, reset, want

    def run(tok, reset, ckpt=True):
        y = embed[tok].to(dtype)
        n = glr.glr_join(_rows(y), None, None, None, None, first)[1].view_as(y)
        saved = []
        for b in blocks:
            y, n, _, s = forward(b, y, n, reset=reset, ckpt=ckpt)
            saved.append(s)
        return n, saved

    for k in range(241):
        tok, reset, want = batch()
        n, saved = run(tok, reset)
        logits = n.float() @ embed.t()
        prob = torch.softmax(logits, -1)
        count = B * L
        loss = -torch.log(prob.gather(-1, want[..., None]) + 1e-9).mean()
        if k % 60 == 0:
            print(f"step {k:3d}  loss {loss.item():.4f}")
        d = prob
        d.scatter_add_(-1, want[..., None], torch.full_like(d[..., :1], -1.0))
        d = d / count
        de = _rows(d).t() @ _rows(n).float()
        dn, dy = (d @ embed).to(dtype), torch.zeros_like(n)
        for j in (1, 0):
            dy, dn, grads = backward(blocks[j], saved[j], dy, dn)
            adam(k, weights[j], moments[j], grads)
            blocks[j] = Params(*(w.to(t.dtype) for w, t in zip(weights[j], blocks[j])))
        adam(k, weights[2], moments[2], [de])

    # the same rows token by token: a state a block, reset where a document begins
    tok, reset, _ = batch()
    n, _ = run(tok, reset)
    h = [torch.zeros(B, H, device="cuda") for _ in blocks]
    worst = 0.0
    for t in range(L):
        yt = embed[tok[:, t]].to(dtype)
        nt = glr.glr_join(yt, None, None, None, None, first)[1]
        for b, s in zip(blocks, h):
            yt, nt = step(b, yt, nt, s, reset=reset[:, t].contiguous())
        worst = max(worst, (nt.float() - n[:, t].float()).abs().max().item())
    print(f"decoded {L} tokens of {B} rows; largest difference from the scan {worst:.4f}")


if __name__ == "__main__":
    main()
