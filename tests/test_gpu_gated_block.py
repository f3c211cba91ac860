"""The example block of the gated recurrence (gated_block.py): its operators run together, against
torch's autograd in float64 on the same values, and token by token against the whole sequence."""
import pytest
import torch

from state_space_sequence_gb300 import dlr, gated_block

pytestmark = pytest.mark.gpu


def plain(par, y, n, reset):
    """The block from its formulas, step by step, for autograd."""
    H = y.shape[-1]
    x, r, i = (n @ par[0]).split(H, -1)
    g = n @ par[1]
    z = -8.0 * torch.nn.functional.softplus(par[2]) * torch.sigmoid(r)
    a, b = z.exp(), torch.sqrt(-torch.expm1(2 * z)) * torch.sigmoid(i) * x
    s, hs = torch.zeros_like(y[:, 0]), []
    for t in range(y.shape[1]):
        s = a[:, t] * torch.where(reset[:, t, None], torch.zeros_like(s), s) + b[:, t]
        hs.append(s)
    u = torch.stack(hs, 1) * g * torch.sigmoid(g)
    norm = lambda z: z / torch.sqrt((z * z).mean(-1, keepdim=True) + 1e-6)
    y = y + par[4] * par[3] * norm(u)
    return y, par[5] * norm(y)


def test_block_gradients_in_float32():
    """Every product and operator in float32: within 2e-5 of each gradient's norm (1e-5 an operator,
    and the library's products in full float32)."""
    torch.backends.cuda.matmul.allow_tf32 = False
    B, L, H = 2, 70, 48
    gen = torch.Generator().manual_seed(3)
    y, n, dy, dn = (torch.randn(B, L, H, generator=gen).cuda() for _ in range(4))
    reset = torch.zeros(B, L, dtype=torch.bool, device="cuda")
    reset[0, 20] = reset[1, 64] = True
    par = gated_block.make_params(H, torch.float32, seed=5)
    y1, n1, _, saved = gated_block.forward(par, y, n, reset=reset, ckpt=False)
    got_y, got_n, grads = gated_block.backward(par, saved, dy, dn)
    args = [t.double().requires_grad_(True) for t in (*par, y, n)]
    ry, rn = plain(args[:6], args[6], args[7], reset)
    ref = torch.autograd.grad([ry, rn], args, [dy.double(), dn.double()])
    for a, q in zip((y1, n1, *grads, got_y, got_n), (ry, rn, *ref)):
        assert (a.double() - q).norm() <= 2e-5 * q.norm()
    assert dlr.device_status() == 0


def test_checkpoints_change_the_gradients_by_their_rounding():
    """e4m3 keeps 3 mantissa bits: values move by at most 2^-4 of themselves (but for those far
    below their group's largest), the gradients by a few percent of their norm, and what the
    forward pass returns not at all."""
    B, L, H = 2, 128, 64
    gen = torch.Generator().manual_seed(4)
    y, n, dy, dn = (torch.randn(B, L, H, generator=gen).to(torch.bfloat16).cuda() for _ in range(4))
    par = gated_block.make_params(H, seed=6)
    a = gated_block.forward(par, y, n, ckpt=False)
    b = gated_block.forward(par, y, n, ckpt=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for p, q in zip(gated_block.backward(par, a[3], dy, dn)[:2],
                    gated_block.backward(par, b[3], dy, dn)[:2]):
        far = (p.double() - q.double()).norm() / p.double().norm()
        assert 0 < far <= 2.0 ** -4


def test_steps_are_the_block():
    B, L, H = 3, 40, 64
    gen = torch.Generator().manual_seed(5)
    y, n = (torch.randn(B, L, H, generator=gen).cuda() for _ in range(2))
    par = gated_block.make_params(H, torch.float32, seed=7)
    torch.backends.cuda.matmul.allow_tf32 = False
    y1, n1, last, _ = gated_block.forward(par, y, n)
    h = torch.zeros(B, H, device="cuda")
    for t in range(L):
        yt, nt = gated_block.step(par, y[:, t], n[:, t], h)
        assert (nt.double() - n1[:, t].double()).norm() <= 2e-5 * n1[:, t].double().norm()
        assert (yt.double() - y1[:, t].double()).norm() <= 2e-5 * y1[:, t].double().norm()
    assert (h.double() - last.double()).norm() <= 2e-5 * last.double().norm()
