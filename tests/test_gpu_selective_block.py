"""The example block of the selective scan (selective_block.py): its operators run together, against
torch's autograd in float64 on the same values, token by token against the whole sequence, and with
the loss over a vocabulary; both example commands run."""
import pytest
import torch

from state_space_sequence_gb300 import dlr, gated_block, selective_block as sb, xent

pytestmark = pytest.mark.gpu


def plain(par, y, n, reset, inputs, h):
    """The block from its formulas, step by step, for autograd."""
    Wxz, taps, tap_bias, Wp, Wdt, dt_bias, A, D, Wo, w, alpha, v = par
    (E, K), N, R = taps.shape, A.shape[1], Wdt.shape[0]
    B, L, _ = y.shape
    x, z = (n @ Wxz).split(E, -1)
    silu = lambda t: t * torch.sigmoid(t)
    os = []
    for t in range(L):
        cut = reset[:, t, None, None]
        inputs = torch.where(cut, torch.zeros_like(inputs), inputs)
        h = torch.where(cut, torch.zeros_like(h), h)
        line = torch.cat([inputs, x[:, t, None]], 1)
        u = silu(tap_bias + (line * taps.t()).sum(1))
        inputs = line[:, 1:]
        low, Bm, Cm = (u @ Wp).split([R, N, N], -1)
        s = torch.nn.functional.softplus(low @ Wdt + dt_bias, threshold=700)
        h = torch.exp(-s[..., None] * torch.exp(A)) * h + (s * u)[..., None] * Bm[:, None]
        os.append(((h * Cm[:, None]).sum(-1) + D * u) * silu(z[:, t]))
    norm = lambda t: t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6)
    y = y + alpha * w * norm(torch.stack(os, 1) @ Wo)
    return y, v * norm(y)


def inputs(B, L, H, seed, dtype=torch.float32):
    gen = torch.Generator().manual_seed(seed)
    return [torch.randn(B, L, H, generator=gen).to(dtype).cuda() for _ in range(4)]


def test_block_gradients_in_float32():
    """Every product and operator in float32: within 5e-5 of each gradient's norm (1e-5 an operator,
    five of them in a row, and the library's products in full float32)."""
    torch.backends.cuda.matmul.allow_tf32 = False
    B, L, H = 2, 40, 24
    y, n, dy, dn = inputs(B, L, H, 3)
    reset = torch.zeros(B, L, dtype=torch.bool, device="cuda")
    reset[0, 17] = reset[1, 32] = True
    par = sb.make_params(H, E=36, N=6, R=5, dtype=torch.float32, seed=5)
    first = sb.State(*(torch.randn_like(t) for t in sb.start(par, B)))
    y1, n1, _, saved = sb.forward(par, y, n, first, reset)
    got_y, got_n, grads = sb.backward(par, saved, dy, dn)
    args = [t.double().requires_grad_(True) for t in (*par, y, n)]
    ry, rn = plain(args[:12], args[12], args[13], reset, *(t.double() for t in first))
    ref = torch.autograd.grad([ry, rn], args, [dy.double(), dn.double()])
    for a, q in zip((y1, n1, *grads, got_y, got_n), (ry, rn, *ref)):
        assert (a.double() - q).norm() <= 5e-5 * q.norm()
    assert dlr.device_status() == 0


def test_two_blocks_and_their_loss_in_float32():
    """A stack under the loss, its gradients down to the embedding: as above, twice, and the loss."""
    torch.backends.cuda.matmul.allow_tf32 = False
    B, L, H, V = 2, 20, 16, 50
    y, n, _, _ = inputs(B, L, H, 4)
    reset = torch.zeros(B, L, dtype=torch.bool, device="cuda")
    reset[:, 0] = True
    pars = [sb.make_params(H, E=20, N=5, R=4, dtype=torch.float32, seed=s) for s in (6, 7)]
    table = torch.randn(V, H, generator=torch.Generator().manual_seed(8)).cuda()
    target = torch.arange(B * L, device="cuda") % V
    target[::6] = -1
    weight = torch.rand(B * L, device="cuda")
    a, b, saved = y, n, []
    for p in pars:
        a, b, _, s = sb.forward(p, a, b, reset=reset)
        saved.append(s)
    loss, lse = xent.xent_loss(b.view(-1, H), table, target)
    dn, dtable = xent.xent_loss_backward(b.view(-1, H), table, target, lse, weight)
    dn, dy, grads = dn.view_as(n), torch.zeros_like(y), []
    for p, s in zip(pars[::-1], saved[::-1]):
        dy, dn, g = sb.backward(p, s, dy, dn)
        grads = [*g, *grads]
    leaves = [t.double().requires_grad_(True) for t in (*pars[0], *pars[1], y, n, table)]
    a, b = leaves[24], leaves[25]
    for k in range(2):
        zero = [t.double() for t in sb.start(pars[k], B)]
        a, b = plain(leaves[12 * k:12 * k + 12], a, b, reset, *zero)
    z = b.reshape(-1, H) @ leaves[26].t()
    ok = target >= 0
    ref = torch.where(ok, torch.logsumexp(z, 1) - z.gather(1, target.clamp(min=0)[:, None])[:, 0], 0.0)
    want = torch.autograd.grad((ref * weight).sum(), leaves)
    assert (loss.double() - ref).norm() <= 1e-4 * ref.norm()
    for g, q in zip((*grads, dy, dn, dtable), want):
        assert (g.double() - q).norm() <= 1e-4 * q.norm()


def test_steps_are_the_block():
    B, L, H = 3, 30, 32
    torch.backends.cuda.matmul.allow_tf32 = False
    y, n, _, _ = inputs(B, L, H, 5)
    par = sb.make_params(H, dtype=torch.float32, seed=7)
    y1, n1, last, _ = sb.forward(par, y, n)
    state = sb.start(par, B)
    for t in range(L):
        yt, nt = sb.step(par, y[:, t], n[:, t], state)
        for a, q in ((nt, n1[:, t]), (yt, y1[:, t])):
            assert (a.double() - q.double()).norm() <= 5e-5 * q.double().norm()
    for a, q in zip(state, last):
        assert (a.double() - q.double()).norm() <= 5e-5 * q.double().norm()


@pytest.mark.parametrize("block", [sb, gated_block])
def test_the_commands_run(block, capsys):
    block.main(steps=2)
    out = capsys.readouterr().out
    assert "step   0  loss" in out and "decoded 192 tokens of 16 rows" in out
    assert dlr.device_status() == 0
