"""The example stacks' gradients of their tied table: the rows that tokens are looked up in are also the rows
of the vocabulary that the loss multiplies with, so a row's gradient has both parts. In float32 against
torch's autograd in float64, as the blocks' own tests: within 1e-4 of each gradient's norm."""
import pytest
import torch

from state_space_sequence_gb300 import dlr, gated_block as gb, selective_block as sb

from test_gpu_gated_block import plain as plain_gated
from test_gpu_selective_block import plain

pytestmark = pytest.mark.gpu


def mean_loss(n, table, target):
    z = n.reshape(-1, n.shape[-1]) @ table.t()
    ok = target >= 0
    hit = z.gather(1, target.clamp(min=0)[:, None])[:, 0]
    return (torch.logsumexp(z, 1) - hit)[ok].mean()


def norm(t):
    return t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6)


def batch(B, L, V):
    g = torch.Generator().manual_seed(1)
    tok = torch.randint(0, V - 3, (B, L), generator=g).cuda()  # some rows are never looked up
    target = torch.randint(0, V, (B * L,), generator=g).cuda()
    target[::5] = -1
    reset = torch.zeros(B, L, dtype=torch.bool, device="cuda")
    reset[:, 0] = reset[1, 9] = True
    return tok, target, reset, torch.randn(V, 16, generator=g).cuda()


def test_the_selective_stack():
    torch.backends.cuda.matmul.allow_tf32 = False
    B, L, H, V = 2, 24, 16, 20
    tok, target, reset, embed = batch(B, L, V)
    first = (1 + 0.1 * torch.randn(H, generator=torch.Generator().manual_seed(2))).cuda()
    pars = [sb.make_params(H, E=20, N=5, R=4, dtype=torch.float32, seed=s) for s in (6, 7)]
    losses, grads, de = sb.gradients(pars, embed, first, tok, target, reset)
    leaves = [t.double().requires_grad_(True) for t in (*pars[0], *pars[1], embed)]
    y = leaves[24][tok]
    n = first.double() * norm(y)
    for k in range(2):
        zero = [t.double() for t in sb.start(pars[k], B)]
        y, n = plain(leaves[12 * k:12 * k + 12], y, n, reset, *zero)
    ref = mean_loss(n, leaves[24], target)
    want = torch.autograd.grad(ref, leaves)
    assert abs(losses.double().sum() / (target >= 0).sum() - ref) <= 1e-4 * ref
    for a, q in zip((*grads[0], *grads[1], de), want):
        assert (a.double() - q).norm() <= 1e-4 * q.norm()
    again = sb.gradients(pars, embed, first, tok, target, reset)
    assert torch.equal(again[2], de) and torch.equal(again[0], losses)
    assert dlr.device_status() == 0


def test_the_gated_stack():
    torch.backends.cuda.matmul.allow_tf32 = False
    B, L, H, V = 2, 24, 16, 20
    tok, target, reset, embed = batch(B, L, V)
    target = target.clamp(min=0)
    first = (1 + 0.1 * torch.randn(H, generator=torch.Generator().manual_seed(2))).cuda()
    pars = [gb.make_params(H, torch.float32, seed=s) for s in (6, 7)]
    losses, grads, de = gb.gradients(pars, embed, first, tok, target, reset, ckpt=False)
    leaves = [t.double().requires_grad_(True) for t in (*pars[0], *pars[1], embed)]
    y = leaves[12][tok]
    n = first.double() * norm(y)
    for k in range(2):
        y, n = plain_gated(leaves[6 * k:6 * k + 6], y, n, reset)
    ref = mean_loss(n, leaves[12], target)
    want = torch.autograd.grad(ref, leaves)
    assert abs(losses.double().mean() - ref) <= 1e-4 * ref
    for a, q in zip((*grads[0], *grads[1], de), want):
        assert (a.double() - q).norm() <= 1e-4 * q.norm()
    again = gb.gradients(pars, embed, first, tok, target, reset, ckpt=False)
    assert torch.equal(again[2], de) and torch.equal(again[0], losses)
    assert dlr.device_status() == 0
