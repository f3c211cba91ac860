"""The loss's gradients value by value. With W the unit matrix the logits are h itself and dh is d, so every
exp(z - lse) can be held to the definition, with the lse that the call was given: z and lse are exact
numbers of up to some hundreds, their difference is off by 2^-24 of itself (z itself by nothing: it has
eight digits), its product with log2(e) by 1.25 * 2^-24 more, and the unit by 2^-22: (4 + 2.25 |z - lse|)
2^-24 of each term in all, and four roundings of the product with dloss and of d's way through three
parts."""
import numpy as np
import pytest
import torch

from state_space_sequence_gb300 import dlr, xent

pytestmark = pytest.mark.gpu


def host(t):
    torch.cuda.synchronize()
    return t.detach().double().cpu().numpy()


def rows(M, V, top, seed):
    """Logits of 8 significant bits: a random one of each row is `top`, the others lie up to some 20 lower."""
    g = torch.Generator().manual_seed(seed)
    unit = 2.0 ** (np.floor(np.log2(max(top, 20.0))) - 7)
    below = torch.randint(0, int(20 / unit) + 1, (M, V), generator=g).double() * unit
    z = top - below
    first = torch.randint(0, V, (M,), generator=g)
    z[torch.arange(M), first] = top
    return z.float().cuda(), first.cuda()


def check(z, target, weight):
    M, V = z.shape
    assert torch.equal(z, z.bfloat16().float())
    W = torch.eye(V, device="cuda")
    _, lse = xent.xent_loss(z, W, target)
    dh, _ = xent.xent_loss_backward(z, W, target, lse, weight)
    x = host(z) - host(lse)[:, None]
    p, w = np.exp(x), host(weight)[:, None]
    d = p.copy()
    d[np.arange(M), target.cpu().numpy()] -= 1.0
    tol = (4 + 2.25 * np.abs(x)) * 2.0 ** -24 * p + 4 * 2.0 ** -24 * np.abs(d)
    off = np.abs(host(dh) - w * d) / (w * tol + 1e-37)
    assert off.max() <= 1, off.max()
    assert dlr.device_status() == 0
    return d


@pytest.mark.parametrize("top", [3.0, 20.0, 100.0, 300.0, 508.0, 1000.0])
@pytest.mark.parametrize("M", [5, 200])
def test_every_term_of_a_row(M, top):
    z, _ = rows(M, 96, top, seed=M)
    g = torch.Generator().manual_seed(1)
    check(z, torch.randint(0, 96, (M,), generator=g).cuda(), torch.rand(M, generator=g).cuda() + 0.1)


@pytest.mark.parametrize("top", [20.0, 100.0, 508.0])
def test_rows_that_are_sure(top):
    """Losses of about 0.006: the target's gradient is what its probability lacks of 1."""
    M, V = 40, 64
    _, first = rows(M, V, top, seed=2)
    unit = 2.0 ** (np.floor(np.log2(top)) - 7)
    z = torch.full((M, V), top - np.ceil(9.25 / unit) * unit, device="cuda")
    z[torch.arange(M), first] = top
    d = check(z, first, torch.ones(M, device="cuda"))
    sure = -d[np.arange(M), first.cpu().numpy()]
    assert (sure > 1e-3).all() and (sure < 0.01).all()
