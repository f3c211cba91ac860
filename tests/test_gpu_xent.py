"""The softmax cross entropy over a vocabulary on the GPU against its float64 definition
(oracle/xent.py). Losses and their logarithms of sums come from exact products summed in float32:
relative L2 <= 1e-5. A gradient of float32 inputs likewise. One in 16 bits has been rounded twice, d
before its products and the result: each at most 2^-8 (bfloat16, 8 significant bits) or 2^-11
(float16, 11) of each value, the first of values whose sums may cancel, so it is held to the norm of
|d| |W| (or |d|^T |h|); float16 also to its smallest step, 2^-24, half of it each."""
import numpy as np
import pytest
import torch

from oracle import xent as ox
from state_space_sequence_gb300 import dlr, xent

pytestmark = pytest.mark.gpu

TOL = 1e-5
ROUND = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def host(t):
    torch.cuda.synchronize()
    return t.detach().double().cpu().numpy()


def near(got, ref, scale=None):
    assert tuple(got.shape) == np.shape(ref)
    g = host(got)
    assert np.isfinite(g).all()
    err = np.linalg.norm(g - ref)
    rnd = ROUND[got.dtype]
    least = 2.0 ** -25 * np.sqrt(g.size) if got.dtype == torch.float16 else 1e-30
    bound = (TOL + rnd) * np.linalg.norm(ref) + least
    if scale is not None:
        bound += (TOL + rnd) * np.linalg.norm(scale)
    assert err <= bound, (err / max(np.linalg.norm(ref), 1e-300), got.dtype)


def problem(M, V, D, dtype, seed=0, sure=6.0):
    g = torch.Generator().manual_seed(seed + M + V + D)
    W = (torch.randn(V, D, generator=g) / D ** 0.5).to(dtype)
    target = torch.randint(0, V, (M,), generator=g)
    h = (torch.randn(M, D, generator=g) + sure * torch.rand(M, 1, generator=g) *
         W[target].float()).to(dtype)
    dloss = torch.rand(M, generator=g) / M
    return h.cuda(), W.cuda(), target.cuda(), dloss.cuda()


def check(h, W, target, dloss, **how):
    f = [host(h), host(W), target.cpu().numpy()]
    counts = (f[2] >= 0) & (f[2] < len(f[1]))
    loss, lse = xent.xent_loss(h, W, target)
    rl, rs, z = ox.loss(*f)
    near(lse[torch.from_numpy(counts).cuda()], rs[counts])
    # a loss is a difference: held to its parts
    err = np.linalg.norm(host(loss) - rl)
    assert err <= TOL * (np.linalg.norm(rl) + np.linalg.norm(rs[counts])), err
    assert (host(loss)[~counts] == 0).all()
    dh, dW = xent.xent_loss_backward(h, W, target, lse, dloss, **how)
    rh, rW = ox.loss_backward(*f, host(dloss))
    d = np.exp(z - rs[:, None])
    d[np.flatnonzero(counts), f[2][counts]] -= 1.0
    d = np.abs(d) * np.where(counts, host(dloss), 0.0)[:, None]
    if dh is not None:
        near(dh, rh, d @ np.abs(f[1]))
        assert (host(dh)[~counts] == 0).all()
    if dW is not None:
        near(dW, rW, d.T @ np.abs(f[0]))
    assert dlr.device_status() == 0
    return loss, lse, dh, dW


CASES = [(1, 1, 1), (1, 2, 8), (3, 5, 7), (2, 300, 64), (16, 1000, 128), (127, 255, 63),
         (128, 256, 64), (129, 257, 65), (200, 513, 72), (300, 2000, 200), (1, 5003, 520),
         (700, 1500, 321), (1030, 100, 40), (64, 9000, 16)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,V,D", CASES)
def test_loss_and_gradients(M, V, D, dtype):
    h, W, target, dloss = problem(M, V, D, dtype)
    if M > 2:  # padded rows, of every kind
        target[0], target[M // 2], target[-1] = -1, -100, V
    check(h, W, target, dloss * (1 if dtype != torch.float16 else 64.0))
