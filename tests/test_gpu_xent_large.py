"""The softmax cross entropy where offsets pass 32 bits, held to closed forms: a vocabulary whose rows
are zero but for a few, and many rows over a small one. Tolerances as in test_gpu_xent.py."""
import numpy as np
import pytest
import torch

from oracle import xent as ox
from state_space_sequence_gb300 import dlr, xent

from test_gpu_xent import TOL, host, near, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,V", [(torch.bfloat16, 1050000), (torch.float32, 400000)])
def test_a_vocabulary_past_32_bits(dtype, V):
    """V D, or the three parts of it, exceed 2^31 elements. With W zero but in `rows` (which stand at
    the ends and around 2^31 elements), every other logit is 0: lse = log(V - rows + sum exp z)."""
    M, D = 18, 2048
    at = 2 ** 31 // D if dtype is torch.bfloat16 else V // 2
    rows = [0, 1, 255, 256, at - 1, at, V // 3, V - 2, V - 1]
    g = torch.Generator().manual_seed(5)
    few = (torch.randn(len(rows), D, generator=g) / D ** 0.5 * 8).to(dtype)
    W = torch.zeros(V, D, dtype=dtype, device="cuda")
    W[rows] = few.cuda()
    target = torch.tensor([rows[k % len(rows)] for k in range(M - 2)] + [V, 777])
    # logits of about 13 +- 8 at some row, so that it has a good part of the sum
    k = torch.arange(M) % len(rows)
    h = (torch.randn(M, D, generator=g) + 0.2 * few[k].float()).to(dtype).cuda()
    dloss = torch.rand(M, generator=g)
    loss, lse = xent.xent_loss(h, W, target.cuda())
    z = host(h) @ few.double().numpy().T
    rs = np.log(V - len(rows) + np.exp(z).sum(1))
    near(lse, rs)
    zt = np.array([z[m, rows.index(t)] if t in rows else 0.0 for m, t in enumerate(target.tolist())])
    counts = target.numpy() < V
    rl = np.where(counts, rs - zt, 0.0)
    assert np.linalg.norm(host(loss) - rl) <= TOL * (np.linalg.norm(rl) + np.linalg.norm(rs))
    dh, dW = xent.xent_loss_backward(h, W, target.cuda(), lse, dloss.cuda())
    weight = np.where(counts, dloss.double().numpy(), 0.0)
    hit = np.array([[float(t == r) for r in rows] for t in target.tolist()])
    d = weight[:, None] * (np.exp(z - rs[:, None]) - hit)
    few = few.double().numpy()
    near(dh, d @ few, np.abs(d) @ np.abs(few))
    near(dW[rows], d.T @ host(h), np.abs(d).T @ np.abs(host(h)))
    # the others: one value of d for each row of h
    rest = weight * np.exp(-rs)
    one = rest @ host(h)
    size = rest @ np.abs(host(h))
    others = [2, 257, at + 1, V // 2 + 1, V - 3]
    near(dW[others], np.tile(one, (len(others), 1)), np.tile(size, (len(others), 1)))
    hit = rest.copy()
    hit[-1] -= weight[-1]  # row 777 is the last one's target
    near(dW[777], hit @ host(h), np.abs(hit) @ np.abs(host(h)))
    plain = torch.ones(V, dtype=torch.bool, device="cuda")
    plain[rows + [777]] = False
    assert torch.equal(dW[plain].amax(0), dW[plain].amin(0))
    assert dlr.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_rows(dtype):
    M, V, D = 100001, 300, 40
    h, W, target, dloss = problem(M, V, D, dtype)
    target[::7] = -1
    f = [host(h), host(W), target.cpu().numpy()]
    loss, lse = xent.xent_loss(h, W, target)
    rl, rs, z = ox.loss(*f)
    counts = f[2] >= 0
    near(lse, rs)
    assert np.linalg.norm(host(loss) - rl) <= TOL * (np.linalg.norm(rl) + np.linalg.norm(rs))
    dh, dW = xent.xent_loss_backward(h, W, target, lse, dloss)
    d = np.exp(z - rs[:, None])
    d[np.flatnonzero(counts), f[2][counts]] -= 1.0
    d *= np.where(counts, host(dloss), 0.0)[:, None]
    near(dh, d @ f[1], np.abs(d) @ np.abs(f[1]))
    near(dW, d.T @ f[0], np.abs(d).T @ np.abs(f[0]))
    assert dlr.device_status() == 0
