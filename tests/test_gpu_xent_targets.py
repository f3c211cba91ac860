"""Losses of sure rows, small beside the logit that they hang on. One vocabulary row has a logit of about 10,
all terms of one sign, the others 0: the loss is log(1 + (V - 1) exp(-z)), off relative to itself by what z is
off by: D / 256 + 8 roundings of 2^-24 of z where it is formed for itself, at most 256 / 16 steps of 2^-23 and
D / 256 roundings in few rows' tiles; the last few operations, and log(V - 1), add 2^-20. The gradient is
exp(z - lse) - 1, lse being rounded to 2^-24 of itself."""
import numpy as np
import pytest
import torch

from state_space_sequence_gb300 import dlr, xent

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def problem(M, V, D, at, dtype, z=9.7, pad=0):
    g = torch.Generator(device="cuda").manual_seed(M + D)
    h = (0.5 + 0.5 * torch.rand(M, D + pad, generator=g, device="cuda")).to(dtype)[:, :D]
    W = torch.zeros(V, D + pad, dtype=dtype, device="cuda")[:, :D]
    W[at] = ((0.5 + 0.5 * torch.rand(D, generator=g, device="cuda")) * (z / (0.5625 * D))).to(dtype)
    return h, W, torch.full((M,), at, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,V,D,at,pad", [(200, 100, 2048, 7, 0), (129, 300, 1000, 299, 0), (200, 100, 4096, 0, 0),
                                          (5000, 400, 1999, 256, 1), (200, 100, 2047, 99, 0),
                                          (100, 100, 2048, 7, 0), (3, 2, 77, 1, 3)])
def test_the_loss_of_a_sure_row(M, V, D, at, pad, dtype):
    h, W, target = problem(M, V, D, at, dtype, pad=pad)
    target[::7] = -1
    ok = target >= 0
    loss, lse = xent.xent_loss(h, W, target)
    z = h.double() @ W[at].double()
    ref = torch.log1p((V - 1) * torch.exp(-z))
    off = (16 * 2.0 ** -23 if M <= 128 else 0.0) + (D / 256 + 8) * 2.0 ** -24
    tol = off * float(z.max()) + 2.0 ** -20
    assert ((loss.double() - ref).abs()[ok] <= tol * ref[ok]).all()
    assert not loss[~ok].any()
    assert ((lse.double() - (z + ref)).abs() <= (tol + 2.0 ** -23 * float(z.max())) +
            (0.0 if M <= 128 else D / 16 * 2.0 ** -23 * float(z.max())) * (~ok)).all()
    dh, _ = xent.xent_loss_backward(h, W, target, lse, torch.ones(M, device="cuda"), wanted=(True, False))
    p = -torch.expm1(-ref)
    want = -p[:, None] * W[at].double() * ok[:, None]
    slack = 2 * HALF[dtype] + tol + 2.0 ** -24 * float(lse.max()) / p[:, None]
    least = 2.0 ** -25 if dtype == torch.float16 else 1e-30
    assert ((dh.double() - want).abs() <= slack * want.abs() + least).all()
    assert dlr.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M", [4, 150])
def test_one_column_and_the_ends_of_the_range(M, dtype):
    """A vocabulary of one, logits of minus and plus infinity, and a NaN that stays its row's."""
    D = 16
    h = torch.ones(M, D, dtype=dtype, device="cuda")
    target = torch.zeros(M, dtype=torch.int64, device="cuda")
    W = torch.full((1, D), 0.25, dtype=dtype, device="cuda")
    loss, lse = xent.xent_loss(h, W, target)
    assert not loss.any() and (lse == 4.0).all()
    dh, dW = xent.xent_loss_backward(h, W, target, lse, torch.ones(M, device="cuda"))
    assert not dh.any() and not dW.any()
    if dtype == torch.float32:  # an infinity's other parts are zeros, whose products with it are not
        return
    W = torch.zeros(3, D, dtype=dtype, device="cuda")
    W[1, 0] = -float("inf")
    loss, lse = xent.xent_loss(h, W, target)
    assert np.allclose(lse.cpu().numpy(), np.log(2.0), rtol=1e-6)
    assert np.allclose(loss.cpu().numpy(), np.log(2.0), rtol=1e-6)
    loss, lse = xent.xent_loss(h, W, target + 1)
    assert (loss == float("inf")).all() and np.allclose(lse.cpu().numpy(), np.log(2.0), rtol=1e-6)
    bad = h.clone()
    bad[2, 3] = float("nan")
    loss, lse = xent.xent_loss(bad, torch.zeros_like(W), target)
    rows = torch.arange(M, device="cuda") != 2
    assert torch.isnan(loss[2]) and torch.isnan(lse[2])
    assert np.allclose(loss[rows].cpu().numpy(), np.log(3.0), rtol=1e-6)
    assert dlr.device_status() == 0
