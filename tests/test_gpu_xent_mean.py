"""Gradients of a mean in 16 bits. All logits 0 over 64 columns: every probability is 1 / 64 and d is dloss
times numbers of six bits, so that dh and dW are those times one number of W (or of h) each and have one
rounding, their own, at most 2^-8 (bfloat16) or 2^-11 (float16), whatever the number of rows that the mean
is over; the float32 products before it and lse's 2^-24 of 4.2 are off by less than 2^-20."""
import math

import pytest
import torch

from state_space_sequence_gb300 import dlr, xent

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M", [24, 192])
def test_one_rounding(M, dtype):
    V = D = 64
    target = (torch.arange(M) % V).cuda()
    h = torch.zeros(M, D, dtype=dtype, device="cuda")
    d = torch.full((M, V), 1 / 64, dtype=torch.float64, device="cuda")
    d[torch.arange(M), target] -= 1.0
    scale = 2.0 ** 12 if dtype == torch.float16 else 1.0  # a loss scale keeps results in float16's range
    worst = 0.0
    for k in range(48):
        count = 7000 + 37 * k
        dloss = torch.full((M,), scale / count, device="cuda")
        c = 1.0 + (2 * k + 1) / 128
        W = (c * torch.eye(V, device="cuda")).to(dtype)
        _, lse = xent.xent_loss(h, W, target)
        dh, _ = xent.xent_loss_backward(h, W, target, lse, dloss, wanted=(True, False))
        ref = d @ W.double() * dloss.double()[:, None]
        off = ((dh.double() - ref).abs() / ref.abs().clamp(min=1e-30)).max().item()
        assert off <= HALF[dtype] + 2.0 ** -20, (count, off)
        worst = max(worst, off)
        # dW: one row of h that is not zero, on columns whose logits W leaves at 0
        h2, W2 = torch.zeros_like(h), torch.zeros_like(W)
        h2[5] = c
        _, lse = xent.xent_loss(h2, W2, target)
        _, dW = xent.xent_loss_backward(h2, W2, target, lse, dloss, wanted=(False, True))
        ref = d.t() @ h2.double() * dloss.double()[0]
        off = ((dW.double() - ref).abs() / ref.abs()).max().item()
        assert off <= HALF[dtype] + 2.0 ** -20, (count, off)
    assert worst > HALF[dtype] / 2 and math.isfinite(worst)
    assert dlr.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_weights_of_any_size(dtype):
    """Weights of zero, of one row alone, enormous and tiny ones, and an infinite one, which stays its row's."""
    M, V, D = 40, 70, 24
    g = torch.Generator().manual_seed(1)
    h, W = (torch.randn(n, D, generator=g).to(dtype).cuda() / 4 for n in (M, V))
    target = torch.randint(0, V, (M,), generator=g).cuda()
    _, lse = xent.xent_loss(h, W, target)
    z = h.double() @ W.double().t()
    d = torch.exp(z - lse.double()[:, None])
    d[torch.arange(M), target] -= 1.0
    for w in (0.0, 1.0, 2.0 ** -12, 2.0 ** 12, 2.0 ** -80, 2.0 ** 90):
        if dtype == torch.float16 and abs(math.log2(w or 1)) > 20:
            continue
        dloss = torch.full((M,), w, device="cuda")
        dloss[::3] *= 0.3
        dloss[7] = 0.0
        dh, dW = xent.xent_loss_backward(h, W, target, lse, dloss)
        e = d * dloss.double()[:, None]
        least = 2.0 ** -25 if dtype == torch.float16 else 0.0
        for a, r, size in ((dh, e @ W.double(), e.abs() @ W.double().abs()),
                           (dW, e.t() @ h.double(), e.abs().t() @ h.double().abs())):
            assert ((a.double() - r).abs() <= (2 * HALF[dtype] + 1e-5) * size + least).all()
        assert not dh[7].any()
    dloss = torch.ones(M, device="cuda")
    dloss[3] = float("inf")
    dh, _ = xent.xent_loss_backward(h, W, target, lse, dloss, wanted=(True, False))
    rows = torch.arange(M) != 3
    r = (d @ W.double())[rows]
    assert ((dh[rows].double() - r).abs() <= (2 * HALF[dtype] + 1e-5) * (d.abs() @ W.double().abs())[rows] +
            2.0 ** -25).all()
    assert not torch.isfinite(dh[3]).any()
    assert dlr.device_status() == 0
