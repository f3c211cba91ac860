"""Decays of 16-bit inputs over a long memory: one rounded number a channel, off by up to 2^-24 of itself
either way, which over 8192 steps is 5e-4 of a state, but over many channels nothing. The exponent's
addend takes out what the special-function unit leaves on one side, 1.9e-8 a step: 1.6e-4 over the
memory. With that known to 0.1e-8 (8e-6) and the mean over 4096 channels good to 3 * 1.4e-4 / 64 = 7e-6,
a mean signed error within 4e-5 tells the right addend from none and from one of the other sign."""
import numpy as np
import pytest
import torch

from state_space_sequence_gb300 import ssm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_the_mean_of_many_long_memories(dtype):
    L, H, N = 8192, 1024, 4
    g = torch.Generator().manual_seed(1)
    step = 2.0 ** -(12 + 3 * torch.rand(H, generator=g))
    A = -(1 + torch.rand(H, N, generator=g))
    zero = torch.zeros(1, L, H, dtype=dtype, device="cuda")
    maps = torch.zeros(1, L, N, dtype=dtype, device="cuda")
    _, last = ssm.ssm_scan(zero, zero, A.cuda(), maps, maps, dt_bias=step.cuda(), softplus=False,
                           h0=torch.ones(1, H, N, device="cuda"))
    ref = np.exp(L * step.double().numpy()[:, None] * A.double().numpy())
    off = last[0].double().cpu().numpy() / ref - 1
    assert abs(off).max() <= 1.5 * 2.0 ** -24 * L + 1e-5
    assert abs(off.mean()) <= 4e-5, off.mean()
