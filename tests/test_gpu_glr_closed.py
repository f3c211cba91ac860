"""Closed input gates of the gated recurrence (include/glr.h): sigmoid(i) keeps its value down to
float32's normal range and is 0 at -inf, so that a token which the gate shuts out adds nothing."""
import numpy as np
import pytest
import torch

from oracle import glr as og
from state_space_sequence_gb300 import glr

pytestmark = pytest.mark.gpu

INF = float("inf")
GATES = [-INF, -85.0, -60.0, -45.0, -42.0, -41.0, -1.0]


def host(t):
    return t.detach().double().cpu().numpy()


def near(got, ref, dtype):
    """Channel by channel: within 1e-5 of the channel's norm in float32 (the exponent's rounding,
    2^-18 in base 2 for gates below -44, is 2.7e-6 of the gate), one rounding more in 16 bits, and
    nothing at all where the channel is 0."""
    tol = 1e-5 + (2.0 ** -8 if dtype is torch.bfloat16 else 0.0)
    for c in range(ref.shape[-1]):
        r = ref[..., c]
        assert np.linalg.norm(host(got[..., c]) - r) <= tol * np.linalg.norm(r), c


def normal(seed, *shape, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H", [7, 8, 66])  # single elements, tensor copies, 4-byte copies
def test_gates_near_zero(H, dtype):
    """x of some 1e20 behind gates from open to shut, one gate to a channel, over several tiles."""
    B, L = 2, 300
    x, r = (normal(1, B, L, H) * 1e20).to(dtype), normal(2, B, L, H, dtype=dtype)
    gate = torch.tensor([GATES[c % len(GATES)] for c in range(H)])
    i = gate.expand(B, L, H).to(dtype).cuda()
    p = torch.linspace(-3.0, 1.0, H, device="cuda")
    y, last, _ = glr.glr_scan(x, r, i, p, save_states=True)
    ry, _, rlast = og.scan(host(x), host(r), host(i), host(p), 8.0)
    near(y, ry, dtype)
    near(last, rlast, torch.float32)
    h = torch.zeros(B, H, device="cuda")
    sy, _, sh = og.scan(*(host(t[:, :1]) for t in (x, r, i)), host(p), 8.0)
    out = glr.glr_step(x[:, 0], r[:, 0], i[:, 0], p, h)
    near(out, sy[:, 0], dtype)
    near(h, sh, torch.float32)


@pytest.mark.parametrize("H", [7, 8, 66])
def test_tokens_masked_by_minus_infinity_add_nothing(H):
    """Tokens of ordinary size with the largest float32 values, of either sign, masked among them."""
    B, L = 2, 300
    x, r, i = (normal(k, B, L, H) for k in range(3))
    p = torch.linspace(-3.0, 1.0, H, device="cuda")
    off = torch.rand(B, L, 1, generator=torch.Generator().manual_seed(9)) < 0.3
    off = off.cuda().expand(B, L, H)
    i = torch.where(off, torch.full_like(i, -INF), i)
    zero, huge = torch.where(off, 0.0, x), torch.where(off, torch.sign(x) * 3e38, x)
    for a, b in zip(glr.glr_scan(zero, r, i, p), glr.glr_scan(huge, r, i, p)):
        assert torch.equal(a, b)
    for t in range(12):
        ha, hb = torch.ones(B, H, device="cuda"), torch.ones(B, H, device="cuda")
        a = glr.glr_step(zero[:, t], r[:, t], i[:, t], p, ha)
        b = glr.glr_step(huge[:, t], r[:, t], i[:, t], p, hb)
        assert torch.equal(a, b) and torch.equal(ha, hb)
