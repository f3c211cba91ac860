"""The scan's decays one by one: states and their gradients of which nothing but exp(s A) is made, against
float64. In float32 a decay is off by the rounding of its exponent, s A log2(e) from three rounded
numbers (2^-24 each, and 2^-26 of log2(e)): 3.25 * 2^-24 of s |A|, by the unit's 2^-22, and where it is
next to 1 by its polynomial's 2^-25; each step rounds the state by 2^-24."""
import numpy as np
import pytest
import torch

from state_space_sequence_gb300 import dlr, ssm

pytestmark = pytest.mark.gpu

RATES = [-1.0, -16.0, -64.0]


def host(t):
    torch.cuda.synchronize()
    return t.detach().double().cpu().numpy()


def decays(L, per_call=40.0):
    """Steps [1, 1, H] (the same in all of a call's L steps) and rates [H, 4] whose exponents over the call
    go from 0.01 to `per_call`; the exact decay of a call, [H, 4]."""
    total = torch.logspace(-2, float(np.log10(per_call)), 33, dtype=torch.float64)
    A = torch.tensor([RATES[k % 3] for k in range(33 * 3)])[:, None] * torch.tensor([1.0, 1.0, 0.5, 0.75])
    s = (total.repeat_interleave(3) / L / -A[:, 0].double()).float()
    return s[None, None].cuda(), A.cuda(), L * s.double().numpy()[:, None] * A.double().numpy()


def bound(L, z):
    return L * 2.0 ** -24 * (1 + 2.0 ** 2) + 3.25 * 2.0 ** -24 * np.abs(z)


def within(got, ref, tol):
    g = host(got)
    assert np.isfinite(g).all()
    assert (np.abs(g - ref) <= tol * np.abs(ref)).all(), (np.abs(g / ref - 1) / tol).max()


def test_a_step_keeps_the_digits_of_small_decays():
    s, A, z = decays(1)
    H, N = A.shape
    gen = torch.Generator().manual_seed(1)
    h = torch.randn(1, H, N, generator=gen).cuda()
    zero, maps = torch.zeros(1, H, device="cuda"), torch.ones(1, N, device="cuda")
    ref = host(h) * np.exp(z)
    assert (bound(1, z) < 1e-5).all()
    y = ssm.ssm_step(zero, s[0], A, maps, maps, h, softplus=False)
    within(h, ref, bound(1, z))
    assert (np.abs(host(y) - ref.sum(-1)) <= 1.1e-5 * np.abs(ref).sum(-1)).all()


@pytest.mark.parametrize("L", [1, 2, 16, 40])
def test_a_scan_keeps_the_digits_of_small_decays(L):
    """And its gradients: dh0 = a G, dA = sum of s a G h, ddt the like, for a loss of the last state."""
    s, A, z = decays(L)
    H, N = A.shape
    gen = torch.Generator().manual_seed(2)
    h0, G = (torch.randn(1, H, N, generator=gen).cuda() for _ in range(2))
    x, maps = torch.zeros(1, L, H, device="cuda"), torch.ones(1, L, N, device="cuda")
    dt = s.expand(1, L, H)
    y, last, st = ssm.ssm_scan(x, dt, A, maps, maps, softplus=False, h0=h0, save_states=True)
    ref, tol = host(h0) * np.exp(z), bound(L, z)
    within(last, ref, tol)
    g = ssm.ssm_scan_backward(x, dt, A, maps, maps, x, st, softplus=False, h0=h0, dh_last=G)
    within(g.dh0, host(G) * np.exp(z), tol)
    # every step's term is the same: s a^L h0 G, a few roundings and L additions more
    dA = host(G)[0] * ref[0] * (L * host(s)[0, 0][:, None])
    within(g.dA, dA, (tol + (L + 6) * 2.0 ** -24)[:])
    terms = host(G)[0] * ref[0] * host(A)
    assert (np.abs(host(g.ddt)[0] - terms.sum(-1)) <= (tol.max(-1) + 1e-6) * np.abs(terms).sum(-1)).all()
    assert dlr.device_status() == 0


@pytest.mark.parametrize("H", [3, 99])
def test_a_cut_sequence_decays_as_a_whole_one(H):
    """400 steps, few channels: the sequence is cut, and the cuts' decays joined."""
    L = 400
    s, A, z = decays(L)
    s, A, z = s[..., :H].contiguous(), A[:H].contiguous(), z[:H]
    N = A.shape[1]
    h0 = torch.randn(1, H, N, generator=torch.Generator().manual_seed(3)).cuda()
    assert ssm.ssm_scan_workspace_size(1, L, H, N) > 0
    x, maps = torch.zeros(1, L, H, device="cuda"), torch.ones(1, L, N, device="cuda")
    dt = s.expand(1, L, H)
    _, last, st = ssm.ssm_scan(x, dt, A, maps, maps, softplus=False, h0=h0, save_states=True)
    # the sum of a cut's steps has a rounding for each of them
    tol = bound(L, z) + L * 2.0 ** -24 * np.abs(z)
    within(last, host(h0) * np.exp(z), tol)
    g = ssm.ssm_scan_backward(x, dt, A, maps, maps, x, st, softplus=False, h0=h0, dh_last=h0)
    within(g.dh0, host(h0) * np.exp(z), tol)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("L", [1, 5, 40, 700])
def test_an_infinite_state_stays_infinite(L, dtype):
    """As exp(s A) times infinity is, whether the decay is 1, next to it or far from it, and in a cut
    sequence, over whose parts the decays underflow."""
    steps = torch.tensor([0.0, 1e-4, 0.01, 0.2, 1.0, 1.5])
    H, N = len(steps), 4
    A = torch.tensor([-1.0, -2.0, -16.0, -0.5]).repeat(H, 1).cuda()
    h = torch.full((1, H, N), float("inf"), device="cuda")
    h[:, :, 1::2] *= -1
    first = h.clone()
    dt = steps.to(dtype).cuda()[None, None].expand(1, L, H)
    x = torch.ones(1, L, H, dtype=dtype, device="cuda")
    B = torch.ones(1, L, N, dtype=dtype, device="cuda")
    C = torch.tensor([1.0, -1.0, 1.0, -1.0], dtype=dtype, device="cuda").expand(1, L, N)
    y, last, st = ssm.ssm_scan(x, dt, A, B, C, softplus=False, h0=h, save_states=True)
    assert torch.equal(last, first) and (y == float("inf")).all()
    assert torch.equal(st, first[:, None].expand(st.shape))
    zero = torch.zeros_like(x)
    finite = torch.zeros_like(st)
    g = ssm.ssm_scan_backward(x, dt, A, B, C, zero, finite, softplus=False, h0=torch.zeros_like(h),
                              dh_last=first)
    assert torch.equal(g.dh0, first)
    y = ssm.ssm_step(x[:, 0], dt[:, 0], A, B[:, 0], C[:, 0], h, softplus=False)
    assert torch.equal(h, first) and (y == float("inf")).all()


def test_a_cut_sequence_that_grows_from_nothing():
    """Steps below zero (without softplus) let a state grow; over a part of a cut sequence its factor
    overflows, but what is zero stays zero, and what begins behind it is what it is."""
    L, H, N = 700, 6, 4
    A = -torch.ones(H, N, device="cuda")
    dt = torch.full((1, L, H), -8.0, device="cuda")
    x, maps = torch.zeros(1, L, H, device="cuda"), torch.ones(1, L, N, device="cuda")
    x[:, -5] = 1.0
    assert ssm.ssm_scan_workspace_size(1, L, H, N) > 0
    _, last, st = ssm.ssm_scan(x, dt, A, maps, maps, softplus=False, save_states=True)
    assert (np.abs(host(last) / (-8 * np.exp(32.0)) - 1) <= 1e-5).all() and not st[:, :-1].any()
    g = ssm.ssm_scan_backward(x, dt, A, maps, maps, torch.zeros_like(x), st, softplus=False,
                              h0=torch.zeros(1, H, N, device="cuda"))
    assert not g.dh0.any() and not g.dx.any()
