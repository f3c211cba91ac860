"""The selective state space block's operators on the GPU against their float64 definitions
(oracle/ssm.py): relative L2 <= 1e-5 for float32 outputs; an output stored in 16 bits adds its
rounding, at most 2^-8 (bfloat16, 8 significant bits) or 2^-11 (float16, 11) of each value, and
2^-25 where that is more: below 2^-14 float16's values are 2^-24 apart."""
import numpy as np
import pytest
import torch

from oracle import ssm as osm
from state_space_sequence_gb300 import dlr, ssm

pytestmark = pytest.mark.gpu

TOL = 1e-5
ROUND = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def host(t):
    torch.cuda.synchronize()
    return None if t is None else t.detach().double().cpu().numpy()


def close(got, ref, scale=None):
    """``scale``: the norm to compare with, where the reference's own may cancel."""
    assert tuple(got.shape) == np.shape(ref)
    g = host(got)
    assert np.isfinite(g).all()
    norm = np.linalg.norm(ref) if scale is None else scale
    err = np.linalg.norm(g - ref)
    least = 2.0 ** -25 * np.sqrt(g.size) if got.dtype == torch.float16 else 1e-30
    assert err <= (TOL + ROUND[got.dtype]) * norm + least, (err / max(norm, 1e-300), got.dtype)


def normal(seed, *shape, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def arrays(layout, n, seed, B, L, H, dtype):
    """n activations [B, L, H] in one of the layouts a caller may have."""
    if layout == "apart":
        return [normal(seed + k, B, L, H, dtype=dtype) for k in range(n)]
    if layout == "columns":  # of one projection's output
        z = normal(seed, B, L, n * H, dtype=dtype)
        return [z[..., k * H:(k + 1) * H] for k in range(n)]
    if layout == "time first":
        return [normal(seed + k, L, B, H, dtype=dtype).transpose(0, 1) for k in range(n)]
    assert layout == "broadcast"  # over the batch, and one of them over time as well
    out = [normal(seed + k, 1, L, H, dtype=dtype).expand(B, L, H) for k in range(n)]
    out[-1] = normal(seed + 77, 1, 1, H, dtype=dtype).expand(B, L, H)
    return out


def resets(seed, B, L, count):
    m = torch.zeros(B, L, dtype=torch.bool)
    g = np.random.default_rng(seed)
    for b in range(B):
        m[b, g.integers(0, L, count)] = True
    return m.cuda()


CONV_CASES = [
    # B, L, H, K, layout, state, resets, activation
    (1, 1, 1, 4, "apart", False, 0, "silu"), (2, 1, 33, 4, "apart", True, 1, "silu"),
    (1, 2, 8, 4, "columns", True, 0, "silu"), (3, 7, 5, 3, "columns", True, 2, "none"),
    (2, 16, 64, 4, "apart", True, 0, "silu"), (2, 17, 64, 2, "columns", False, 3, "silu"),
    (1, 33, 66, 4, "time first", False, 0, "silu"), (3, 129, 31, 4, "broadcast", True, 2, "silu"),
    (2, 200, 130, 3, "columns", True, 64, "silu"), (1, 1000, 96, 8, "time first", True, 5, "silu"),
    (2, 65, 264, 4, "columns", False, 9, "silu"), (5, 321, 17, 5, "apart", True, 4, "none"),
    (2, 40, 40, 1, "apart", False, 3, "silu"), (4, 3, 256, 8, "apart", True, 1, "silu"),
    (3, 515, 520, 4, "columns", True, 40, "silu"),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,L,H,K,layout,start,cuts,act", CONV_CASES)
def test_convolution_and_its_gradients(B, L, H, K, layout, start, cuts, act, dtype):
    seed = B + 10 * L + H
    x, dy = arrays(layout, 2, seed, B, L, H, dtype)
    w, bias = normal(seed + 20, H, K) / K ** 0.5, normal(seed + 21, H)
    state, dlast = (normal(seed + k, B, K - 1, H, dtype=dtype) if start else None
                    for k in (22, 23))
    reset = resets(seed, B, L, cuts) if cuts else None
    cut = None if reset is None else reset.cpu().numpy()
    f = [host(t) for t in (x, w)]
    y, last = ssm.ssm_conv(x, w, bias, state, reset, act)
    ry, rl, _ = osm.conv(*f, host(bias), host(state), cut, act)
    close(y, ry)
    if K > 1:
        assert np.array_equal(host(last), rl)
    else:
        assert last is None
    out = None
    if layout == "columns":
        out = torch.full((B, L, 2 * H), float("nan"), dtype=dtype, device="cuda")[..., H:]
    got = ssm.ssm_conv_backward(x, w, dy, bias, state, reset, act, dlast=dlast, out=out)
    ref = osm.conv_backward(*f, host(dy), host(bias), host(state), cut, act, host(dlast))
    for a, r in zip(got, ref):
        if a is not None:
            close(a, r)
    assert (got[3] is None) == (not start)
    assert dlr.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,H,K", [(1, 1, 4), (3, 33, 2), (5, 64, 4), (2, 520, 8), (7, 24, 1),
                                   (300, 136, 3)])
def test_convolution_steps(B, H, K, dtype):
    """Token by token, in place and beside, the sequence's results; marked entries begin anew."""
    L = 6
    x = normal(1, B, L, H, dtype=dtype)
    w, bias = normal(2, H, K), normal(3, H)
    reset = resets(4, B, L, 1)
    state = normal(5, B, K - 1, H, dtype=dtype) if K > 1 else None
    y, last = ssm.ssm_conv(x, w, bias, state, reset)
    for t in range(L):
        cut = reset[:, t].contiguous()
        if t % 2 or K == 1:
            o = ssm.ssm_conv_step(x[:, t], w, state, bias, cut)
        else:
            nxt = torch.empty_like(state)
            o = ssm.ssm_conv_step(x[:, t], w, state, bias, cut, state_out=nxt)
            state = nxt
        assert (o.double() - y[:, t].double()).norm() <= (TOL + ROUND[dtype]) * y[:, t].double().norm()
    assert K == 1 or torch.equal(state, last)


def rates(seed, H, N):
    """Decay rates from a few steps to some thousands at the steps below."""
    return -torch.exp(normal(seed, H, N)) * torch.arange(1, N + 1, device="cuda")


def step_bias(H):
    d = torch.exp(torch.linspace(np.log(0.001), np.log(0.1), H, dtype=torch.float64)) if H > 1 \
        else torch.tensor([0.01], dtype=torch.float64)
    return torch.log(torch.expm1(d)).float().cuda()


SCAN_CASES = [
    # B, L, H, N, G, layout, carried state, resets, gate and skip
    (1, 1, 1, 1, 1, "apart", False, 0, True), (2, 1, 33, 16, 1, "apart", True, 1, True),
    (1, 2, 2, 3, 1, "columns", True, 0, False), (3, 7, 5, 4, 1, "columns", False, 2, True),
    (2, 15, 64, 16, 1, "apart", True, 0, True), (2, 16, 64, 16, 2, "columns", True, 3, True),
    (1, 17, 66, 5, 3, "time first", False, 0, True), (3, 129, 31, 7, 1, "broadcast", True, 2, True),
    (2, 200, 132, 16, 4, "columns", True, 64, True), (1, 1000, 96, 8, 1, "time first", True, 5, False),
    (2, 333, 258, 16, 1, "columns", False, 0, True), (5, 321, 17, 33, 1, "apart", True, 1, True),
    (1, 2500, 8, 64, 1, "apart", True, 3, True), (1, 9001, 3, 2, 1, "apart", False, 0, False),
    (2, 700, 520, 16, 1, "columns", True, 9, True), (2, 100, 72, 20, 3, "columns", True, 4, True),
    (1, 257, 129, 64, 1, "apart", False, 7, True), (40, 33, 256, 16, 8, "apart", True, 2, True),
    (1, 4000, 64, 1, 1, "columns", True, 30, True), (70, 50, 640, 16, 1, "columns", True, 1, True),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,L,H,N,G,layout,start,cuts,full", SCAN_CASES)
def test_scan_and_its_gradients(B, L, H, N, G, layout, start, cuts, full, dtype):
    seed = B + 10 * L + H + N
    x, dt, z = arrays(layout, 3, seed, B, L, H, dtype)
    dy = arrays("time first" if layout == "time first" else "apart", 1, seed + 50, B, L, H, dtype)[0]
    Bm, Cm = (t.unflatten(-1, (G, N)) for t in
              arrays("columns" if layout == "columns" else "apart", 2, seed + 30, B, L, G * N, dtype))
    if G == 1 and B == 1:  # without the dimension of groups
        Bm, Cm = Bm[:, :, 0], Cm[:, :, 0]
    A, bias = rates(seed + 5, H, N), step_bias(H)
    D = normal(seed + 6, H) if full else None
    z = z if full else None
    h0, dhl = (normal(seed + k, B, H, N) if start else None for k in (60, 61))
    reset = resets(seed, B, L, cuts) if cuts else None
    cut = None if reset is None else reset.cpu().numpy()
    how = dict(D=D, z=z, dt_bias=bias, h0=h0, reset=reset)
    f = [host(t) for t in (x, dt, A, Bm, Cm)]
    fo = [host(D), host(z), host(bias), True, host(h0), cut]
    y, last, states = ssm.ssm_scan(x, dt, A, Bm, Cm, save_states=True, **how)
    ry, before, rlast, _ = osm.scan(*f, *fo)
    close(y, ry)
    close(last, rlast)
    assert tuple(states.shape) == (B, -(-L // ssm.STATE_STEPS), H, N)
    if cut is None:  # at a marked step the kept state is the one that the step forgets
        close(states, before[:, ::ssm.STATE_STEPS])
    out = None
    if layout == "columns":
        nan = lambda n: torch.full((B, L, n), float("nan"), dtype=dtype, device="cuda")
        o1, o2 = nan(3 * H), nan(2 * G * N)
        m = [o2[..., :G * N].view_as(Bm) if G == 1 and B == 1 else o2[..., :G * N].unflatten(-1, (G, N)),
             o2[..., G * N:].view_as(Cm) if G == 1 and B == 1 else o2[..., G * N:].unflatten(-1, (G, N))]
        out = (o1[..., :H], o1[..., H:2 * H], *m, o1[..., 2 * H:] if full else None)
    g = ssm.ssm_scan_backward(x, dt, A, Bm, Cm, dy, states, dh_last=dhl, out=out, **how)
    ref = osm.scan_backward(*f, host(dy), *fo, host(dhl))
    for k, (a, r) in enumerate(zip(g, ref)):
        if a is None:
            continue
        r = r.reshape(a.shape)
        scale = None
        if k in (2, 7):  # sums of either sign over all steps
            scale = np.linalg.norm(r) + np.linalg.norm(ref[1])
        if k == 8:
            scale = np.linalg.norm(r) + (np.linalg.norm(host(dhl)) if dhl is not None else 0)
        close(a, r, scale)
    assert (g.dD is None) == (g.dz is None) == (not full)
    assert (g.dh0 is None) == (h0 is None)
    assert dlr.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,H,N,G,full", [(1, 1, 1, 1, True), (3, 33, 16, 1, False), (5, 64, 16, 2, True),
                                          (2, 130, 5, 1, True), (9, 24, 64, 3, True),
                                          (2, 40, 33, 1, True), (260, 136, 8, 1, True)])
def test_scan_steps(B, H, N, G, full, dtype):
    """Token by token, in place and beside, the sequence's results; marked entries begin anew."""
    L = 5
    x, dt, z = (normal(k, B, L, H, dtype=dtype) for k in (1, 2, 3))
    Bm, Cm = (normal(k, B, L, G, N, dtype=dtype) for k in (4, 5))
    A, bias, D = rates(6, H, N), step_bias(H), normal(7, H) if full else None
    h, reset = normal(8, B, H, N), resets(9, B, L, 1)
    f = [host(t) for t in (x, dt, A, Bm, Cm)]
    ry, _, rh, _ = osm.scan(*f, host(D), host(z) if full else None, host(bias), True, host(h),
                            reset.cpu().numpy())
    for t in range(L):
        how = dict(D=D, z=z[:, t] if full else None, dt_bias=bias, reset=reset[:, t].contiguous())
        a = (x[:, t], dt[:, t], A, *((m[:, t, 0] if G == 1 else m[:, t]) for m in (Bm, Cm)), h)
        if t % 2:
            o = ssm.ssm_step(*a, **how)
        else:
            nxt = torch.empty_like(h)
            o = ssm.ssm_step(*a, h_out=nxt, **how)
            h = nxt
        close(o, ry[:, t])
    close(h, rh)


@pytest.mark.parametrize("dtype", TYPES)
def test_without_softplus_and_bias(dtype):
    B, L, H, N = 2, 50, 40, 6
    x, dy = normal(1, B, L, H, dtype=dtype), normal(2, B, L, H, dtype=dtype)
    dt = (normal(3, B, L, H).abs() * 0.1).to(dtype)
    Bm, Cm = (normal(k, B, L, N, dtype=dtype) for k in (4, 5))
    A = rates(6, H, N)
    y, last, st = ssm.ssm_scan(x, dt, A, Bm, Cm, softplus=False, save_states=True)
    f = [host(t) for t in (x, dt, A, Bm, Cm)]
    ry, _, rl, _ = osm.scan(*f, sp=False)
    close(y, ry)
    close(last, rl)
    g = ssm.ssm_scan_backward(x, dt, A, Bm, Cm, dy, st, softplus=False)
    ref = osm.scan_backward(*f, host(dy), sp=False)
    for k in range(5):
        close(g[k], ref[k].reshape(g[k].shape))
    assert g.dD is None and g.dz is None and g.ddt_bias is None and g.dh0 is None
