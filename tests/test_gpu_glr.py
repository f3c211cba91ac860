"""The gated recurrent block's operators on the GPU against their float64 definitions
(oracle/glr.py): relative L2 <= 1e-5 for float32 outputs; an output stored in 16 bits adds its
rounding, at most 2^-8 (bfloat16, 8 significant bits) or 2^-11 (float16, 11) of each value."""
import numpy as np
import pytest
import torch

from oracle import glr as og
from state_space_sequence_gb300 import dlr, glr

pytestmark = pytest.mark.gpu

TOL = 1e-5
ROUND = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def host(t):
    torch.cuda.synchronize()
    return t.detach().double().cpu().numpy()


def close(got, ref, scale=None):
    """``scale``: the norm to compare with, where the reference's own may cancel."""
    assert tuple(got.shape) == np.shape(ref)
    g = host(got)
    assert np.isfinite(g).all()
    norm = np.linalg.norm(ref) if scale is None else scale
    err = np.linalg.norm(g - ref)
    assert err <= (TOL + ROUND[got.dtype]) * norm + 1e-30, (err / max(norm, 1e-300), got.dtype)


def normal(seed, *shape, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def decay_param(H):
    """p of decays whose memories run from a few steps to a few thousand."""
    a0 = np.linspace(0.7, 0.9998, H) if H > 1 else np.array([0.99])
    return torch.from_numpy(np.log(np.expm1(-np.log(a0))).astype(np.float32)).cuda()


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
    out[1] = normal(seed + 77, 1, 1, H, dtype=dtype).expand(B, L, H)
    return out


def resets(seed, B, L, count):
    m = torch.zeros(B, L, dtype=torch.bool)
    g = np.random.default_rng(seed)
    for b in range(B):
        m[b, g.integers(0, L, count)] = True
    return m.cuda()


SCAN_CASES = [
    # B, L, H, layout, h0, resets
    (1, 1, 1, "apart", False, 0), (2, 1, 33, "apart", True, 1), (1, 2, 2, "columns", True, 0),
    (3, 7, 5, "columns", False, 2), (2, 63, 64, "apart", True, 0), (2, 64, 64, "columns", True, 3),
    (1, 65, 66, "time first", False, 0), (3, 129, 31, "broadcast", True, 2),
    (2, 200, 130, "columns", True, 64), (1, 1000, 96, "time first", True, 5),
    (2, 1025, 258, "columns", False, 0), (5, 321, 17, "apart", True, 1),
    (1, 5000, 8, "apart", True, 3), (1, 70001, 3, "apart", False, 0),
    (4, 4000, 640, "columns", True, 9),  # more tiles to a block than it remembers places for
    # few chains with many tiles at work: runs of tiles, ended by resets and by the row's end
    (1, 40000, 32, "apart", True, 0), (1, 9000, 64, "columns", True, 40),
    (2, 21000, 20, "apart", False, 3),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,L,H,layout,start,cuts", SCAN_CASES)
def test_scan_and_its_gradients(B, L, H, layout, start, cuts, dtype):
    seed = B + 10 * L + H
    x, r, i = arrays(layout, 3, seed, B, L, H, dtype)
    dy = arrays("time first" if layout == "time first" else "apart", 1, seed + 50, B, L, H, dtype)[0]
    p = decay_param(H)
    h0, dhl = (normal(seed + k, B, H) if start else None for k in (60, 61))
    reset = resets(seed, B, L, cuts) if cuts else None
    y, last, states = glr.glr_scan(x, r, i, p, 4.0, h0, reset, save_states=True)
    cut = None if reset is None else reset.cpu().numpy()
    f = [host(t) for t in (x, r, i, p)]
    ry, before, rlast = og.scan(*f, 4.0, None if h0 is None else host(h0), cut)
    close(y, ry)
    close(last, rlast)
    assert tuple(states.shape) == (B, -(-L // glr.STATE_STEPS), H)
    if cut is None:  # at a marked step the kept state is the one that the step forgets
        close(states, before[:, ::glr.STATE_STEPS])
    out = None
    if layout == "columns":
        dz = torch.full((B, L, 3 * H), float("nan"), dtype=dtype, device="cuda")
        out = (dz[..., :H], dz[..., H:2 * H], dz[..., 2 * H:])
    got = glr.glr_scan_backward(x, r, i, p, dy, states, 4.0, h0, reset, dhl, out=out)
    ref = og.scan_backward(*f, 4.0, host(dy), None if h0 is None else host(h0), cut,
                           None if dhl is None else host(dhl))
    for g, q in zip(got[:4], ref[:4]):
        close(g, q)
    assert (got[4] is None) == (h0 is None)
    if h0 is not None:
        close(got[4], ref[4], scale=np.linalg.norm(ref[4]) + np.linalg.norm(host(dhl)))
    assert dlr.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H", [33, 65, 66, 128, 258])
def test_nothing_is_written_outside_the_rows(H, dtype):
    """y, dx, dr and di as the middle rows of larger buffers: what stands around them stays, for
    rows that end anywhere in a warp's steps, with one and with several tiles to a block."""
    B, room = 2, 128
    p = decay_param(H)
    for L in (1, 7, 8, 9, 112, 113, 250, 905, 1017, 1025, 1030, 1032, 2025):
        x, r, i, dy = arrays("apart", 4, L, B, L, H, dtype)
        bufs = [torch.full((B, L + 2 * room, H), 7.0, dtype=dtype, device="cuda") for _ in range(4)]
        y, dx, dr, di = (b[:, room:room + L] for b in bufs)
        _, _, st = glr.glr_scan(x, r, i, p, out=y, save_states=True)
        glr.glr_scan_backward(x, r, i, p, dy, st, out=(dx, dr, di))
        for b in bufs:
            assert (b[:, :room] == 7).all() and (b[:, room + L:] == 7).all(), L
            assert torch.isfinite(b).all()


def test_scan_of_no_steps():
    x = torch.empty(2, 0, 5, device="cuda")
    p, h0, dhl = decay_param(5), normal(1, 2, 5), normal(2, 2, 5)
    y, last = glr.glr_scan(x, x, x, p, h0=h0)
    assert y.shape == (2, 0, 5) and torch.equal(last, h0)
    assert not glr.glr_scan(x, x, x, p)[1].any()
    _, _, states = glr.glr_scan(x, x, x, p, h0=h0, save_states=True)
    dx, dr, di, dp, dh0 = glr.glr_scan_backward(x, x, x, p, x, states, h0=h0, dh_last=dhl)
    assert not dp.any() and torch.equal(dh0, dhl) and dx.shape == x.shape


@pytest.mark.parametrize("L,at", [(100, 50), (200, 64), (200, 190), (1000, 333), (64, 1)])
def test_nothing_passes_a_reset(L, at):
    """An infinity or a NaN before a marked step reaches nothing behind it, and gradients that are
    not finite behind it reach nothing before it."""
    B, H = 2, 66
    x, r, i, dy = arrays("apart", 4, L, B, L, H, torch.float32)
    p, h0 = decay_param(H), normal(9, B, H)
    reset = torch.zeros(B, L, dtype=torch.uint8, device="cuda")
    reset[:, at] = 1
    y, last, st = glr.glr_scan(x, r, i, p, h0=h0, reset=reset, save_states=True)
    alone, last1, _ = glr.glr_scan(x[:, at:], r[:, at:], i[:, at:], p, save_states=True)
    close(y[:, at:], host(alone))
    xb, hb = x.clone(), h0.clone()
    xb[:, at - 1] = float("nan")
    xb[:, 0, ::2] = float("inf")
    hb[0] = float("nan")
    yb, lastb, _ = glr.glr_scan(xb, r, i, p, h0=hb, reset=reset, save_states=True)
    assert torch.equal(yb[:, at:], y[:, at:]) and torch.equal(lastb, last)
    assert not torch.isfinite(yb[:, at - 1]).any()
    g = glr.glr_scan_backward(x, r, i, p, dy, st, h0=h0, reset=reset)
    dyb = dy.clone()
    dyb[:, at:] = float("nan")
    gb = glr.glr_scan_backward(x, r, i, p, dyb, st, h0=h0, reset=reset,
                               dh_last=torch.full_like(h0, float("inf")))
    for a, b in zip(g[:3], gb[:3]):
        assert torch.equal(a[:, :at], b[:, :at])
    assert torch.equal(g[4], gb[4])


def test_scan_extremes():
    """Gates at their ends: a closed recurrence gate keeps the state whole, a decay parameter from
    vanishing to immediate forgetting stays finite, and a NaN gate shows in its channel alone."""
    B, L, H = 1, 130, 6
    x, r, i, dy = arrays("apart", 4, 5, B, L, H, torch.float32)
    p, h0 = torch.tensor([-200.0, -30.0, 0.0, 3.0, 50.0, 1e4], device="cuda"), normal(3, B, H)
    r[..., 2] = -float("inf")
    r[..., 3] = float("inf")
    i[..., 1] = -float("inf")
    i[..., 4] = float("inf")
    y, last, st = glr.glr_scan(x, r, i, p, h0=h0, save_states=True)
    f = [host(t) for t in (x, r, i, p)]
    ry, _, rlast = og.scan(*f, 8.0, host(h0))
    close(y, ry)
    assert torch.equal(y[..., 2], h0[:, None, 2].expand(B, L))
    got = glr.glr_scan_backward(x, r, i, p, dy, st, h0=h0)
    ref = og.scan_backward(*f, 8.0, host(dy), host(h0))
    for g, q in zip(got, ref):
        for c in range(H):  # channel by channel: their sizes differ
            close(g[..., c], q[..., c], scale=np.linalg.norm(q[..., c]) + 1e-12)
    r[..., 70, 0] = float("nan")
    y2, _ = glr.glr_scan(x, r, i, p, h0=h0)
    assert torch.equal(y2[..., 1:], y[..., 1:]) and torch.equal(y2[:, :70], y[:, :70])
    assert torch.isnan(y2[:, 70:, 0]).all()


def test_offsets_past_32_bits():
    """Rows more than 2^31 elements into their buffer."""
    st, H = 2 ** 30 + 8, 40
    buf = torch.zeros(2 * st + 3 * H, dtype=torch.bfloat16, device="cuda")
    small = normal(4, 1, 3, 3 * H, dtype=torch.bfloat16)
    z = buf.as_strided((1, 3, 3 * H), (0, st, 1))
    z.copy_(small)
    p, dy = decay_param(H), normal(5, 1, 3, H, dtype=torch.bfloat16)

    def both(z, out):
        a = [z[..., k * H:(k + 1) * H] for k in range(3)]
        y, last, s = glr.glr_scan(*a, p, save_states=True)
        return [y, last, *glr.glr_scan_backward(*a, p, dy, s, out=out)[:4]]
    ref = both(small, None)
    obuf = torch.zeros_like(buf).as_strided((1, 3, 3 * H), (0, st, 1))
    got = both(z, tuple(obuf[..., k * H:(k + 1) * H] for k in range(3)))
    for a, b in zip(ref, got):
        assert torch.equal(a, b)
    rows = z[0, :, :H]
    w = torch.ones(H, device="cuda")
    al = torch.ones(1, device="cuda")
    a = glr.glr_join(rows, rows, rows, w, al, w)
    b = glr.glr_join(*[small[0, :, :H]] * 3, w, al, w)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_scan_in_pieces_is_the_scan():
    B, L, H = 2, 500, 96
    x, r, i = arrays("columns", 3, 6, B, L, H, torch.float32)
    p = decay_param(H)
    y, last = glr.glr_scan(x, r, i, p)
    h, ys = None, []
    for a, b in ((0, 1), (1, 130), (130, 131), (131, 500)):
        o, h = glr.glr_scan(x[:, a:b], r[:, a:b], i[:, a:b], p, h0=h)
        ys.append(o)
    close(torch.cat(ys, 1), host(y))
    close(h, host(last))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,H", [(1, 1), (1, 512), (7, 33), (64, 258)])
def test_step(B, H, dtype):
    x, r, i = (t[:, 0] for t in arrays("columns", 3, B + H, B, 1, H, dtype))
    p, h = decay_param(H), normal(1, B, H)
    reset = resets(2, 1, B, 1)[0]
    ry, before, rh = og.scan(*(host(t)[:, None] for t in (x, r, i)), host(p), 8.0, host(h),
                             reset.cpu().numpy()[:, None])
    out = torch.empty_like(h)
    y = glr.glr_step(x, r, i, p, h, reset=reset, h_out=out)
    close(y, ry[:, 0])
    close(out, rh)
    keep = h.clone()
    y2 = glr.glr_step(x, r, i, p, keep, reset=reset)  # in place
    assert torch.equal(keep, out) and torch.equal(y, y2)


def test_steps_are_the_scan():
    B, L, H = 3, 70, 64
    x, r, i = arrays("columns", 3, 8, B, L, H, torch.float32)
    p, h = decay_param(H), torch.zeros(3, 64, device="cuda")
    y, last = glr.glr_scan(x, r, i, p)
    ys = torch.stack([glr.glr_step(x[:, t], r[:, t], i[:, t], p, h) for t in range(L)], 1)
    close(ys, host(y))
    close(h, host(last))


def test_scan_gradient_against_differences():
    """The derivative of <y, dy> + <h_last, dh_last> along a direction, from float32 forward passes
    of step e = 1/32. Each pass is within 1e-6 of the exact result, so the quotient is off by at most
    1e-6 * |terms| / e = 3.2e-5 |terms| from rounding, with |terms| = |y| |dy|, and by e^2 / 6
    times a third derivative of the size of the terms: 2e-4 |terms|."""
    B, L, H, e = 2, 150, 40, 2.0 ** -5
    x, r, i, dy = arrays("apart", 4, 3, B, L, H, torch.float32)
    p, h0, dhl = decay_param(H), normal(7, B, H), normal(8, B, H)
    args = [x, r, i, p, h0]
    y, _, st = glr.glr_scan(x, r, i, p, h0=h0, save_states=True)
    dx, dr, di, dp, dh0 = glr.glr_scan_backward(x, r, i, p, dy, st, h0=h0, dh_last=dhl)
    terms = float(y.double().norm() * dy.double().norm())
    for k, g in enumerate((dx, dr, di, dp, dh0)):
        d = normal(20 + k, *g.shape) / 8

        def loss(sign):
            a = list(args)
            a[k] = a[k] + sign * e * d
            o, last = glr.glr_scan(*a[:4], h0=a[4])
            return float((o.double() * dy).sum() + (last.double() * dhl).sum())
        got = float((g.double() * d).sum())
        assert abs((loss(1) - loss(-1)) / (2 * e) - got) <= 2.4e-4 * terms


JOIN_CASES = [(1, 1), (3, 5), (5, 32), (2, 33), (4, 64), (33, 100), (7, 515), (3, 1000), (130, 256),
              (2, 2048), (1500, 136), (3, 4100), (2, 8200), (1, 16384)]


def join_args(M, H, dtype, seed=0, layout="apart"):
    if layout == "columns":
        z = normal(seed + M + H, M, 3 * H, dtype=dtype)
        x, h, g = z[:, :H], z[:, H:2 * H], z[:, 2 * H:]
    else:
        x, h, g = (normal(seed + M + H + k, M, H, dtype=dtype) for k in range(3))
    w, v = 1 + 0.3 * normal(seed + 5, H), 1 + 0.3 * normal(seed + 6, H)
    return x, h, g, w, torch.tensor([0.7], device="cuda"), v


def check_join_grads(got, ref, dy, dn, w, parts=None):
    for k, (a, q) in enumerate(zip(got, ref)):
        assert (a is None) == (q is None)
        if a is None:
            continue
        # a channel's sum over rows, and dalpha's over channels too, may cancel: they are held
        # to the size of their terms
        close(a, q, scale=None if k < 3 else parts[k])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("norm,act", [("rms", "silu"), ("layer", "sigmoid"), ("rms", "none"),
                                      ("layer", "silu")])
@pytest.mark.parametrize("M,H", JOIN_CASES)
def test_join_and_its_gradients(M, H, norm, act, dtype):
    x, h, g, w, al, v = join_args(M, H, dtype, layout="columns" if M % 2 else "apart")
    if act == "none":
        g = None
    if H == 1:
        # a norm's gradient of one channel is q (1 - zhat^2), which cancels but for eps (and one
        # channel less its mean is zero): only rounding would be compared away from z = 0
        x, h = x * 0, h * 0
    y, n = glr.glr_join(x, h, g, w, al, v, norm, act)
    f = [None if t is None else host(t) for t in (x, h, g, w, al, v)]
    f[4] = f[4][0]
    ry, rn = og.join(*f, norm, act)
    close(y, ry)
    close(n, rn)
    dy, dn = normal(11, M, H, dtype=dtype), normal(12, M, H, dtype=dtype)
    got = glr.glr_join_backward(dy, dn, x, h, g, w, al, v, norm, act)
    ref = og.join_backward(host(dy), host(dn), *f, norm, act)
    un = og.norm(f[1] * og.act(f[2], act)[0], norm, 1e-6)[0]
    yn = og.norm(ry, norm, 1e-6)[0]
    D = ref[0]
    parts = {3: 0.7 * np.linalg.norm(D * un), 4: np.linalg.norm(f[3] * D * un),
             5: np.linalg.norm(host(dn) * yn)}
    check_join_grads(got, ref, dy, dn, w, parts)
    assert dlr.device_status() == 0


@pytest.mark.parametrize("parts", ["no next", "no dy", "norm only"])
@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_join_without_some_parts(parts, norm):
    M, H = 9, 72
    x, h, g, w, al, v = join_args(M, H, torch.float32)
    dy, dn = normal(11, M, H), normal(12, M, H)
    if parts == "no next":
        v = dn = None
    if parts == "no dy":
        dy = None
    if parts == "norm only":
        h = g = w = al = dy = None
    y, n = glr.glr_join(x, h, g, w, al, v, norm)
    f = [None if t is None else host(t) for t in (x, h, g, w, al, v)]
    if f[4] is not None:
        f[4] = f[4][0]
    for a, q in zip((y, n), og.join(*f, norm)):
        assert (a is None) == (q is None)
        if a is not None:
            close(a, q)
    got = glr.glr_join_backward(dy, dn, x, h, g, w, al, v, norm)
    ref = og.join_backward(*(None if t is None else host(t) for t in (dy, dn)), *f, norm)
    big = {k: 40.0 for k in (3, 4, 5)}  # about the norm of the 648 terms of size 1 behind each sum
    check_join_grads(got, ref, dy, dn, w, big)


def test_join_in_place_and_no_rows():
    x, h, g, w, al, v = join_args(6, 96, torch.bfloat16)
    y, n = glr.glr_join(x, h, g, w, al, v)
    x2, h2 = x.clone(), h.clone()
    glr.glr_join(x2, h2, g, w, al, v, out=(x2, h2))
    assert torch.equal(x2, y) and torch.equal(h2, n)
    dy, dn = normal(1, 6, 96, dtype=torch.bfloat16), normal(2, 6, 96, dtype=torch.bfloat16)
    a = glr.glr_join_backward(dy, dn, x, h, g, w, al, v)
    d = dy.clone()
    b = glr.glr_join_backward(d, dn, x, h, g, w, al, v,
                              out=(d, torch.empty_like(h), torch.empty_like(g)))
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    e = x[:0]
    y, n = glr.glr_join(e, e, e, w, al, v)
    assert y.shape == (0, 96)
    _, _, _, dw, da, dv = glr.glr_join_backward(e, e, e, e, e, w, al, v)
    assert not dw.any() and not da.any() and not dv.any()


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_empty_rows_and_rows_that_are_not_finite(norm):
    """A row of zeros has finite results; a NaN or an infinity stays in its own row."""
    M, H = 8, 264
    x, h, g, w, al, v = join_args(M, H, torch.float32)
    x[2], h[2], g[3] = 0, 0, -float("inf")
    dy, dn = normal(1, M, H), normal(2, M, H)
    y, n = glr.glr_join(x, h, g, w, al, v, norm)
    got = glr.glr_join_backward(dy, dn, x, h, g, w, al, v, norm)
    for t in (y, n, *got[:2], got[2][:3]):
        assert torch.isfinite(t).all()
    assert not n[2].any()
    hb = h.clone()
    hb[5, 7] = float("nan")
    hb[6, 0] = float("inf")
    yb, nb = glr.glr_join(x, hb, g, w, al, v, norm)
    gb = glr.glr_join_backward(dy, dn, x, hb, g, w, al, v, norm)
    ok = torch.tensor([0, 1, 2, 3, 4, 7], device="cuda")
    for a, b in zip((y, n, *got[:3]), (yb, nb, *gb[:3])):
        assert torch.equal(a[ok].nan_to_num(9.0), b[ok].nan_to_num(9.0))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,H", [(1, 1), (3, 31), (5, 32), (2, 33), (7, 100), (9, 1000), (4, 96)])
def test_checkpoints_are_the_format(M, H, dtype):
    t = normal(M + H, M, H) * torch.exp(3 * normal(7, M, 1))
    t[0, 0] = 0.0
    if M > 4:
        t[1] = 0.0
        t[2, 3], t[2, 20], t[3, 5] = float("inf"), -float("inf"), float("nan")
        t[4] *= 1e-30
    t = t.to(dtype)
    wide = torch.zeros(M, H + 3, dtype=dtype, device="cuda")
    wide[:, :H] = t
    for src in (t, wide[:, :H]):
        c = glr.glr_ckpt_pack(src)
        codes, scales, values = og.ckpt_pack(host(src))
        assert np.array_equal(c.scales.cpu().numpy(), scales)
        assert np.array_equal(c.codes.cpu().numpy(), codes)
        got = host(glr.glr_ckpt_unpack(c))
        assert np.array_equal(got, values, equal_nan=True)
        if dtype is torch.bfloat16:
            assert np.array_equal(host(glr.glr_ckpt_unpack(c, torch.bfloat16)), values,
                                  equal_nan=True)


def test_checkpoint_scales_at_their_limits():
    """Values at the largest float32, next to 448 times a power of two, and far below 2^-127."""
    top = np.float32(448.0)
    t = np.zeros((1, 32 * 5), np.float32)
    t[0, 0] = np.finfo(np.float32).max
    t[0, 32] = top * 2
    t[0, 64] = np.nextafter(np.float32(top * 2), np.float32(np.inf))
    t[0, 96] = 1e-44
    t[0, 128] = -(2.0 ** -126)
    c = glr.glr_ckpt_pack(torch.from_numpy(t).cuda())
    codes, scales, values = og.ckpt_pack(t)
    assert np.array_equal(c.codes.cpu().numpy(), codes)
    assert np.array_equal(c.scales.cpu().numpy(), scales)
    with np.errstate(over="ignore"):  # the largest float32 rounds to 2^128 in e4m3: infinity
        assert np.array_equal(host(glr.glr_ckpt_unpack(c)), values.astype(np.float32))


@pytest.mark.parametrize("M,H,act", [(5, 64, "silu"), (4, 100, "sigmoid"), (3, 515, "silu"),
                                     (9, 96, "none"), (300, 1024, "silu")])
@pytest.mark.parametrize("dtype", TYPES)
def test_join_with_checkpoints(M, H, act, dtype):
    """The join keeps what glr_ckpt_pack makes of h and g, its results are those without, and its
    gradients are those at the values kept."""
    x, h, g, w, al, v = join_args(M, H, dtype)
    if act == "none":
        g = None
    y, n = glr.glr_join(x, h, g, w, al, v, act=act)
    y2, n2, kept = glr.glr_join(x, h, g, w, al, v, act=act, ckpt=True)
    assert torch.equal(y, y2) and torch.equal(n, n2)
    for t, c in zip((h, g), kept):
        assert (t is None) == (c is None)
        if t is not None:
            alone = glr.glr_ckpt_pack(t)
            assert torch.equal(alone.codes, c.codes) and torch.equal(alone.scales, c.scales)
    dy, dn = normal(1, M, H, dtype=dtype), normal(2, M, H, dtype=dtype)
    got = glr.glr_join_backward(dy, dn, x, None, None, w, al, v, act=act, ckpt=kept)
    hk, gk = (None if c is None else host(glr.glr_ckpt_unpack(c)) for c in kept)
    f = (host(x), hk, gk, host(w), float(al), host(v))
    ref = og.join_backward(host(dy), host(dn), *f, "rms", act)
    un = og.norm(hk * og.act(gk, act)[0], "rms", 1e-6)[0]
    yn = og.norm(og.join(*f, "rms", act)[0], "rms", 1e-6)[0]
    parts = {3: 0.7 * np.linalg.norm(ref[0] * un), 4: np.linalg.norm(f[3] * ref[0] * un),
             5: np.linalg.norm(host(dn) * yn)}
    check_join_grads(got, ref, dy, dn, w, parts)


def test_join_gradient_against_differences():
    """As for the scan: float32 passes of step 1/32 along a direction, within 2.4e-4 of the terms."""
    M, H, e = 6, 80, 2.0 ** -5
    args = list(join_args(M, H, torch.float32))
    dy, dn = normal(1, M, H), normal(2, M, H)
    y, n = glr.glr_join(*args)
    terms = float(y.double().norm() * dy.double().norm() + n.double().norm() * dn.double().norm())
    for k, g in enumerate(glr.glr_join_backward(dy, dn, *args)):
        d = normal(30 + k, *g.shape) / 8

        def loss(sign):
            a = list(args)
            a[k] = a[k] + sign * e * d
            o, q = glr.glr_join(*a)
            return float((o.double() * dy).sum() + (q.double() * dn).sum())
        got = float((g.double() * d).sum())
        assert abs((loss(1) - loss(-1)) / (2 * e) - got) <= 2.4e-4 * terms


def test_results_do_not_depend_on_the_run_or_the_workspace():
    for B, L, H in ((3, 3000, 192), (1, 30000, 64)):
        check_repeats(B, L, H)


def check_repeats(B, L, H):
    x, r, i, dy = arrays("apart", 4, 1, B, L, H, torch.bfloat16)
    p, reset = decay_param(H), resets(3, B, L, 4)
    need = max(glr.glr_scan_workspace_size(B, L, H), glr.glr_scan_backward_workspace_size(B, L, H),
               glr.glr_join_backward_workspace_size(B * L, H))
    rows = [t.view(B * L, H) for t in (x, r, i)]
    w, al = 1 + 0.1 * normal(2, H), torch.ones(1, device="cuda")
    ref = None
    for fill in (0, 255, 255, 7):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        y, last, st = glr.glr_scan(x, r, i, p, reset=reset, save_states=True, workspace=ws)
        back = glr.glr_scan_backward(x, r, i, p, dy, st, reset=reset, workspace=ws)
        join = glr.glr_join_backward(dy.view(B * L, H), rows[0], *rows, w, al, w, workspace=ws)
        got = [t.clone() for t in (y, last, st, *back[:4], *join)]
        if ref is None:
            ref = got
        for a, b in zip(ref, got):
            assert torch.isfinite(a).all() and torch.equal(a, b)


SLEEP_CYCLES = 20_000_000  # about 10 ms


def test_calls_run_on_the_stream_they_are_given():
    """Inputs written on a side stream behind a sleep; the calls' own memory belongs to it too."""
    B, L, H = 2, 700, 128
    src = arrays("apart", 4, 1, B, L, H, torch.bfloat16)
    p = decay_param(H)
    w, al = 1 + 0.1 * normal(2, H), torch.ones(1, device="cuda")
    s = torch.cuda.Stream()

    def calls(x, r, i, dy, stream):
        y, last, st = glr.glr_scan(x, r, i, p, save_states=True, stream=stream)
        out = [y, last, *glr.glr_scan_backward(x, r, i, p, dy, st, stream=stream)[:4]]
        out.append(glr.glr_step(x[:, 0], r[:, 0], i[:, 0], p, last.clone() if stream is None
                                else torch.zeros_like(last), stream=stream))
        a = [t.view(B * L, H) for t in (x, r, i)]
        y, n, kept = glr.glr_join(*a, w, al, w, ckpt=True, stream=stream)
        out += [y, n, *glr.glr_join_backward(dy.view(B * L, H), y, a[0], None, None, w, al, w,
                                             ckpt=kept, stream=stream)]
        out.append(glr.glr_ckpt_unpack(glr.glr_ckpt_pack(a[0], stream=stream), stream=stream))
        return out
    ref = calls(*src, None)
    ref[6] = glr.glr_step(*(t[:, 0] for t in src[:3]), p, torch.zeros(B, H, device="cuda"))
    torch.cuda.synchronize()
    late = [torch.zeros_like(t) for t in src]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(SLEEP_CYCLES)
        for o, t in zip(late, src):
            o.copy_(t)
    got = calls(*late, s)
    assert not s.query()
    s.synchronize()
    for a, b in zip(ref, got):
        assert torch.equal(a, b)


def test_refusals():
    """What a call cannot do it refuses before it launches anything."""
    B, L, H = 2, 10, 16
    x, r, i = arrays("apart", 3, 1, B, L, H, torch.bfloat16)
    p = decay_param(H)
    with pytest.raises(TypeError):
        glr.glr_scan(x.cpu(), r, i, p)
    with pytest.raises(TypeError):
        glr.glr_scan(x, r.float(), i, p)
    with pytest.raises(TypeError):
        glr.glr_scan(x.double(), r.double(), i.double(), p)
    with pytest.raises(ValueError):
        glr.glr_scan(x, r[:, :5], i, p)
    with pytest.raises(ValueError):
        glr.glr_scan(x.transpose(1, 2), r.transpose(1, 2), i.transpose(1, 2), decay_param(L))
    with pytest.raises(ValueError):
        glr.glr_scan(x, r, i, p[:3].contiguous())
    with pytest.raises(TypeError):
        glr.glr_scan(x, r, i, p.bfloat16())
    with pytest.raises(TypeError):
        glr.glr_scan(x, r, i, p, reset=torch.zeros(B, L, device="cuda"))
    with pytest.raises(dlr.DLRError):
        glr.glr_scan(x, r, i, p, scale=-1.0)
    with pytest.raises(dlr.DLRError):
        glr.glr_scan(x, r, i, p, out=x)                           # y over x
    with pytest.raises(dlr.DLRError):
        glr.glr_scan(x, r, i, p, out=torch.empty(1, L, H, dtype=x.dtype,
                                                 device="cuda").expand(B, L, H))
    with pytest.raises(dlr.DLRError):
        glr.glr_scan(*(t.repeat(1, 20, 1) for t in (x, r, i)), p,
                     workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    w, al = torch.ones(H, device="cuda"), torch.ones(1, device="cuda")
    a = [t.reshape(B * L, H) for t in (x, r, i)]
    with pytest.raises(KeyError):
        glr.glr_join(*a, w, al, w, norm="batch")
    with pytest.raises(ValueError):
        glr.glr_join(*a, w, al, w, act="none")
    with pytest.raises(dlr.DLRError):
        glr.glr_join(*a, w, al, w, eps=0.0)
    with pytest.raises(dlr.DLRError):
        glr.glr_join(*a, w, None, w)
    with pytest.raises(dlr.DLRError):
        glr.glr_join(*a, w, al, w, out=(a[1], torch.empty_like(a[0])))   # y over h
    with pytest.raises(dlr.DLRError):
        glr.glr_join(torch.ones(1, 16385, device="cuda"), None, None, None, None,
                     torch.ones(16385, device="cuda"))
    with pytest.raises(dlr.DLRError):
        glr.glr_join_backward(a[0], None, *a, w, al, w)           # dn missing
    with pytest.raises(ValueError):
        glr.glr_ckpt_unpack(glr.Ckpt8(torch.zeros(2, 40, dtype=torch.uint8, device="cuda"),
                                      torch.zeros(2, 1, dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()
    assert dlr.device_status() == 0
