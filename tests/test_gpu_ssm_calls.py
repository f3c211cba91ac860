"""The selective state space block's calls as programs make them: what stands around their results, rows
with marks and values that are not finite, long memories, offsets past 32 bits, pieces of a sequence,
streams, captured graphs, workspaces, repeated and simultaneous calls, differences, and refusals."""
import numpy as np
import pytest
import torch

from oracle import ssm as osm
from state_space_sequence_gb300 import dlr, glr, ssm

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def host(t):
    torch.cuda.synchronize()
    return t.detach().double().cpu().numpy()


def normal(seed, *shape, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def rates(seed, H, N):
    return -torch.exp(normal(seed, H, N)) * torch.arange(1, N + 1, device="cuda")


def scan_args(B, L, H, N, dtype, seed=1, G=None):
    """Positional and keyword arguments of a scan with everything that it may have but marks."""
    x, dt, z = (normal(seed + k, B, L, H, dtype=dtype) for k in range(3))
    shape = (B, L, N) if G is None else (B, L, G, N)
    Bm, Cm = (normal(seed + k, *shape, dtype=dtype) for k in (3, 4))
    how = dict(D=normal(seed + 5, H), z=z, dt_bias=normal(seed + 6, H) - 3.0,
               h0=normal(seed + 7, B, H, N))
    return [x, dt, rates(seed + 8, H, N), Bm, Cm], how


def scan_oracle(args, how, reset=None):
    return osm.scan(*map(host, args), host(how["D"]), host(how["z"]), host(how["dt_bias"]), True,
                    host(how["h0"]), reset)


def frame(B, L, H, dtype):
    """A buffer of 7s and its middle rows and channels [B, L, H] as a view."""
    room = torch.full((B, L + 2, H + 6), 7.0, dtype=dtype, device="cuda")
    return room, room[:, 1:-1, 3:-3]


def untouched(room):
    inner = room.clone()
    inner[:, 1:-1, 3:-3] = 7.0
    return bool((inner == 7.0).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L,H,N,G", [(1, 1, 1, 1), (17, 33, 5, 3), (40, 66, 16, 2), (31, 128, 64, 1)])
def test_nothing_is_written_outside_the_rows(L, H, N, G, dtype):
    B = 2
    args, how = scan_args(B, L, H, N, dtype, G=G)
    rooms = [frame(B, L, H, dtype) for _ in range(4)]
    maps = [torch.full((B, L + 2, G * N + 6), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    inner = [m[:, 1:-1, 3:-3].unflatten(-1, (G, N)) for m in maps]
    y, last, st = ssm.ssm_scan(*args, save_states=True, out=rooms[0][1], **how)
    plain = ssm.ssm_scan(*args, **how)
    assert torch.equal(plain[0], y) and torch.equal(plain[1], last)
    dy = normal(50, B, L, H, dtype=dtype)
    g = ssm.ssm_scan_backward(*args, dy, st, dh_last=last,
                              out=(rooms[1][1], rooms[2][1], *inner, rooms[3][1]), **how)
    ref = ssm.ssm_scan_backward(*args, dy, st, dh_last=last, **how)
    for a, b in zip(g, ref):
        assert torch.equal(a, b)
    for room, _ in rooms:
        assert untouched(room)
    for m in maps:
        assert untouched(m)
    rooms = [frame(B, L, H, dtype) for _ in range(2)]
    w = normal(9, H, 4)
    a = ssm.ssm_conv(args[0], w, out=rooms[0][1])
    b = ssm.ssm_conv_backward(args[0], w, dy, out=rooms[1][1])
    assert torch.equal(a[0], ssm.ssm_conv(args[0], w)[0])
    assert torch.equal(b[0], ssm.ssm_conv_backward(args[0], w, dy)[0])
    assert untouched(rooms[0][0]) and untouched(rooms[1][0])


def test_no_steps():
    B, H, N, K = 3, 20, 4, 4
    x = torch.empty(B, 0, H, device="cuda")
    m = torch.empty(B, 0, N, device="cuda")
    A, h0 = rates(1, H, N), normal(2, B, H, N)
    y, last, st = ssm.ssm_scan(x, x, A, m, m, h0=h0, save_states=True)
    assert y.shape == (B, 0, H) and torch.equal(last, h0) and st.shape == (B, 0, H, N)
    assert not ssm.ssm_scan(x, x, A, m, m)[1].any()
    g = ssm.ssm_scan_backward(x, x, A, m, m, x, st, D=normal(3, H), dt_bias=normal(4, H), h0=h0,
                              dh_last=2 * h0)
    assert torch.equal(g.dh0, 2 * h0) and not g.dA.any() and not g.dD.any() and not g.ddt_bias.any()
    assert not ssm.ssm_scan_backward(x, x, A, m, m, x, st, h0=h0).dh0.any()
    w, state = normal(5, H, K), normal(6, B, K - 1, H)
    y, last = ssm.ssm_conv(x, w, state=state)
    assert y.shape == (B, 0, H) and torch.equal(last, state)
    dx, dw, db, ds = ssm.ssm_conv_backward(x, w, x, bias=normal(7, H), state=state, dlast=3 * state)
    assert torch.equal(ds, 3 * state) and not dw.any() and not db.any()


@pytest.mark.parametrize("L,at", [(40, 0), (40, 15), (40, 16), (700, 333), (700, 699), (33, 32)])
def test_nothing_passes_a_mark(L, at):
    """Before the mark everything is infinite or NaN; from it on results and gradients are those of the
    sequence that begins there, and the gradients before it know nothing of what follows."""
    B, H, N = 2, 40, 6
    args, how = scan_args(B, L, H, N, torch.float32)
    bad = [t.clone() for t in args]
    for k, v in ((0, float("nan")), (1, float("inf")), (3, -float("inf")), (4, float("nan"))):
        bad[k][:, :at] = v
    h0 = torch.full_like(how["h0"], float("nan"))
    z = how["z"].clone()
    reset = torch.zeros(B, L, dtype=torch.bool, device="cuda")
    reset[:, at] = True
    tail = [t[:, at:] if t.dim() > 2 else t for t in args]
    dy, dhl = normal(20, B, L, H), normal(21, B, H, N)
    how_t = dict(D=how["D"], z=z[:, at:], dt_bias=how["dt_bias"])
    y, last, st = ssm.ssm_scan(*bad, reset=reset, save_states=True, **{**how, "h0": h0})
    ty, tl, ts = ssm.ssm_scan(*tail, save_states=True, **how_t)
    ok = lambda a, b: (a.double() - b.double()).norm() <= 1e-5 * b.double().norm() + 1e-30
    assert ok(y[:, at:], ty) and ok(last, tl)
    g = ssm.ssm_scan_backward(*bad, dy, st, reset=reset, dh_last=dhl, **{**how, "h0": h0})
    t = ssm.ssm_scan_backward(*tail, dy[:, at:], ts, dh_last=dhl, **how_t)
    for a, b in ((g.dx, t.dx), (g.ddt, t.ddt), (g.dB, t.dB), (g.dC, t.dC), (g.dz, t.dz)):
        assert ok(a[:, at:], b)
    if at:
        late = dy.clone()
        late[:, at:] = float("nan")
        clean = ssm.ssm_scan(*args, reset=reset, save_states=True, **how)[2]
        g = ssm.ssm_scan_backward(*args, late, clean, reset=reset, dh_last=dhl, **how)
        head = [v[:, :at] if v.dim() > 2 else v for v in args]
        how_h = {**how, "z": z[:, :at]}
        hs = ssm.ssm_scan(*head, save_states=True, **how_h)[2]
        t = ssm.ssm_scan_backward(*head, dy[:, :at], hs, **how_h)
        for a, b in ((g.dx, t.dx), (g.ddt, t.ddt), (g.dB, t.dB), (g.dC, t.dC)):
            assert ok(a[:, :at], b)
        assert ok(g.dh0, t.dh0)


@pytest.mark.parametrize("K", [2, 3, 4, 5, 8])
@pytest.mark.parametrize("at", [0, 1, 6, 7, 8, 63, 64, 99])
def test_nothing_passes_a_mark_of_the_convolution(K, at):
    B, L, H = 2, 100, 40
    x, dy, w = normal(1, B, L, H), normal(2, B, L, H), normal(3, H, K)
    bad = x.clone()
    bad[:, :at] = float("nan")
    state = torch.full((B, K - 1, H), float("inf"), device="cuda")
    reset = torch.zeros(B, L, dtype=torch.bool, device="cuda")
    reset[:, at] = True
    y, last = ssm.ssm_conv(bad, w, state=state, reset=reset)
    ty, tl = ssm.ssm_conv(x[:, at:], w)
    assert torch.equal(y[:, at:], ty) and torch.equal(last, tl)
    dx, _, _, ds = ssm.ssm_conv_backward(bad, w, dy, state=state, reset=reset)
    tx = ssm.ssm_conv_backward(x[:, at:], w, dy[:, at:])[0]
    assert torch.equal(dx[:, at:], tx)
    if at == 0:
        assert not ds.any()
    # inputs further back than the taps reach may be anything
    far = x.clone()
    far[:, :at] = float("inf")
    y, last = ssm.ssm_conv(far, w)
    assert torch.isfinite(y[:, at + K - 1:]).all()
    # and what follows a mark gives nothing to what stands before it
    late = dy.clone()
    late[:, at:] = float("nan")
    dx, _, _, ds = ssm.ssm_conv_backward(x, w, late, state=torch.zeros_like(state), reset=reset)
    assert torch.isfinite(dx[:, :at]).all() and torch.isfinite(ds).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_steps_of_minus_infinity_leave_the_state(dtype):
    """Padding by dt = -inf: s = 0, such steps leave the state bit for bit (the steps before them may be
    added up in another order in a longer call) and nothing is learnt of them."""
    B, L, H, N = 2, 50, 24, 16
    args, how = scan_args(B, L, H, N, dtype)
    args[1][:, 20:] = -float("inf")
    y, last, st = ssm.ssm_scan(*args, save_states=True, **how)
    part = lambda a, b: [t[:, a:b] if t.dim() > 2 else t for t in args]
    cut = ssm.ssm_scan(*part(0, 20), **{**how, "z": how["z"][:, :20]})
    rest = ssm.ssm_scan(*part(20, L), **{**how, "z": how["z"][:, 20:], "h0": cut[1]})
    assert torch.equal(rest[1], cut[1])
    assert (last - cut[1]).double().norm() <= 1e-5 * last.double().norm()
    g = ssm.ssm_scan_backward(*args, normal(20, B, L, H, dtype=dtype), st, **how)
    assert not g.ddt[:, 20:].any() and not g.dB[:, 20:].any()
    for t in g:
        assert torch.isfinite(t).all()
    h = last.clone()
    ssm.ssm_step(*(t[:, 30] if t.dim() > 2 else t for t in args), h, D=how["D"], z=how["z"][:, 30],
                 dt_bias=how["dt_bias"])
    assert torch.equal(h, last)


@pytest.mark.parametrize("dtype", TYPES)
def test_long_memories(dtype):
    """A constant step of 2^-13 (a memory of 8192 steps) and a constant input: the sum of a geometric
    series. In 16 bits the decay is one rounded number, off by at most 2^-24 + 2^-25 of itself (the
    unit's error next to 1 as measured, 1.5 units in the last place below 1), which over the memory
    makes 8192 * 1.5 * 2^-24 = 7.4e-4 of the state. float32 keeps 1 - a, so 1e-5."""
    B, L, H, N = 1, 20000, 2, 1
    one = torch.ones(B, L, H, dtype=dtype, device="cuda")
    dt = torch.full((B, L, H), 2.0 ** -13, dtype=dtype, device="cuda")
    m = torch.ones(B, L, N, dtype=dtype, device="cuda")
    A = -torch.ones(H, N, device="cuda")
    _, last = ssm.ssm_scan(one, dt, A, m, m, softplus=False)
    s = 2.0 ** -13
    ref = s * -np.expm1(-s * L) / -np.expm1(-s)
    bound = 1e-5 if dtype is torch.float32 else 7.4e-4
    assert abs(float(last[0, 0, 0]) / ref - 1) <= bound


def test_extremes_of_the_gate_and_the_step():
    """Steps from far below float32's smallest to large ones, gates of +-80, rates of zero: finite and
    as defined."""
    B, L, H, N = 1, 64, 16, 4
    args, how = scan_args(B, L, H, N, torch.float32)
    args[1][:, :, :8] = torch.linspace(-120, 60, 64, device="cuda")[None, :, None]
    how["z"][:, ::2] = 80.0
    how["z"][:, 1::2] = -80.0
    args[2][::2] = 0.0
    y, last, st = ssm.ssm_scan(*args, save_states=True, **how)
    ry, _, rl, _ = scan_oracle(args, how)
    for a, r in ((y, ry), (last, rl)):
        assert np.isfinite(host(a)).all()
        assert np.linalg.norm(host(a) - r) <= 1e-5 * np.linalg.norm(r)
    for t in ssm.ssm_scan_backward(*args, normal(20, B, L, H), st, **how):
        assert torch.isfinite(t).all()


def test_offsets_past_32_bits():
    """Rows whose elements lie 2^32 and more apart (the batch in one buffer of 9 GB)."""
    B, L, H, N = 2, 35, 64, 16
    far = (1 << 32) + 4 * H
    buf = torch.zeros(far + L * 4 * H, dtype=torch.bfloat16, device="cuda")
    view = lambda k: buf.as_strided((B, L, H), (far, 4 * H, 1), k * H)
    args, how = scan_args(B, L, H, N, torch.bfloat16)
    x, dt, z = view(0), view(1), view(2)
    for a, b in zip((x, dt, z), (args[0], args[1], how["z"])):
        a.copy_(b)
    y, last, st = ssm.ssm_scan(*args, save_states=True, **how)
    out = view(3)
    y2, last2, st2 = ssm.ssm_scan(x, dt, *args[2:], save_states=True, out=out, **{**how, "z": z})
    assert torch.equal(y, y2) and torch.equal(last, last2) and torch.equal(st, st2)
    dy = normal(20, B, L, H, dtype=torch.bfloat16)
    ref = ssm.ssm_scan_backward(*args, dy, st, **how)
    maps = [torch.empty_like(args[3]) for _ in range(2)]
    rest = [torch.empty_like(args[0]) for _ in range(2)]
    got = ssm.ssm_scan_backward(x, dt, *args[2:], dy, st, out=(out, rest[0], *maps, rest[1]),
                                **{**how, "z": z})
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
    w = normal(9, H, 4)
    assert torch.equal(ssm.ssm_conv(x, w, out=out)[0], ssm.ssm_conv(args[0], w)[0])
    assert torch.equal(ssm.ssm_conv_backward(x, w, dy, out=out)[0],
                       ssm.ssm_conv_backward(args[0], w, dy)[0])


def test_many_channels_and_batches_past_32_bits_of_states():
    """States of more than 2^31 elements, in a step: 2^17 entries of 1040 channels of 16 states."""
    B, H, N = 1 << 17, 1040, 16
    h = torch.zeros(B, H, N, device="cuda")
    h[-1] = 1.0
    x = torch.ones(B, H, dtype=torch.bfloat16, device="cuda")
    m = torch.ones(1, N, dtype=torch.bfloat16, device="cuda").expand(B, N)
    A = -torch.ones(H, N, device="cuda")
    y = ssm.ssm_step(x, x, A, m, m, h)
    s = np.log1p(np.e)
    for b, before in ((0, 0.0), (B // 2, 0.0), (B - 1, 1.0)):
        ref = np.exp(-s) * before + s
        assert abs(h[b].double().cpu().numpy() - ref).max() <= 1e-5 * ref
        assert abs(y[b].double().cpu().numpy() - N * ref).max() <= (2.0 ** -8 + 1e-5) * N * ref


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H", [40, 1024])
def test_a_sequence_in_pieces_is_the_sequence(H, dtype):
    """Forwards from the states that the pieces leave, backwards from the gradients that they send."""
    B, L, N, K, cuts = 2, 300, 16, 4, (0, 1, 2, 50, 147, 300)
    args, how = scan_args(B, L, H, N, dtype)
    w, bias = normal(30, H, K), normal(31, H)
    dy, dhl = normal(32, B, L, H, dtype=dtype), normal(33, B, H, N)
    u, end = ssm.ssm_conv(args[0], w, bias, state=normal(34, B, K - 1, H, dtype=dtype))
    state = normal(34, B, K - 1, H, dtype=dtype)
    h, ys, us, kept = how["h0"], [], [], []
    for a, b in zip(cuts, cuts[1:]):
        kept.append(state)
        o, state = ssm.ssm_conv(args[0][:, a:b], w, bias, state=state)
        us.append(o)
    assert torch.equal(torch.cat(us, 1), u) and torch.equal(state, end)
    g, dl, dxs, dw = dy, normal(35, B, K - 1, H, dtype=dtype), [], 0
    whole = ssm.ssm_conv_backward(args[0], w, dy, bias, state=kept[0], dlast=dl)
    f32 = dtype is torch.float32
    if f32:  # in 16 bits what the pieces send on is rounded on the way
        for (a, b), s in reversed(list(zip(zip(cuts, cuts[1:]), kept))):
            dx, dwp, _, dl = ssm.ssm_conv_backward(args[0][:, a:b], w, dy[:, a:b], bias, state=s,
                                                   dlast=dl)
            dxs.insert(0, dx)
            dw = dw + dwp
        for p, q in ((torch.cat(dxs, 1), whole[0]), (dw, whole[1]), (dl, whole[3])):
            assert (p.double() - q.double()).norm() <= 1e-5 * q.double().norm()
    y, last, st = ssm.ssm_scan(*args, save_states=True, **how)
    ref = ssm.ssm_scan_backward(*args, dy, st, dh_last=dhl, **how)
    states = []
    for a, b in zip(cuts, cuts[1:]):
        part = [t[:, a:b] if t.dim() > 2 else t for t in args]
        hw = {**how, "z": how["z"][:, a:b], "h0": h}
        o, h2, s = ssm.ssm_scan(*part, save_states=True, **hw)
        states.append((part, hw, s))
        ys.append(o)
        h = h2
    tol = 1e-5 + HALF[dtype]
    assert (torch.cat(ys, 1).double() - y.double()).norm() <= tol * y.double().norm()
    assert (h.double() - last.double()).norm() <= 1e-5 * last.double().norm()
    dh, dxs, dA = dhl, [], 0
    for (a, b), (part, hw, s) in reversed(list(zip(zip(cuts, cuts[1:]), states))):
        g = ssm.ssm_scan_backward(*part, dy[:, a:b], s, dh_last=dh, **hw)
        dxs.insert(0, g.dx)
        dA, dh = dA + g.dA, g.dh0
    assert (torch.cat(dxs, 1).double() - ref.dx.double()).norm() <= tol * ref.dx.double().norm()
    assert (dA - ref.dA).double().norm() <= 1e-5 * (ref.dA.double().norm() + ref.ddt.double().norm())
    assert (dh - ref.dh0).double().norm() <= 1e-5 * ref.dh0.double().norm()


def run_all(args, how, w, dy, stream=None, ws=None):
    x = args[0]
    B, L, H = x.shape
    hw = {**how, "h0": None}
    u, last = ssm.ssm_conv(x, w, stream=stream)
    out = [u, last, *ssm.ssm_conv_backward(x, w, dy, workspace=ws, stream=stream)[:2]]
    y, h, st = ssm.ssm_scan(*args, save_states=True, workspace=ws, stream=stream, **hw)
    out += [y, h, st]
    out += [t for t in ssm.ssm_scan_backward(*args, dy, st, workspace=ws, stream=stream, **hw)
            if t is not None]
    return out


def test_results_do_not_depend_on_the_run_or_the_workspace():
    for B, L, H, N in ((3, 1000, 192, 16), (1, 5000, 64, 5)):
        args, how = scan_args(B, L, H, N, torch.bfloat16)
        w, dy = normal(9, H, 4), normal(10, B, L, H, dtype=torch.bfloat16)
        need = max(ssm.ssm_scan_workspace_size(B, L, H, N),
                   ssm.ssm_scan_backward_workspace_size(B, L, H, N),
                   ssm.ssm_conv_backward_workspace_size(B, L, H, 4))
        ref = None
        for fill in (0, 255, 255, 7):
            ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
            got = run_all(args, how, w, dy, ws=ws)
            ref = ref or got
            for a, b in zip(ref, got):
                assert torch.isfinite(a).all() and torch.equal(a, b)


SLEEP_CYCLES = 20_000_000  # about 10 ms


def test_calls_run_on_the_stream_they_are_given():
    """Inputs written on a side stream behind a sleep; the calls' own memory belongs to it too."""
    B, L, H, N = 2, 700, 128, 16
    args, how = scan_args(B, L, H, N, torch.bfloat16)
    w, dy = normal(9, H, 4), normal(10, B, L, H, dtype=torch.bfloat16)
    s = torch.cuda.Stream()
    h = torch.zeros(B, H, N, device="cuda")
    row = lambda a: [t[:, 0] if t.dim() > 2 else t for t in a]
    ref = run_all(args, how, w, dy)
    ref.append(ssm.ssm_step(*row(args), h.clone()))
    ref.append(ssm.ssm_conv_step(args[0][:, 0], w, args[0][:, 1:4].contiguous()))
    late = [torch.zeros_like(t) for t in args]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(SLEEP_CYCLES)
        for o, t in zip(late, args):
            o.copy_(t)
        first = late[0][:, 1:4].contiguous()
    got = run_all(late, how, w, dy, stream=s)
    got.append(ssm.ssm_step(*row(late), h, stream=s))
    got.append(ssm.ssm_conv_step(late[0][:, 0], w, first, stream=s))
    assert not s.query()
    s.synchronize()
    for a, b in zip(ref, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("H", [64, 2048])
def test_captured_and_replayed(H):
    """A training pass in a graph, replayed on new inputs; two graphs that share one workspace, one
    after the other; steps that advance a state in place."""
    B, L, N = 1, 400, 16
    args, how = scan_args(B, L, H, N, torch.bfloat16)
    w, dy = normal(9, H, 4), normal(10, B, L, H, dtype=torch.bfloat16)
    need = max(ssm.ssm_scan_workspace_size(B, L, H, N),
               ssm.ssm_scan_backward_workspace_size(B, L, H, N),
               ssm.ssm_conv_backward_workspace_size(B, L, H, 4))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    h, taps = torch.zeros(B, H, N, device="cuda"), torch.zeros(B, 3, H, dtype=w.dtype, device="cuda")
    taps = taps.to(torch.bfloat16)
    run_all(args, how, w, dy, ws=ws)
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g in graphs:
        with torch.cuda.graph(g):
            o = run_all(args, how, w, dy, ws=ws)
            u = ssm.ssm_conv_step(args[0][:, 0], w, taps)
            o.append(ssm.ssm_step(u, *(t[:, 0] if t.dim() > 2 else t for t in args[1:]), h))
            outs.append(o)
    for seed in (101, 202):
        new, _ = scan_args(B, L, H, N, torch.bfloat16, seed=seed)
        for a, b in zip(args, new):
            a.copy_(b)
        before, tb = h.clone(), taps.clone()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        ref = run_all(args, how, w, dy)
        for o in outs:
            for a, b in zip(o, ref):
                assert torch.equal(a, b)
        for o in outs:
            u = ssm.ssm_conv_step(args[0][:, 0], w, tb)
            y = ssm.ssm_step(u, *(t[:, 0] if t.dim() > 2 else t for t in args[1:]), before)
            assert torch.equal(y, o[-1])
        assert torch.equal(before, h) and torch.equal(tb, taps)


def test_two_calls_at_once():
    """The same calls on two streams at the same time, each with its own results and workspaces."""
    B, L, H, N = 2, 600, 256, 16
    sets = [scan_args(B, L, H, N, torch.bfloat16, seed=s) for s in (1, 60)]
    w, dy = normal(9, H, 4), normal(10, B, L, H, dtype=torch.bfloat16)
    ref = [run_all(a, k, w, dy) for a, k in sets]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [run_all(a, k, w, dy, stream=s) for (a, k), s in zip(sets, streams)]
        torch.cuda.synchronize()
        for p, q in zip(ref, got):
            for a, b in zip(p, q):
                assert torch.equal(a, b)


def test_gradients_against_differences():
    """float32 passes of step 1/64 along a direction: the rounding of a pass is about 1e-6 of the terms,
    times 64; the truncation is that of the third derivative along directions of length 1/8 or less in
    a gated product, below (1/64)^2 * 1/8 * 8: together 2.5e-4 of the terms bounds both."""
    B, L, H, N, e = 2, 24, 8, 4, 2.0 ** -6
    args, how = scan_args(B, L, H, N, torch.float32)
    dy, dhl = normal(20, B, L, H), normal(21, B, H, N)
    names = ["D", "z", "dt_bias", "h0"]
    leaves = args + [how[n] for n in names]

    def run(v):
        return ssm.ssm_scan(*v[:5], **dict(zip(names, v[5:])))
    y, last = run(leaves)
    st = ssm.ssm_scan(*args, save_states=True, **how)[2]
    terms = float(y.double().norm() * dy.double().norm() + last.double().norm() * dhl.double().norm())
    g = ssm.ssm_scan_backward(*args, dy, st, dh_last=dhl, **how)
    grads = [g.dx, g.ddt, g.dA, g.dB, g.dC, g.dD, g.dz, g.ddt_bias, g.dh0]
    for k, gk in enumerate(grads):
        d = normal(40 + k, *gk.shape) / 8

        def loss(sign):
            v = list(leaves)
            v[k] = v[k] + sign * e * d
            o, h = run(v)
            return float((o.double() * dy).sum() + (h.double() * dhl).sum())
        diff = (loss(1) - loss(-1)) / (2 * e)
        assert abs(diff - float((gk.double() * d).sum())) <= 2.5e-4 * terms, k
    x, w, b, s = args[0], normal(22, H, 4) / 2, normal(23, H), normal(24, B, 3, H)
    dl = normal(25, B, 3, H)
    leaves = [x, w, b, s]
    run = lambda v: ssm.ssm_conv(v[0], v[1], v[2], state=v[3])
    y, last = run(leaves)
    terms = float(y.double().norm() * dy.double().norm() + last.double().norm() * dl.double().norm())
    for k, gk in enumerate(ssm.ssm_conv_backward(x, w, dy, b, state=s, dlast=dl)):
        d = normal(50 + k, *gk.shape) / 8

        def loss(sign):
            v = list(leaves)
            v[k] = v[k] + sign * e * d
            o, h = run(v)
            return float((o.double() * dy).sum() + (h.double() * dl).sum())
        diff = (loss(1) - loss(-1)) / (2 * e)
        assert abs(diff - float((gk.double() * d).sum())) <= 2.5e-4 * terms, k


def test_refusals():
    """What a call cannot do it refuses before it launches anything."""
    B, L, H, N = 2, 10, 16, 4
    args, how = scan_args(B, L, H, N, torch.bfloat16)
    x, dt, A, Bm, Cm = args

    def scan(exc, match=None, **change):
        a = dict(x=x, dt=dt, A=A, B=Bm, C=Cm, **how)
        a.update(change)
        with pytest.raises(exc, match=match):
            ssm.ssm_scan(**a)
    scan(TypeError, x=x.cpu())
    scan(TypeError, dt=dt.float())
    scan(ValueError, dt=dt[:, :5])
    scan(ValueError, z=how["z"].transpose(1, 2).contiguous().transpose(1, 2))
    scan(ValueError, B=Bm[:, :, :3])
    scan(ValueError, B=Bm[:, :5])
    scan(ValueError, B=Bm[:, :, None].expand(B, L, 3, N), C=Cm[:, :, None].expand(B, L, 3, N))
    scan(ValueError, B=Bm.transpose(1, 2).contiguous().transpose(1, 2))
    scan(TypeError, C=Cm.float())
    scan(TypeError, A=A.bfloat16())
    scan(ValueError, A=A[:, :3].contiguous())
    scan(TypeError, A=A.t().contiguous().t())
    scan(ValueError, D=A[:3, 0].contiguous())
    scan(ValueError, h0=how["h0"][:1])
    scan(TypeError, reset=torch.zeros(B, L, device="cuda"))
    scan(dlr.DLRError, out=x)                                   # y over an input
    scan(dlr.DLRError, out=torch.empty(1, L, H, dtype=x.dtype, device="cuda").expand(B, L, H))
    wide = torch.zeros(B, L, 65, dtype=x.dtype, device="cuda")
    scan(dlr.DLRError, B=wide, C=wide, A=torch.zeros(H, 65, device="cuda"),
         h0=torch.zeros(B, H, 65, device="cuda"))               # too many states
    y, last, st = ssm.ssm_scan(*args, save_states=True, **how)
    with pytest.raises(ValueError):
        ssm.ssm_scan_backward(*args, y, st[:, :0], **how)
    with pytest.raises(ValueError):
        ssm.ssm_scan_backward(*args, y, st, out=(*(torch.empty_like(x) for _ in range(2)),
                                                 torch.empty_like(Bm), torch.empty_like(Cm), None),
                              **how)
    with pytest.raises(dlr.DLRError):
        ssm.ssm_scan_backward(*args, y, st, workspace=torch.empty(16, dtype=torch.uint8,
                                                                  device="cuda"), **how)
    with pytest.raises(ValueError):
        ssm.ssm_step(x[:, 0], dt[:, 0], A, Bm[:, 0], Cm[:, 0, :3], last)
    w, rows = normal(1, H, 4), torch.zeros(B, 3, H, dtype=x.dtype, device="cuda")
    with pytest.raises(dlr.DLRError):
        ssm.ssm_conv(x, normal(1, H, 9))
    with pytest.raises(ValueError):
        ssm.ssm_conv(x, w, state=rows[:, :2].contiguous())
    with pytest.raises(TypeError):
        ssm.ssm_conv(x, w, state=rows.float())
    with pytest.raises(KeyError):
        ssm.ssm_conv(x, w, act="gelu")
    with pytest.raises(dlr.DLRError):
        ssm.ssm_conv(x, w, out=x)
    with pytest.raises(dlr.DLRError):
        ssm.ssm_conv_step(x[:, 0], w, None)
    with pytest.raises(dlr.DLRError):
        ssm.ssm_conv_step(x[:, 0], w[:, :1].contiguous(), rows[:, :0].contiguous(),
                          state_out=rows[:, :0].contiguous(), out=x[:, 0])
    torch.cuda.synchronize()
    assert dlr.device_status() == 0


def test_every_call_refuses_another_device(monkeypatch):
    """And writes nothing: the states that a step would have replaced are as they were."""
    B, L, H, N = 2, 4, 16, 4
    args, how = scan_args(B, L, H, N, torch.float32)
    x, w = args[0], normal(1, H, 4)
    st = ssm.ssm_scan(*args, save_states=True, **how)[2]
    h, rows = torch.ones(B, H, N, device="cuda"), torch.ones(B, 3, H, device="cuda")
    one = [t[:, 0] if t.dim() > 2 else t for t in args]
    side = torch.cuda.Stream()
    calls = [lambda s: ssm.ssm_conv(x, w, stream=s),
             lambda s: ssm.ssm_conv_backward(x, w, x, stream=s),
             lambda s: ssm.ssm_conv_step(x[:, 0], w, rows, stream=s),
             lambda s: ssm.ssm_scan(*args, stream=s, **how),
             lambda s: ssm.ssm_scan_backward(*args, x, st, stream=s, **how),
             lambda s: ssm.ssm_step(*one, h, stream=s)]
    monkeypatch.setattr(glr, "_current_device", lambda: x.get_device() + 1)
    for call in calls:
        for s in (None, side):
            with pytest.raises(ValueError):
                call(s)
    torch.cuda.synchronize()
    assert (h == 1).all() and (rows == 1).all()
