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


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [4097, 45000, 50257])
def test_targets_in_every_place_of_a_tile(V, dtype):
    """Few rows over many columns, where tiles are narrower: targets on both sides of every border of
    16 columns of a stretch, and at the ends."""
    D = 24
    edge = torch.arange(0, 2048, 16)
    target = torch.cat([edge, edge + 15, torch.tensor([V - 1, V - 2, V - 17])])[:250]
    h, W, _, _ = problem(len(target), V, D, dtype, seed=3)
    dloss = torch.rand(len(target), device="cuda")
    check(h, W, target.cuda(), dloss)
    check(h[:16], W, target[-16:].cuda(), dloss[:16].contiguous())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("layout", ["apart", "columns", "odd columns", "every other row"])
def test_layouts(layout, dtype):
    M, V, D = 200, 700, 136
    h, W, target, dloss = problem(M, V, D, dtype, seed=1)
    dloss = dloss * (64.0 if dtype == torch.float16 else 1)

    def lay(t):
        n, d = t.shape
        if layout == "columns":
            big = torch.zeros(n, 2 * d, dtype=dtype, device="cuda")
            big[:, d:] = t
            return big[:, d:]
        if layout == "odd columns":
            big = torch.zeros(n, d + 3, dtype=dtype, device="cuda")
            big[:, 1:d + 1] = t
            return big[:, 1:d + 1]
        if layout == "every other row":
            big = torch.zeros(2 * n, d, dtype=dtype, device="cuda")
            big[::2] = t
            return big[::2]
        return t
    a = xent.xent_loss(h, W, target)
    b = xent.xent_loss(lay(h), lay(W), target)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ref = xent.xent_loss_backward(h, W, target, a[1], dloss)
    rooms = [torch.full((n + 2, D + 8), 7.0, dtype=dtype, device="cuda") for n in (M, V)]
    out = [r[1:-1, 5:-3] for r in rooms]
    got = xent.xent_loss_backward(lay(h), lay(W), target, b[1], dloss, out=out)
    for x, y in zip(ref, got):
        assert torch.equal(x, y)
    for r in rooms:
        r[1:-1, 5:-3] = 7.0
        assert (r == 7.0).all()
    # one row for all tokens, and one for the whole vocabulary
    same = h[:1].expand(M, D)
    x, y = xent.xent_loss(same, W, target), xent.xent_loss(same.contiguous(), W, target)
    assert torch.equal(x[0], y[0])


@pytest.mark.parametrize("dtype", TYPES)
def test_only_what_is_wanted(dtype):
    h, W, target, dloss = problem(70, 300, 64, dtype)
    _, lse = xent.xent_loss(h, W, target)
    both = xent.xent_loss_backward(h, W, target, lse, dloss)
    dh, none = xent.xent_loss_backward(h, W, target, lse, dloss, wanted=(True, False))
    assert none is None and torch.equal(dh, both[0])
    none, dW = xent.xent_loss_backward(h, W, target, lse, dloss, wanted=(False, True))
    assert none is None and torch.equal(dW, both[1])
    assert xent.xent_loss_backward(h, W, target, lse, dloss, wanted=(False, False)) == (None, None)


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_without_a_target_may_hold_anything(dtype):
    """NaN and infinities in them reach neither the losses, nor dW, nor other rows."""
    M, V, D = 150, 400, 72
    h, W, target, dloss = problem(M, V, D, dtype)
    gone = torch.arange(M) % 3 == 1
    target[gone] = -100
    bad, worse = h.clone(), dloss.clone()
    bad[gone] = float("nan")
    bad[1] = float("inf")
    worse[gone] = float("nan")
    a = xent.xent_loss(h, W, target)
    b = xent.xent_loss(bad, W, target)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1][~gone], b[1][~gone])
    x = xent.xent_loss_backward(h, W, target, a[1], dloss)
    y = xent.xent_loss_backward(bad, W, target, b[1], worse)
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    none = torch.full_like(target, -1)
    loss, lse = xent.xent_loss(h, W, none)
    dh, dW = xent.xent_loss_backward(h, W, none, lse, dloss)
    assert not loss.any() and not dh.any() and not dW.any()


@pytest.mark.parametrize("dtype", TYPES)
def test_large_logits(dtype):
    """Logits of some hundreds: the largest is taken off, losses are its distance to the target's. A
    logit of size Z is a float32 number, off by 2^-24 Z, its product's sum by as much again for each of
    its D / 16 + 1 additions that lose anything (five here), so exp(z - lse) is off by 12 * 2^-24 Z of
    itself at most, lse's share included."""
    M, V, D = 60, 500, 64
    h, W, target, dloss = problem(M, V, D, dtype)
    h = (h * 100).to(dtype)
    dloss = dloss * (64.0 if dtype == torch.float16 else 1)
    f = [host(h), host(W), target.cpu().numpy()]
    loss, lse = xent.xent_loss(h, W, target)
    rl, rs, z = ox.loss(*f)
    assert np.linalg.norm(host(lse) - rs) <= TOL * np.linalg.norm(rs)
    assert np.linalg.norm(host(loss) - rl) <= TOL * (np.linalg.norm(rl) + np.linalg.norm(rs))
    slack = 12 * 2.0 ** -24 * np.abs(z).max() + 2 * ROUND[dtype]
    d = np.exp(z - rs[:, None])
    d[np.arange(M), f[2]] -= 1.0
    d = np.abs(d) * host(dloss)[:, None]
    for g, r, size in zip(xent.xent_loss_backward(h, W, target, lse, dloss),
                          ox.loss_backward(*f, host(dloss)), (d @ np.abs(f[1]), d.T @ np.abs(f[0]))):
        least = 2.0 ** -25 * np.sqrt(r.size) if dtype == torch.float16 else 0.0
        assert np.linalg.norm(host(g) - r) <= slack * np.linalg.norm(size) + least


def test_float16_gradients_of_tiny_weights():
    """dloss far below float16's range for d: the largest is brought to 2^13 or more, so that what d
    loses is relative to it. The result itself is in float16: a loss scale brings it into range."""
    M, V, D = 40, 300, 64
    h, W, target, dloss = problem(M, V, D, torch.float16)
    _, lse = xent.xent_loss(h, W, target)
    ref = ox.loss_backward(host(h), host(W), target.cpu().numpy(), host(dloss))
    for k in (2.0 ** 10, 2.0 ** 13, 1.0):
        dh, dW = xent.xent_loss_backward(h, W, target, lse, dloss * k)
        for g, r in ((dh, ref[0]), (dW, ref[1])):
            r = r * k
            least = 2.0 ** -25 * np.sqrt(r.size)  # half of float16's smallest step
            assert np.linalg.norm(host(g) - r) <= 3 * 2.0 ** -11 * np.linalg.norm(r) + least


@pytest.mark.parametrize("dtype", TYPES)
def test_several_pieces_of_the_vocabulary(dtype):
    """More rows than one piece's d holds for all columns: dh is summed over the pieces."""
    M, V, D = (70000, 2500, 24) if dtype != torch.float32 else (40000, 2500, 24)
    h, W, target, dloss = problem(M, V, D, dtype, sure=3.0)
    target[::7] = -1
    dloss = dloss * (2.0 ** 15 if dtype == torch.float16 else 1)
    loss, lse = xent.xent_loss(h, W, target)
    dh, dW = xent.xent_loss_backward(h, W, target, lse, dloss)
    z = h.double() @ W.double().t()
    ok = target >= 0
    ref = torch.logsumexp(z, 1)
    assert (lse[ok].double() - ref[ok]).norm() <= TOL * ref[ok].norm()
    d = torch.exp(z - ref[:, None])
    d[ok, target[ok]] -= 1.0
    d *= torch.where(ok, dloss.double(), 0.0)[:, None]
    near(dh, (d @ W.double()).cpu().numpy(), (d.abs() @ W.double().abs()).cpu().numpy())
    near(dW, (d.t() @ h.double()).cpu().numpy(), (d.abs().t() @ h.double().abs()).cpu().numpy())


def test_float32_sums_over_a_long_vocabulary():
    """The tensor core's additions cut off; a second accumulator keeps that from adding up."""
    M, V, D = 130, 60000, 40
    h, W, target, dloss = problem(M, V, D, torch.float32)
    loss, lse, dh, dW = check(h, W, target, dloss)
    rh, rW = ox.loss_backward(host(h), host(W), target.cpu().numpy(), host(dloss))
    assert np.linalg.norm(host(dh) - rh) <= TOL * np.linalg.norm(rh)
    assert np.linalg.norm(host(dW) - rW) <= TOL * np.linalg.norm(rW)


def test_no_rows():
    h, W, target, dloss = problem(3, 100, 40, torch.bfloat16)
    e, t, f = h[:0], target[:0], dloss[:0]
    loss, lse = xent.xent_loss(e, W, t)
    assert loss.shape == lse.shape == (0,)
    dh, dW = xent.xent_loss_backward(e, W, t, lse, f)
    assert dh.shape == (0, 40) and not dW.any()
    room = torch.full((100, 50), 7.0, dtype=torch.bfloat16, device="cuda")
    xent.xent_loss_backward(e, W, t, lse, f, out=(None, room[:, :40]))
    assert not room[:, :40].any() and (room[:, 40:] == 7).all()


def test_gradient_against_differences():
    """float32 passes of step 1/16 along a direction: rounding 1e-6 of the losses' sum times 16, and a
    truncation of (1/16)^2 / 6 of a third derivative along directions that move logits by about 1/8:
    2e-4 of the losses' sum bounds both."""
    M, V, D, e = 20, 90, 32, 2.0 ** -4
    h, W, target, _ = problem(M, V, D, torch.float32)
    w = torch.rand(M, device="cuda")
    loss, lse = xent.xent_loss(h, W, target)
    terms = float((lse.double() * w).abs().sum())
    for k, g in enumerate(xent.xent_loss_backward(h, W, target, lse, w)):
        gen = torch.Generator().manual_seed(k)
        d = torch.randn(*g.shape, generator=gen).cuda() / (8 if k == 0 else 8 * D ** 0.5)

        def total(s):
            a = [h, W]
            a[k] = a[k] + s * e * d
            return float((xent.xent_loss(*a, target)[0].double() * w).sum())
        diff = (total(1) - total(-1)) / (2 * e)
        assert abs(diff - float((g.double() * d).sum())) <= 2e-4 * terms


def passes(h, W, target, dloss, stream=None, ws=None):
    loss, lse = xent.xent_loss(h, W, target, workspace=ws, stream=stream)
    return [loss, lse, *xent.xent_loss_backward(h, W, target, lse, dloss, workspace=ws,
                                                stream=stream)]


@pytest.mark.parametrize("M,V,D", [(300, 3000, 200), (70000, 2500, 24), (5, 4000, 515)])
def test_results_do_not_depend_on_the_run_or_the_workspace(M, V, D):
    for dtype in TYPES[:2]:
        if dtype == torch.float32 and M > 1000:
            continue
        p = problem(M, V, D, dtype)
        need = max(xent.xent_loss_workspace_size(dtype, M, V, D),
                   xent.xent_loss_backward_workspace_size(dtype, M, V, D))
        ref = None
        for fill in (0, 255, 255, 7):
            ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
            got = passes(*p, ws=ws)
            ref = ref or got
            for a, b in zip(ref, got):
                assert torch.isfinite(a).all() and torch.equal(a, b)


def test_streams_graphs_and_two_calls_at_once():
    M, V, D = 200, 2000, 128
    sets = [problem(M, V, D, torch.bfloat16, seed=s) for s in (1, 2)]
    ref = [passes(*p) for p in sets]
    s = torch.cuda.Stream()
    late = [torch.zeros_like(t) for t in sets[0]]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        for o, t in zip(late, sets[0]):
            o.copy_(t)
    got = passes(*late, stream=s)
    assert not s.query()
    s.synchronize()
    for a, b in zip(ref[0], got):
        assert torch.equal(a, b)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        both = [passes(*p, stream=q) for p, q in zip(sets, streams)]
        torch.cuda.synchronize()
        for p, q in zip(ref, both):
            for a, b in zip(p, q):
                assert torch.equal(a, b)
    need = max(xent.xent_loss_workspace_size(torch.bfloat16, M, V, D),
               xent.xent_loss_backward_workspace_size(torch.bfloat16, M, V, D))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    held = [t.clone() for t in sets[0]]
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append(passes(*held, ws=ws))
    for p, r in zip(sets[::-1], ref[::-1]):
        for a, b in zip(held, p):
            a.copy_(b)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o in outs:
            for a, b in zip(o, r):
                assert torch.equal(a, b)


def test_refusals(monkeypatch):
    M, V, D = 10, 50, 16
    h, W, target, dloss = problem(M, V, D, torch.bfloat16)
    _, lse = xent.xent_loss(h, W, target)
    for exc, a in ((TypeError, (h.cpu(), W, target)), (TypeError, (h, W.float(), target)),
                   (TypeError, (h.double(), W.double(), target)), (ValueError, (h, W[:, :8], target)),
                   (ValueError, (h[0], W, target)), (TypeError, (h, W, target.int())),
                   (ValueError, (h, W, target[:3])), (TypeError, (h, W, target.cpu())),
                   (ValueError, (h.t().contiguous().t(), W, target))):
        with pytest.raises(exc):
            xent.xent_loss(*a)
    with pytest.raises(ValueError):
        xent.xent_loss_backward(h, W, target, lse[:3], dloss)
    with pytest.raises(TypeError):
        xent.xent_loss_backward(h, W, target, lse, dloss.half())
    with pytest.raises(dlr.DLRError):
        xent.xent_loss_backward(h, W, target, lse, dloss, out=(h, None))       # over an input
    with pytest.raises(dlr.DLRError):
        xent.xent_loss(h, W, target, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        xent.xent_loss_workspace_size(torch.int32, M, V, D)
    from state_space_sequence_gb300 import glr
    monkeypatch.setattr(glr, "_current_device", lambda: h.get_device() + 1)
    with pytest.raises(ValueError):
        xent.xent_loss(h, W, target)
    with pytest.raises(ValueError):
        xent.xent_loss_backward(h, W, target, lse, dloss)
    torch.cuda.synchronize()
    assert dlr.device_status() == 0
