"""The float64 definitions of the gated recurrent block (oracle/glr.py) against what fixes them:
central differences for every gradient, packed sequences against the same sequences alone, and
the extremes of the 8-bit format. CPU only."""
import numpy as np
import pytest

from oracle import glr as og


def rnd(seed, *shapes):
    g = np.random.default_rng(seed)
    return [g.standard_normal(s) for s in shapes]


def differences(f, a, step=1e-6):
    """d f / d a by central differences, f a scalar."""
    out = np.empty_like(a)
    for k in np.ndindex(*a.shape):
        keep = a[k]
        a[k] = keep + step
        up = f()
        a[k] = keep - step
        out[k] = (up - f()) / (2 * step)
        a[k] = keep
    return out


@pytest.mark.parametrize("start,mask", [(False, False), (True, False), (True, True)])
def test_scan_gradients_match_differences(start, mask):
    """Central differences of step 1e-6 carry a rounding error of about 1e-16 * |loss| / 1e-6 and a
    truncation error of order 1e-12: 1e-7 of the largest entry bounds both."""
    B, L, H, c = 2, 5, 3, 3.0
    x, r, i, dy, h0, dhl, p = rnd(1, *[(B, L, H)] * 4, (B, H), (B, H), (H,))
    h0 = h0 if start else None
    reset = np.zeros((B, L), bool)
    if mask:
        reset[0, 2] = reset[1, 0] = reset[1, 4] = True

    def loss():
        y, _, last = og.scan(x, r, i, p, c, h0, reset)
        return (y * dy).sum() + (last * dhl).sum()
    got = og.scan_backward(x, r, i, p, c, dy, h0, reset, dhl)
    for a, g in zip((x, r, i, p) + ((h0,) if start else ()), got):
        d = differences(loss, a)
        assert np.abs(d - g).max() <= 1e-7 * max(1.0, np.abs(d).max())


def test_packed_rows_are_their_sequences_alone():
    H, c = 3, 8.0
    x, r, i, p, h0 = rnd(2, (1, 9, H), (1, 9, H), (1, 9, H), (H,), (1, H))
    reset = np.zeros((1, 9), bool)
    reset[0, [0, 4, 5]] = True
    y, _, _ = og.scan(x, r, i, p, c, h0, reset)
    for a, b in ((0, 4), (4, 5), (5, 9)):
        alone, _, _ = og.scan(x[:, a:b], r[:, a:b], i[:, a:b], p, c)
        assert np.array_equal(alone, y[:, a:b])


def test_a_closed_gate_keeps_the_state():
    """sigmoid(-inf) = 0: a = 1 and b = 0."""
    h0 = np.array([[1.5, -2.0]])
    x = np.ones((1, 4, 2))
    y, _, last = og.scan(x, np.full((1, 4, 2), -np.inf), x, np.zeros(2), 8.0, h0)
    assert np.array_equal(last, h0) and np.array_equal(y, np.broadcast_to(h0[:, None], y.shape))


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("gate", ["silu", "sigmoid", "none"])
@pytest.mark.parametrize("parts", ["both", "y", "n", "norm only"])
def test_join_gradients_match_differences(kind, gate, parts):
    M, H = 3, 5
    x, h, g, dy, dn, w, v, al = rnd(3, *[(M, H)] * 5, (H,), (H,), (1,))
    if gate == "none":
        g = None
    if parts == "y":
        v = dn = None
    if parts == "n":
        dy = None
    if parts == "norm only":
        h = g = w = dy = None

    def loss():
        y, n = og.join(x, h, g, w, al[0], v, kind, gate)
        return (0.0 if dy is None else (y * dy).sum()) + (0.0 if v is None else (n * dn).sum())
    got = og.join_backward(dy, dn, x, h, g, w, al[0], v, kind, gate)
    for a, q in zip((x, h, g, w, al if h is not None else None, v), got):
        assert (a is None) == (q is None)
        if a is not None:
            d = differences(loss, a)
            assert np.abs(d - q).max() <= 1e-7 * max(1.0, np.abs(d).max())


def test_checkpoint_format():
    assert E4M3_is_right()
    codes, scales, values = og.ckpt_pack(np.array([[448.0, 1.0, -0.0, 449.0 * 0]]))
    assert scales[0, 0] == 127 and codes[0, 0] == 126 and values[0, 0] == 448.0
    # the least scale that holds the largest value without saturating
    _, scales, values = og.ckpt_pack(np.array([[449.0]]))
    assert scales[0, 0] == 128 and values[0, 0] == 448.0  # 224.5 rounds to 224
    # an empty group, and values that are not finite
    codes, scales, values = og.ckpt_pack(np.array([[np.inf, 2.0, np.nan]]))
    assert np.isnan(values[0, [0, 2]]).all() and values[0, 1] == 2.0
    assert og.ckpt_pack(np.zeros((1, 40)))[1].tolist() == [[0, 0]]


def E4M3_is_right():
    return len(og.E4M3) == 127 and og.E4M3[0] == 0 and og.E4M3[1] == 2.0 ** -9 and \
        og.E4M3[-1] == 448.0 and (np.diff(og.E4M3) > 0).all()
