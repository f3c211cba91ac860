"""The float64 definitions of the selective state space block (oracle/ssm.py) and of its loss
(oracle/xent.py) against what fixes them: central differences for every gradient, packed sequences
against the same sequences alone, and known special cases. CPU only."""
import numpy as np
import pytest

from oracle import dlr_layer, glr as og, ssm as osm, xent as ox


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


def agree(f, leaves, grads):
    """Central differences of step 1e-6 carry a rounding error of about 1e-16 * |loss| / 1e-6 and a
    truncation error of order 1e-12: 1e-7 of the largest entry bounds both."""
    for a, g in zip(leaves, grads):
        if a.size == 0:  # a convolution of one tap has no state
            continue
        d = differences(f, a)
        assert np.abs(d - g.reshape(d.shape)).max() <= 1e-7 * max(1.0, np.abs(d).max())


@pytest.mark.parametrize("groups", [1, 2])
@pytest.mark.parametrize("sp", [True, False])
def test_scan_gradients_match_differences(groups, sp):
    B, L, H, N = 2, 5, 4, 3
    x, dt, z, dy, A, D, bias, h0, dhl = rnd(1, *[(B, L, H)] * 4, (H, N), (H,), (H,), *[(B, H, N)] * 2)
    Bm, Cm = rnd(2, *[(B, L, groups, N)] * 2)
    A = -np.exp(A)
    reset = np.zeros((B, L), bool)
    reset[0, 2] = reset[1, 0] = reset[1, 4] = True

    def loss():
        y, _, last, _ = osm.scan(x, dt, A, Bm, Cm, D, z, bias, sp, h0, reset)
        return (y * dy).sum() + (last * dhl).sum()
    agree(loss, (x, dt, A, Bm, Cm, D, z, bias, h0),
          osm.scan_backward(x, dt, A, Bm, Cm, dy, D, z, bias, sp, h0, reset, dhl))


@pytest.mark.parametrize("K,act", [(1, "silu"), (2, "none"), (4, "silu")])
def test_convolution_gradients_match_differences(K, act):
    B, L, H = 2, 6, 3
    x, dy, w, bias, state, dl = rnd(3, *[(B, L, H)] * 2, (H, K), (H,), *[(B, K - 1, H)] * 2)
    reset = np.zeros((B, L), bool)
    reset[0, 3] = reset[1, 1] = True

    def loss():
        y, last, _ = osm.conv(x, w, bias, state, reset, act)
        return (y * dy).sum() + (last * dl).sum()
    agree(loss, (x, w, bias, state), osm.conv_backward(x, w, dy, bias, state, reset, act, dl))


def test_loss_gradients_match_differences():
    h, W, w = rnd(4, (5, 3), (7, 3), (5,))
    target = np.array([0, 6, -1, 3, 7])

    def loss():
        return (ox.loss(h, W, target)[0] * w).sum()
    agree(loss, (h, W), ox.loss_backward(h, W, target, w))


def test_packed_rows_are_their_sequences_alone():
    H, N, K = 3, 2, 4
    x, dt, z, A, w = rnd(5, *[(1, 9, H)] * 3, (H, N), (H, K))
    Bm, Cm, h0, s0 = rnd(6, (1, 9, N), (1, 9, N), (1, H, N), (1, K - 1, H))
    reset = np.zeros((1, 9), bool)
    reset[0, [0, 4, 5]] = True
    y = osm.scan(x, dt, -np.exp(A), Bm, Cm, None, z, None, True, h0, reset)[0]
    u = osm.conv(x, w, None, s0, reset)[0]
    for a, b in ((0, 4), (4, 5), (5, 9)):
        s = slice(a, b)
        alone = osm.scan(x[:, s], dt[:, s], -np.exp(A), Bm[:, s], Cm[:, s], None, z[:, s])[0]
        assert np.array_equal(alone, y[:, s])
        assert np.array_equal(osm.conv(x[:, s], w)[0], u[:, s])


def test_constant_maps_are_a_bank_of_recurrences():
    """A step, input map and output map that do not change are a DLR bank with real decays: lambda =
    exp(s A), weights C s B."""
    B, L, H, N = 2, 40, 3, 5
    (x, A), (b, c) = rnd(7, (B, L, H), (H, N)), rnd(8, (N,), (N,))
    A, s = -np.exp(A), 0.1
    one = np.ones((B, L, 1))
    y = osm.scan(x, np.full((B, L, H), s), A, one * b, one * c, sp=False)[0]
    log_re = np.sqrt(-s * A)
    W = np.stack([np.broadcast_to(c * s * b, (H, N)), np.zeros((H, N))], -1)
    ref = dlr_layer(x.transpose(0, 2, 1), (log_re, np.zeros((H, N)), W)).transpose(0, 2, 1)
    assert np.abs(y - ref).max() <= 1e-5 * np.abs(ref).max()


def test_a_convolution_is_numpys():
    x, w = rnd(9, (1, 30, 2), (2, 4))
    y = osm.conv(x, w, act="none")[0]
    for c in range(2):
        assert np.allclose(y[0, :, c], np.convolve(x[0, :, c], w[c, ::-1])[:30], atol=1e-13)
    assert np.allclose(osm.silu(np.array([0.0, 800.0, -800.0])), [0.0, 800.0, 0.0])
    assert og.sigmoid(np.array(0.0)) == 0.5


def test_uniform_logits_lose_the_logarithm_of_the_vocabulary():
    loss, lse, _ = ox.loss(np.zeros((2, 3)), np.ones((10, 3)), np.array([4, -1]))
    assert np.allclose(lse, np.log(10)) and np.allclose(loss, [np.log(10), 0])
