"""The sums over rows of the join's gradients (include/glr.h) where their terms cancel."""
import numpy as np
import pytest
import torch

from state_space_sequence_gb300 import glr

pytestmark = pytest.mark.gpu


def rows(M, H, stride):
    """Rows of H channels, `stride` elements apart."""
    return torch.zeros(M, stride, device="cuda")[:, :H]


@pytest.mark.parametrize("stride", [1024, 1027])  # with and without 16-byte accesses
@pytest.mark.parametrize("M", [64, 4096])  # at most a row, and several, to a block
def test_dalpha_keeps_what_cancels(M, stride):
    """dalpha = sum w D uhat of rows whose every product is exact in float32: |h| = 1 makes the root
    mean square 1 (an eps of 1e-12 is lost beside it), w = 1 and D = dy. Each term is 2^16 or, in
    every other row, -2^16, with a multiple of 1/8 of at most 1 added: a thread's share of a row (16
    channels, below 2^21) is exact in float32, the row's sum of some 2^26 is not, and all rows'
    sum is that of the small parts, some hundreds. What is left is one rounding of the result."""
    H = 1024
    g = np.random.default_rng(M + stride)
    sign = g.choice([-1.0, 1.0], (M, H))
    small = g.integers(-8, 9, (M, H)) / 8.0
    big = np.where(np.arange(M) % 2 == 0, 65536.0, -65536.0)[:, None]
    x, h, dy = (rows(M, H, stride) for _ in range(3))
    h.copy_(torch.from_numpy(sign))
    dy.copy_(torch.from_numpy(sign * (big + small)))
    assert np.array_equal(dy.double().cpu().numpy(), sign * (big + small))
    one, w = torch.ones(1, device="cuda"), torch.ones(H, device="cuda")
    for ckpt in (False, True):  # 1 and -1 are kept exactly in 8 bits
        kept = glr.glr_join(x, h, None, w, one, None, act="none", eps=1e-12, ckpt=True)[2]
        a = (None, None) if ckpt else (h, None)
        dalpha = glr.glr_join_backward(dy, None, x, *a, w, one, None, act="none", eps=1e-12,
                                       ckpt=kept if ckpt else None)[4]
        want = small.sum()
        assert abs(want) > 1
        assert abs(dalpha.item() - want) <= 2.0 ** -24 * abs(want)
