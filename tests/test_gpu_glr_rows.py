"""The join and its gradients (include/glr.h) over more rows than the GPU takes at a time, so that
every block goes on from row to row: the copies of the next row, its checkpoint scales, the sums
kept across rows. Row by row against the float64 definition, on the rows that a block takes late too."""
import numpy as np
import pytest
import torch

from oracle import glr as og
from state_space_sequence_gb300 import dlr, glr

pytestmark = pytest.mark.gpu

ROUND = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def host(t):
    return t.detach().double().cpu().numpy()


def normal(seed, *shape, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def rows_near(got, ref):
    """Every row within 1e-5 of its norm, and one rounding of its type: with relative errors of
    2^-24 an operation and some 40 of them in a chain, 2.4e-6 would be the most on a line."""
    off = np.linalg.norm(host(got) - ref, axis=1)
    assert (off <= (1e-5 + ROUND[got.dtype]) * np.linalg.norm(ref, axis=1)).all()


# 16-byte accesses, single channels, and one and several warps to a row; an SM holds at most 32 blocks
# of one warp, so 10000 rows are several to each of a GPU's blocks
CASES = [(10000, 136, "rms", "silu"), (10000, 136, "layer", "sigmoid"), (10000, 131, "rms", "silu"),
         (3000, 771, "layer", "silu"), (3000, 1024, "rms", "silu"), (1500, 2056, "rms", "none"),
         (400, 8200, "layer", "silu")]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,H,norm,act", CASES)
def test_many_rows(M, H, norm, act, dtype):
    x, h, g, dy, dn = (normal(k + H, M, H, dtype=dtype) for k in range(5))
    g = None if act == "none" else g
    # rows of sizes that differ, so that a row's numbers used in another's place would show
    for k, t in enumerate((x, h, dy, dn)):
        t.mul_(torch.exp2(torch.arange(M, device="cuda").mul(k + 1).remainder(7) - 3.0)[:, None])
    w, v = 1 + 0.3 * normal(5, H), 1 + 0.3 * normal(6, H)
    al = torch.full((1,), 0.7, device="cuda")
    y, n, kept = glr.glr_join(x, h, g, w, al, v, norm, act, ckpt=True)
    f = [None if t is None else host(t) for t in (x, h, g, w, al, v)]
    f[4] = f[4][0]
    for a, q in zip((y, n), og.join(*f, norm, act)):
        rows_near(a, q)
    for t, c in zip((h, g), kept):
        assert (t is None) == (c is None)
        if t is not None:
            alone = glr.glr_ckpt_pack(t)
            assert torch.equal(alone.codes, c.codes) and torch.equal(alone.scales, c.scales)
    for ckpt in (False, True):
        if ckpt:
            f[1:3] = [None if c is None else host(glr.glr_ckpt_unpack(c)) for c in kept]
        got = glr.glr_join_backward(dy, dn, x, *((None, None) if ckpt else (h, g)), w, al, v, norm, act,
                                    ckpt=kept if ckpt else None)
        ref = og.join_backward(host(dy), host(dn), *f, norm, act)
        for a, q in zip(got[:3], ref[:3]):
            assert (a is None) == (q is None)
            if a is not None:
                rows_near(a, q)
        un = og.norm(f[1] * og.act(f[2], act)[0], norm, 1e-6)[0]
        yn = og.norm(og.join(*f, norm, act)[0], norm, 1e-6)[0]
        terms = ref[0] * un
        # sums of M terms of either sign, each off by some 2^-21 of itself: held to 2^-17 of the
        # root of their squares' sum, channel by channel
        for a, q, t in ((got[3], ref[3], 0.7 * terms), (got[5], ref[5], host(dn) * yn)):
            assert (np.abs(host(a) - q) <= 2.0 ** -17 * np.linalg.norm(t, axis=0)).all()
        assert abs(got[4].item() - ref[4][0]) <= 2.0 ** -17 * np.linalg.norm(f[3] * terms)
    assert dlr.device_status() == 0
