"""The gated recurrence (include/glr.h) where a row ends within a warp's eight steps: every result as
the middle rows of a larger buffer, so that a step too many shows beside it, and every result's
values, those of the sums and of the carried states included, where it would enter them. Sizes with
more tiles than the GPU takes at a time, so that blocks go on to a second one."""
import numpy as np
import pytest
import torch

from oracle import glr as og
from state_space_sequence_gb300 import dlr, glr

pytestmark = pytest.mark.gpu

TOL = 1e-5  # of an output's norm, as for any other call; one rounding more in 16 bits
ROUND = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def host(t):
    return t.detach().double().cpu().numpy()


def close(got, ref, scale=None):
    norm = np.linalg.norm(ref) if scale is None else scale
    assert np.linalg.norm(host(got) - ref) <= (TOL + ROUND[got.dtype]) * norm


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H", [65, 258, 264])  # single 16-bit elements, 4-byte and tensor copies
@pytest.mark.parametrize("L", [3, 250, 904, 905, 1017, *range(1025, 1034), 2026])
def test_rows_that_end_within_a_warps_steps(L, H, dtype):
    B, room = 2, 16
    gen = torch.Generator().manual_seed(L + H)
    x, r, i, dy = (torch.randn(B, L, H, generator=gen).to(dtype).cuda() for _ in range(4))
    h0, dhl = (torch.randn(B, H, generator=gen).cuda() for _ in range(2))
    p = torch.linspace(-6.0, 1.0, H, device="cuda")
    reset = torch.zeros(B, L, dtype=torch.bool)
    reset[0, [L // 2, L - 1]] = True
    reset = reset.cuda()
    bufs = [torch.full((B, L + 2 * room, H), 7.0, dtype=dtype, device="cuda") for _ in range(4)]
    y, dx, dr, di = (b[:, room:room + L] for b in bufs)
    _, last, st = glr.glr_scan(x, r, i, p, h0=h0, reset=reset, save_states=True, out=y)
    _, _, _, dp, dh0 = glr.glr_scan_backward(x, r, i, p, dy, st, h0=h0, reset=reset, dh_last=dhl,
                                             out=(dx, dr, di))
    for b in bufs:
        assert (b[:, :room] == 7).all() and (b[:, room + L:] == 7).all()
    f, cut = [host(t) for t in (x, r, i, p)], reset.cpu().numpy()
    ry, _, rlast = og.scan(*f, 8.0, host(h0), cut)
    ref = og.scan_backward(*f, 8.0, host(dy), host(h0), cut, host(dhl))
    for got, q in zip((y, last, dx, dr, di, dp), (ry, rlast, *ref[:4])):
        close(got, q)
    close(dh0, ref[4], scale=np.linalg.norm(ref[4]) + np.linalg.norm(host(dhl)))
    assert dlr.device_status() == 0
