"""Cases of the selective block's operators and of the loss over a vocabulary for the bounds-checked
build, run in a child process with DLR_BOUNDS_CHECK=1: every entry point on sizes that reach the
kernels' tails, whole and ragged rows, cut sequences, few rows and several tiles; each result against
its float64 definition, and after each call the device status and the first failing site. Prints one
JSON line: {"checked": bool, "cases": [[name, rel_l2, status, site], ...]}."""
import json
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from oracle import ssm as osm  # noqa: E402
from oracle import xent as ox  # noqa: E402
from state_space_sequence_gb300 import dlr, ssm, xent  # noqa: E402

TYPES = (torch.float32, torch.bfloat16, torch.float16)


def host(t):
    torch.cuda.synchronize()
    return None if t is None else t.detach().double().cpu().numpy()


def normal(seed, *shape, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def run():
    cases = []

    def record(name, results):
        """results: (got, reference) or (got, reference, what its terms may add up to)."""
        err = 0.0
        for got, ref, *scale in results:
            norm = np.linalg.norm(ref) + sum(np.linalg.norm(s) for s in scale)
            err = max(err, float(np.linalg.norm(host(got) - ref) / max(norm, 1e-30)))
        cases.append([name, err, int(dlr.device_status()), int(dlr.bounds_site())])

    for k, (B, L, H, K) in enumerate([(1, 1, 3, 4), (2, 37, 66, 4), (3, 130, 136, 3), (2, 300, 264, 8),
                                      (70, 2, 520, 2)]):
        for dtype in TYPES:
            name = f"B{B} L{L} H{H} K{K} {dtype}"
            x, dy = normal(k, B, L, H, dtype=dtype), normal(k + 1, B, L, H, dtype=dtype)
            w, bias = normal(k + 2, H, K) / K ** 0.5, normal(k + 3, H)
            state, dlast = (normal(k + j, B, K - 1, H, dtype=dtype) for j in (4, 5))
            reset = torch.zeros(B, L, dtype=torch.bool, device="cuda")
            reset[0, L // 2] = True
            f, cut = [host(x), host(w)], reset.cpu().numpy()
            y, last = ssm.ssm_conv(x, w, bias, state, reset)
            ry, rl, _ = osm.conv(*f, host(bias), host(state), cut)
            record(f"convolution {name}", [(y, ry), (last, rl)])
            got = ssm.ssm_conv_backward(x, w, dy, bias, state, reset, dlast=dlast)
            ref = osm.conv_backward(*f, host(dy), host(bias), host(state), cut, dlast=host(dlast))
            record(f"convolution gradients {name}", list(zip(got, ref)))
            first = host(state)
            z = ssm.ssm_conv_step(x[:, 0], w, state, bias)
            ry, rl, _ = osm.conv(f[0][:, :1], f[1], host(bias), first)
            record(f"convolution step {name}", [(z, ry[:, 0]), (state, rl)])

    for k, (B, L, H, G, N) in enumerate([(2, 5, 3, 1, 1), (1, 333, 66, 1, 16), (2, 300, 64, 2, 8),
                                         (1, 700, 40, 1, 64), (2, 130, 264, 1, 32)]):
        for dtype in TYPES:
            name = f"B{B} L{L} H{H} G{G} N{N} {dtype}"
            x, dt, z, dy = (normal(10 * k + j, B, L, H, dtype=dtype) for j in range(4))
            Bm, Cm = (normal(10 * k + j, B, L, G, N, dtype=dtype) for j in (4, 5))
            A = -torch.exp(normal(10 * k + 6, H, N) * 0.5)
            D, bias = normal(10 * k + 7, H), normal(10 * k + 8, H) - 2
            h0, dhl = normal(10 * k + 9, B, H, N), normal(10 * k + 10, B, H, N)
            reset = torch.zeros(B, L, dtype=torch.bool, device="cuda")
            reset[0, L // 2] = True
            how = {"D": D, "z": z, "dt_bias": bias}
            f = [host(t) for t in (x, dt, A, Bm, Cm)]
            rest, cut = [host(t) for t in (D, z, bias)], reset.cpu().numpy()
            y, last, st = ssm.ssm_scan(x, dt, A, Bm, Cm, h0=h0, reset=reset, save_states=True, **how)
            ry, _, rl, _ = osm.scan(*f, *rest, True, host(h0), cut)
            record(f"scan {name}", [(y, ry), (last, rl)])
            g = ssm.ssm_scan_backward(x, dt, A, Bm, Cm, dy, st, h0=h0, reset=reset, dh_last=dhl, **how)
            ref = osm.scan_backward(*f, host(dy), *rest, True, host(h0), cut, host(dhl))
            got = (g.dx, g.ddt, g.dA, g.dB, g.dC, g.dD, g.dz, g.ddt_bias, g.dh0)
            record(f"scan gradients {name}", [(a, r) for a, r in zip(got, ref)])
            first = host(h0)
            z1 = ssm.ssm_step(x[:, 0], dt[:, 0], A, Bm[:, 0], Cm[:, 0], h0, D=D, z=z[:, 0], dt_bias=bias)
            ry, _, rl, _ = osm.scan(*(t[:, :1] for t in f[:2]), f[2], *(t[:, :1] for t in f[3:]), rest[0],
                                    rest[1][:, :1], rest[2], True, first)
            record(f"scan step {name}", [(z1, ry[:, 0]), (h0, rl)])

    for M, V, D in [(1, 3, 5), (16, 1000, 72), (130, 515, 65), (300, 700, 264)]:
        for dtype in TYPES:
            h, W = normal(M, M, D, dtype=dtype), (normal(V, V, D) / D ** 0.5).to(dtype)
            target = torch.randint(0, V, (M,), generator=torch.Generator().manual_seed(D)).cuda()
            dloss = torch.rand(M, generator=torch.Generator().manual_seed(M)).cuda()
            loss, lse = xent.xent_loss(h, W, target)
            f = [host(h), host(W), target.cpu().numpy()]
            rl, rs, zz = ox.loss(*f)
            record(f"loss M{M} V{V} D{D} float32 of {str(dtype)[6:8]}", [(loss, rl, rs), (lse, rs)])
            dh, dW = xent.xent_loss_backward(h, W, target, lse, dloss)
            rh, rW = ox.loss_backward(*f, host(dloss))
            d = np.exp(zz - rs[:, None])
            d[np.arange(M), f[2]] -= 1.0
            d = np.abs(d) * host(dloss)[:, None]
            record(f"loss gradients M{M} V{V} D{D} {dtype}",
                   [(dh, rh, d @ np.abs(f[1])), (dW, rW, d.T @ np.abs(f[0]))])
    return {"checked": dlr.bounds_checked(), "cases": cases}


if __name__ == "__main__":
    print(json.dumps(run()))
