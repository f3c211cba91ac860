"""Cases of the gated recurrent block for the bounds-checked build, run in a child process with
DLR_BOUNDS_CHECK=1: every entry point on sizes that reach the kernels' tails, every way in and out
of shared memory, chains over several tiles a block; each result against its float64 definition,
and after each call the device status and the first failing site. Prints one JSON line:
{"checked": bool, "cases": [[name, rel_l2, status, site], ...]}."""
import json
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from oracle import glr as og  # noqa: E402
from state_space_sequence_gb300 import dlr, glr  # noqa: E402


def host(t):
    torch.cuda.synchronize()
    return t.detach().double().cpu().numpy()


def normal(seed, *shape, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def run():
    cases = []

    def record(name, pairs):
        err = max(float(np.linalg.norm(host(a) - b) / max(np.linalg.norm(b), 1e-30))
                  for a, b in pairs)
        cases.append([name, err, int(dlr.device_status()), int(dlr.bounds_site())])

    for B, L, H, dtype in [(2, 5, 3, torch.float32), (3, 333, 66, torch.float32),
                           (2, 700, 64, torch.float32), (2, 250, 65, torch.bfloat16),
                           (2, 250, 66, torch.float16), (2, 250, 72, torch.bfloat16),
                           (3, 2500, 640, torch.bfloat16)]:
        x, r, i, dy = (normal(k + L, B, L, H, dtype=dtype) for k in range(4))
        p, h0, dhl = normal(4, H) - 3, normal(5, B, H), normal(6, B, H)
        reset = torch.zeros(B, L, dtype=torch.bool, device="cuda")
        reset[0, L // 2] = True
        y, last, st = glr.glr_scan(x, r, i, p, h0=h0, reset=reset, save_states=True)
        f, cut = [host(t) for t in (x, r, i, p)], reset.cpu().numpy()
        ry, _, rl = og.scan(*f, 8.0, host(h0), cut)
        record(f"scan B{B} L{L} H{H} {dtype}", [(y, ry), (last, rl)])
        got = glr.glr_scan_backward(x, r, i, p, dy, st, h0=h0, reset=reset, dh_last=dhl)
        ref = og.scan_backward(*f, 8.0, host(dy), host(h0), cut, host(dhl))
        record(f"scan gradients B{B} L{L} H{H} {dtype}", list(zip(got, ref)))
        z = glr.glr_step(x[:, 0], r[:, 0], i[:, 0], p, h0)
        sy, _, sh = og.scan(*(t[:, :1] for t in f[:3]), f[3], 8.0, host(normal(5, B, H)))
        record(f"step B{B} H{H} {dtype}", [(z, sy[:, 0]), (h0, sh)])
    for M, H, dtype, act in [(3, 5, torch.float32, "silu"), (5, 515, torch.float32, "sigmoid"),
                             (4, 64, torch.bfloat16, "silu"), (700, 136, torch.float16, "silu"),
                             (3, 2056, torch.bfloat16, "none"), (2, 9000, torch.float32, "silu"),
                             (2, 8200, torch.bfloat16, "silu")]:
        x, h, g, dy, dn = (normal(k + H, M, H, dtype=dtype) for k in range(5))
        g = None if act == "none" else g
        w, v, al = 1 + 0.1 * normal(7, H), 1 + 0.1 * normal(8, H), torch.full((1,), 0.5, device="cuda")
        for norm in ("rms", "layer"):
            y, n, kept = glr.glr_join(x, h, g, w, al, v, norm=norm, act=act, ckpt=True)
            f = [None if t is None else host(t) for t in (x, h, g, w)] + [0.5, host(v)]
            record(f"join {norm} M{M} H{H} {dtype} {act}", list(zip((y, n), og.join(*f, norm, act))))
            got = glr.glr_join_backward(dy, dn, x, h, g, w, al, v, norm=norm, act=act)
            ref = og.join_backward(host(dy), host(dn), *f, norm, act)
            record(f"join gradients {norm} M{M} H{H} {dtype} {act}",
                   [(a, b) for k, (a, b) in enumerate(zip(got, ref)) if a is not None and k < 3])
            got = glr.glr_join_backward(dy, dn, x, None, None, w, al, v, norm=norm, act=act,
                                        ckpt=kept)
            k = [None if c is None else og.ckpt_pack(host(t))[2] for t, c in zip((h, g), kept)]
            ref = og.join_backward(host(dy), host(dn), f[0], *k, *f[3:], norm, act)
            record(f"join gradients kept {norm} M{M} H{H} {dtype} {act}",
                   [(a, b) for k, (a, b) in enumerate(zip(got, ref)) if a is not None and k < 3])
        c = glr.glr_ckpt_pack(h)
        record(f"checkpoint M{M} H{H} {dtype}", [(glr.glr_ckpt_unpack(c), og.ckpt_pack(host(h))[2])])
    return {"checked": dlr.bounds_checked(), "cases": cases}


if __name__ == "__main__":
    print(json.dumps(run()))
