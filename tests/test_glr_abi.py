"""C-ABI checks of include/glr.h that need no GPU: every declared function is exported, sizes are
answered, and invalid arguments are refused on the host before anything is launched."""
import ctypes
import os
import re
import struct

import pytest

from state_space_sequence_gb300 import build as dlr_build
from state_space_sequence_gb300 import glr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5


@pytest.fixture(scope="module")
def lib():
    dlr_build.build()
    return glr._load()


def test_every_declared_function_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "glr.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(glr_[a-z0-9_]+)\s*\(", text))
    assert {"glr_scan", "glr_scan_backward", "glr_step", "glr_join", "glr_join_backward",
            "glr_ckpt_pack", "glr_ckpt_unpack", "glr_states", "glr_scan_workspace_size",
            "glr_abi_version"} <= names
    for n in names:
        assert hasattr(lib, n), n
    assert lib.glr_abi_version() == 1
    assert f"#define GLR_STATE_STEPS {glr.STATE_STEPS}" in text
    assert f"#define GLR_CKPT_GROUP {glr.CKPT_GROUP}" in text


def test_sizes(lib):
    assert [lib.glr_states(n) for n in (0, 1, 8, 9, 4096)] == [0, 1, 1, 2, 512]
    assert lib.glr_scan_workspace_size(0, 10, 10) == 0
    assert lib.glr_scan_workspace_size(1, 10, 0) == 0
    assert lib.glr_scan_workspace_size(1, 1 << 31, 1) == 0
    assert lib.glr_scan_workspace_size(2, 200, 64) > 0
    assert lib.glr_scan_workspace_size(2, 8, 64) == 0           # a row that one block takes
    assert lib.glr_scan_backward_workspace_size(2, 100, 64) > 0
    assert lib.glr_join_backward_workspace_size(5, 16385) == 0
    assert lib.glr_join_backward_workspace_size(5, 1024) > 0


# addresses far apart that are never followed: every call below is refused on the host
A = [k << 40 for k in range(1, 20)]


def scan(type=1, B=2, L=200, H=64, c=8.0, x=(A[0], 12800, 64), r=(A[1], 12800, 64),
         i=(A[2], 12800, 64), p=A[3], h0=0, reset=0, y=(A[4], 12800, 64), h_last=A[5], states=A[6], ws=A[7],
         n=1 << 30):
    return struct.pack("4qd19q", type, B, L, H, c, *x, *r, *i, p, h0, reset, *y, h_last, states,
                       ws, n)


@pytest.mark.parametrize("status,change", [
    (INVALID, {"type": 3}), (INVALID, {"B": 0}), (INVALID, {"L": -1}), (INVALID, {"H": 0}),
    (INVALID, {"c": -1.0}), (INVALID, {"c": float("nan")}), (INVALID, {"c": 1e300}),
    (INVALID, {"x": (0, 12800, 64)}), (INVALID, {"x": (A[0] + 1, 12800, 64)}),
    (INVALID, {"r": (A[1], -1, 64)}), (INVALID, {"p": 0}), (INVALID, {"p": A[3] + 2}),
    (INVALID, {"h0": A[8] + 1}), (INVALID, {"y": (A[4], 12800, 63)}),   # its rows meet
    (INVALID, {"y": (A[4], 64, 64)}), (INVALID, {"y": (A[0], 12800, 64)}),
    (INVALID, {"y": (A[0] + 64, 12800, 64)}), (INVALID, {"h_last": A[6]}),
    (INVALID, {"states": A[7]}), (INVALID, {"h0": A[5]}),
    # columns of one buffer that meet: 64 wide, 63 apart
    (INVALID, {"x": (A[0], 25600, 128), "y": (A[0] + 2 * 63, 25600, 128)}),
    (UNSUPPORTED, {"L": 1 << 31}), (UNSUPPORTED, {"H": (1 << 24) + 1}),
    (UNSUPPORTED, {"B": 1 << 30}),
    (WORKSPACE, {"ws": 0}), (WORKSPACE, {"ws": A[7] + 8}), (WORKSPACE, {"n": 16}),
])
def test_scan_refusals(lib, status, change):
    assert lib.glr_scan(scan(**change), None) == status


def test_null_arguments(lib):
    for f in ("glr_scan", "glr_scan_backward", "glr_step", "glr_join", "glr_join_backward"):
        assert getattr(lib, f)(None, None) == INVALID


def test_scan_backward_refusals(lib):
    v = lambda k: (A[k], 6400, 64)

    def args(L=100, dx=v(4), dr=v(5), di=v(6), states=A[7], dp=A[8], dh0=0, ws=A[9], n=1 << 30,
             dy=v(3)):
        return struct.pack("4qd30q", 1, 2, L, 64, 8.0, *v(0), *v(1), *v(2), *dy, A[10], 0, 0,
                           states, 0, *dx, *dr, *di, dp, dh0, ws, n)
    call = lambda **k: lib.glr_scan_backward(args(**k), None)
    assert call(states=0) == INVALID
    assert call(dp=0) == INVALID
    assert call(L=0, dp=0) == INVALID
    assert call(dx=v(5)) == INVALID                     # two outputs in one place
    assert call(dx=v(3)) == INVALID                     # over an input
    assert call(dr=(A[5], 6400, 0)) == INVALID
    assert call(dh0=A[7]) == INVALID
    assert call(n=16) == WORKSPACE


def test_step_refusals(lib):
    def args(B=4, H=64, h=A[4], out=A[4], y=A[5]):
        return struct.pack("3qd16q", 0, B, H, 8.0, A[0], 64, 0, A[1], 64, 0, A[2], 64, 0, A[3], h, 0,
                           y, 64, 0, out)
    assert lib.glr_step(args(B=0), None) == INVALID
    assert lib.glr_step(args(h=0), None) == INVALID
    assert lib.glr_step(args(out=A[4] + 64), None) == INVALID   # neither in place nor apart
    assert lib.glr_step(args(y=A[4]), None) == INVALID


def join(M=4, H=64, norm=0, act=0, eps=1e-6, x=A[0], h=A[1], g=A[2], w=A[3], al=A[4], v=A[5], y=A[6],
         n=A[7], hc=0, hs=0, gc=0, gs=0, stride=64):
    return struct.pack("5qd22q", 1, M, H, norm, act, eps, x, 0, stride, h, 0, stride, g, 0, stride,
                       w, al, v, y, 0, stride, n, 0, stride, hc, hs, gc, gs)


@pytest.mark.parametrize("status,change", [
    (INVALID, {"M": -1}), (INVALID, {"norm": 2}), (INVALID, {"act": 3}), (INVALID, {"eps": 0.0}),
    (INVALID, {"eps": float("inf")}), (INVALID, {"eps": 1e-60}), (INVALID, {"x": 0}),
    (INVALID, {"h": 0}), (INVALID, {"g": 0}), (INVALID, {"act": 2}), (INVALID, {"w": 0}),
    (INVALID, {"al": 0}), (INVALID, {"v": 0}), (INVALID, {"n": 0}), (INVALID, {"y": A[1]}),
    (INVALID, {"y": A[0] + 2}), (INVALID, {"n": A[0]}), (INVALID, {"n": A[6]}),
    (INVALID, {"hc": A[8]}), (INVALID, {"hc": A[8], "hs": A[9]}),
    (INVALID, {"hc": A[8], "hs": A[9], "gc": A[1], "gs": A[10]}),
    (INVALID, {"stride": 63}), (UNSUPPORTED, {"H": 16385}),
])
def test_join_refusals(lib, status, change):
    assert lib.glr_join(join(**change), None) == status


def test_join_of_no_rows_launches_nothing(lib):
    assert lib.glr_join(join(M=0, x=0, h=0, g=0, y=0, n=0), None) == 0


def test_join_backward_refusals(lib):
    r = lambda p: (p, 0, 64)

    def args(act=0, dy=A[0], dn=A[1], x=A[2], h=A[3], g=A[4], ck=(0, 0, 0, 0), w=A[5], al=A[6], v=A[7],
             dx=A[8], dh=A[9], dg=A[10], dw=A[11], da=A[12], dv=A[13], ws=A[14], n=1 << 30):
        return struct.pack("5qd36q", 1, 4, 64, 0, act, 1e-6, *r(dy), *r(dn), *r(x), *r(h), *r(g),
                           *ck, w, al, v, *r(dx), *r(dh), *r(dg), dw, da, dv, ws, n)
    call = lambda **k: lib.glr_join_backward(args(**k), None)
    for k in ("dn", "x", "h", "g", "al", "dx", "dh", "dg", "dw", "da", "dv"):
        assert call(**{k: 0}) == INVALID, k
    assert call(w=0, v=0) == INVALID
    assert call(act=2) == INVALID                                   # a gate without one
    assert call(ck=(A[15], A[16], A[17], A[18])) == INVALID         # both h and its checkpoint
    assert call(ck=(A[15], A[16], 0, 0), h=0, g=0) == INVALID       # no checkpoint of g
    assert call(dx=A[2]) == INVALID
    assert call(dh=A[3]) == INVALID
    assert call(dw=A[13]) == INVALID
    assert call(n=100) == WORKSPACE


def test_checkpoint_refusals(lib):
    f = lib.glr_ckpt_pack
    assert f(3, 1, 64, A[0], 64, A[1], A[2], None) == INVALID
    assert f(1, -1, 64, A[0], 64, A[1], A[2], None) == INVALID
    assert f(1, 1, 64, A[0], 64, 0, A[2], None) == INVALID
    assert f(1, 1, 64, A[0], 64, A[0], A[2], None) == INVALID
    assert f(1, 1 << 20, 1 << 30, A[0], 1 << 30, A[1], A[2], None) == UNSUPPORTED
    assert f(1, 0, 64, 0, 64, 0, 0, None) == 0
    assert lib.glr_ckpt_unpack(1, 2, 64, A[0], A[1], A[2], 63, None) == INVALID
