"""C-ABI checks of include/ssm.h and include/xent.h that need no GPU: every declared function is
exported, the argument structs have the fields that the binding packs, sizes are answered, and
invalid arguments are refused on the host before anything is launched."""
import os
import re
import struct

import pytest

from state_space_sequence_gb300 import build as dlr_build
from state_space_sequence_gb300 import ssm, xent

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5

# addresses far apart that are never followed: every call below is refused on the host
A = [k << 40 for k in range(1, 40)]


@pytest.fixture(scope="module")
def lib():
    dlr_build.build()
    xent._load()
    return ssm._load()


def header(name):
    return re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", name)).read(), flags=re.S)


def test_every_declared_function_is_exported(lib):
    for name, prefix in (("ssm.h", "ssm_"), ("xent.h", "xent_")):
        names = set(re.findall(rf"\b({prefix}[a-z0-9_]+)\s*\(", header(name)))
        assert f"{prefix}abi_version" in names and len(names) >= 5
        for n in names:
            assert hasattr(lib, n), n
        assert getattr(lib, f"{prefix}abi_version")() == 1
    text = header("ssm.h")
    assert f"#define SSM_STATE_STEPS {ssm.STATE_STEPS}" in text
    assert f"#define SSM_MAX_TAPS {ssm.MAX_TAPS}" in text
    assert f"#define SSM_MAX_STATES {ssm.MAX_STATES}" in text


def test_structs_have_the_fields_that_are_packed():
    """Every field is 8 bytes wide, a view three of them."""
    size = {}
    for name in ("ssm.h", "xent.h"):
        for body, struct_name in re.findall(r"typedef struct \{(.*?)\} (\w+);", header(name), re.S):
            n = 0
            for line in filter(None, (x.strip() for x in body.split(";"))):
                n += len(line.split(",")) * (3 if line.startswith("glr_") else 1)
            size[struct_name] = 8 * n
    mod = {"ssm_conv_args": ssm._CONV, "ssm_conv_backward_args": ssm._CONV_BACK,
           "ssm_conv_step_args": ssm._CONV_STEP, "ssm_scan_args": ssm._SCAN,
           "ssm_scan_backward_args": ssm._SCAN_BACK, "ssm_step_args": ssm._STEP,
           "xent_loss_args": xent._LOSS, "xent_loss_backward_args": xent._BACK}
    assert set(mod) == set(size)
    for name, pack in mod.items():
        assert pack.__self__.size == size[name], name


def test_sizes(lib):
    assert [lib.ssm_states(n) for n in (0, 1, 16, 17, 4096)] == [0, 1, 1, 2, 256]
    w = lib.ssm_scan_workspace_size
    assert w(0, 10, 10, 4, 1) == w(1, 10, 0, 4, 1) == w(1, 10, 10, 65, 1) == w(1, 10, 10, 4, 3) == 0
    assert w(1, 1 << 31, 1, 1, 1) == 0
    assert w(4, 4096, 4096, 16, 1) == 0 and w(1, 4096, 64, 16, 1) > 0
    b = lib.ssm_scan_backward_workspace_size
    assert b(2, 100, 64, 16, 1) > 0 and b(2, 100, 64, 16, 5) == 0 and b(2, 0, 64, 16, 1) == 0
    c = lib.ssm_conv_backward_workspace_size
    assert c(2, 100, 64, 4) > 0 and c(2, 100, 64, 9) == c(2, 100, 64, 0) == 0
    for f in (lib.xent_loss_workspace_size, lib.xent_loss_backward_workspace_size):
        assert f(1, 10, 100, 64) > 0
        assert f(3, 10, 100, 64) == f(1, 0, 100, 64) == f(1, 10, 0, 64) == f(1, 1, 1, 1 << 21) == 0
    # a piece's gradient of the logits stays within its bound, however many columns there are
    assert lib.xent_loss_backward_workspace_size(1, 8192, 1 << 20, 64) < 512 << 20


def test_null_arguments(lib):
    for f in ("ssm_conv", "ssm_conv_backward", "ssm_conv_step", "ssm_scan", "ssm_scan_backward",
              "ssm_step", "xent_loss", "xent_loss_backward"):
        assert getattr(lib, f)(None, None) == INVALID


V = (lambda k, st=64, n=200: (A[k], n * st, st))


def conv(type=1, B=2, L=200, H=64, K=4, act=0, x=V(0), w=A[1], bias=A[2], state=A[3], reset=A[4],
         y=V(5), last=A[6]):
    return struct.pack("17q", type, B, L, H, K, act, *x, w, bias, state, reset, *y, last)


@pytest.mark.parametrize("status,change", [
    (INVALID, {"type": 3}), (INVALID, {"B": 0}), (INVALID, {"L": -1}), (INVALID, {"H": 0}),
    (INVALID, {"K": 0}), (UNSUPPORTED, {"K": 9}), (INVALID, {"act": 2}),
    (INVALID, {"K": 1}),                                        # no rows to carry
    (INVALID, {"x": (0, 12800, 64)}), (INVALID, {"x": (A[0] + 1, 12800, 64)}),
    (INVALID, {"x": (A[0], -1, 64)}), (INVALID, {"w": 0}), (INVALID, {"w": A[1] + 2}),
    (INVALID, {"bias": A[2] + 1}), (INVALID, {"state": A[3] + 1}), (INVALID, {"last": A[6] + 1}),
    (INVALID, {"y": (A[5], 12800, 63)}), (INVALID, {"y": V(0)}), (INVALID, {"last": A[3]}),
    (INVALID, {"last": A[5] + 128}), (INVALID, {"y": (A[5], 1 << 40, 1 << 40)}),
    (UNSUPPORTED, {"L": 1 << 31}), (UNSUPPORTED, {"H": (1 << 24) + 1}),
    (UNSUPPORTED, {"B": 1 << 30, "L": 1 << 20}),
    (INVALID, {"L": 0, "last": A[3] + 2}),                      # neither in place nor apart
])
def test_convolution_refusals(lib, status, change):
    assert lib.ssm_conv(conv(**change), None) == status


def test_convolution_backward_refusals(lib):
    def args(K=4, L=200, x=V(0), dy=V(1), w=A[2], state=A[4], dlast=A[6], dx=V(7), dw=A[8], db=A[9],
             ds=A[10], ws=A[11], n=1 << 30):
        return struct.pack("25q", 1, 2, L, 64, K, 0, *x, *dy, w, A[3], state, A[5], dlast, *dx, dw, db,
                           ds, ws, n)
    call = lambda **k: lib.ssm_conv_backward(args(**k), None)
    for k in ("dw", "w"):
        assert call(**{k: 0}) == INVALID, k
    for k in ("x", "dy", "dx"):
        assert call(**{k: (0, 12800, 64)}) == INVALID, k
    assert call(dx=V(1)) == INVALID and call(dx=V(0)) == INVALID   # over an input
    assert call(ds=A[4]) == INVALID and call(db=A[8]) == INVALID
    assert call(K=1) == INVALID
    assert call(n=16) == WORKSPACE and call(ws=A[11] + 4) == WORKSPACE and call(ws=0) == WORKSPACE
    assert call(L=0, dw=0) == INVALID and call(L=0, ds=A[8]) == INVALID


def test_convolution_step_refusals(lib):
    def args(B=4, K=4, x=(A[0], 64, 0), w=A[1], state=A[3], y=(A[5], 64, 0), out=A[3]):
        return struct.pack("16q", 0, B, 64, K, 0, *x, w, A[2], state, 0, *y, out)
    call = lambda **k: lib.ssm_conv_step(args(**k), None)
    assert call(B=0) == INVALID and call(w=0) == INVALID and call(y=(A[0], 64, 0)) == INVALID
    assert call(state=0) == INVALID and call(out=0) == INVALID and call(K=1) == INVALID
    assert call(out=A[3] + 64) == INVALID                          # neither in place nor apart
    assert call(y=(A[5], 63, 0)) == INVALID


def scan(type=1, B=2, L=200, H=64, N=16, G=1, sp=1, x=V(0), dt=V(1), z=V(2), Bm=V(3, 16), Cm=V(4, 16),
         rate=A[5], D=A[6], bias=A[7], h0=A[8], reset=A[9], y=V(10), last=A[11], states=A[12],
         ws=A[13], n=1 << 30):
    return struct.pack("34q", type, B, L, H, N, G, sp, *x, *dt, *z, *Bm, *Cm, rate, D, bias, h0, reset,
                       *y, last, states, ws, n)


@pytest.mark.parametrize("status,change", [
    (INVALID, {"type": -1}), (INVALID, {"B": 0}), (INVALID, {"L": -1}), (INVALID, {"H": 0}),
    (INVALID, {"N": 0}), (UNSUPPORTED, {"N": 65}), (INVALID, {"G": 0}), (INVALID, {"G": 3}),
    (INVALID, {"sp": 2}), (INVALID, {"x": (0, 1, 1)}), (INVALID, {"dt": (A[1] + 1, 12800, 64)}),
    (INVALID, {"z": (A[2], -64, 64)}), (INVALID, {"Bm": (0, 3200, 16)}), (INVALID, {"Cm": (0, 3200, 16)}),
    (INVALID, {"rate": 0}), (INVALID, {"rate": A[5] + 1}), (INVALID, {"D": A[6] + 2}),
    (INVALID, {"bias": A[7] + 2}), (INVALID, {"h0": A[8] + 2}), (INVALID, {"last": A[11] + 2}),
    (INVALID, {"states": A[12] + 2}), (INVALID, {"y": V(0)}), (INVALID, {"y": V(2)}),
    (INVALID, {"y": (A[10], 64, 64)}), (INVALID, {"y": (A[10], 12800, 0)}), (INVALID, {"last": A[8]}),
    (INVALID, {"last": A[12]}), (INVALID, {"states": A[13]}), (INVALID, {"states": A[5]}),
    (WORKSPACE, {"ws": 0}), (WORKSPACE, {"ws": A[13] + 8}), (WORKSPACE, {"n": 16}),
    (UNSUPPORTED, {"L": 1 << 31}), (UNSUPPORTED, {"H": 1 << 25}), (UNSUPPORTED, {"B": 1 << 26}),
    (INVALID, {"x": (A[0], 1 << 40, 1 << 40)}),
    (INVALID, {"L": 0, "last": A[8] + 16}),
])
def test_scan_refusals(lib, status, change):
    assert lib.ssm_scan(scan(**change), None) == status


def test_scan_backward_refusals(lib):
    base = dict(x=V(0), dt=V(1), z=V(2), Bm=V(3, 16), Cm=V(4, 16), dy=V(5), rate=A[6], D=A[7],
                bias=A[8], h0=A[9], reset=A[10], states=A[11], dhl=A[12], dx=V(13), ddt=V(14), dz=V(15),
                dBm=V(16, 16), dCm=V(17, 16), dA=A[18], dD=A[19], db=A[20], dh0=A[21], ws=A[22],
                n=1 << 40, L=200)

    def call(**k):
        a = {**base, **k}
        L = a.pop("L")
        flat = [v for t in a.values() for v in (t if isinstance(t, tuple) else (t,))]
        return lib.ssm_scan_backward(struct.pack("53q", 1, 2, L, 64, 16, 1, 1, *flat), None)
    none = (0, 0, 0)
    for k in ("x", "dt", "Bm", "Cm", "dy", "dx", "ddt", "dBm", "dCm", "dz"):
        assert call(**{k: none}) == INVALID, k
    for k in ("rate", "states", "dA", "dD"):
        assert call(**{k: 0}) == INVALID, k
    assert call(D=0) == INVALID                                    # dD without D
    assert call(z=none) == INVALID                                 # dz without z
    for k in ("dx", "ddt", "dz"):
        assert call(**{k: V(5)}) == INVALID and call(**{k: V(0)}) == INVALID
    assert call(dBm=V(17, 16)) == INVALID and call(dBm=V(3, 16)) == INVALID
    assert call(dA=A[6]) == INVALID and call(dh0=A[12]) == INVALID and call(db=A[19]) == INVALID
    assert call(n=16) == WORKSPACE and call(ws=0) == WORKSPACE
    assert call(L=0, dA=0) == INVALID and call(L=0, dh0=A[18]) == INVALID


def test_step_refusals(lib):
    def args(B=4, N=16, G=1, Bm=(A[3], 16, 0), rate=A[5], h=A[8], y=(A[10], 64, 0), out=A[8]):
        v = lambda k: (A[k], 64, 0)
        return struct.pack("30q", 0, B, 64, N, G, 1, *v(0), *v(1), *v(2), *Bm, A[4], 16, 0, rate, A[6],
                           A[7], h, 0, *y, out)
    call = lambda **k: lib.ssm_step(args(**k), None)
    assert call(B=0) == INVALID and call(h=0) == INVALID and call(out=0) == INVALID
    assert call(rate=0) == INVALID and call(Bm=(0, 16, 0)) == INVALID and call(G=5) == INVALID
    assert call(N=65) == UNSUPPORTED and call(B=1 << 26) == UNSUPPORTED
    assert call(out=A[8] + 16) == INVALID                          # neither in place nor apart
    assert call(y=(A[0], 64, 0)) == INVALID and call(y=(A[10], 60, 0)) == INVALID


def test_loss_refusals(lib):
    def args(type=1, M=10, V=100, D=64, h=(A[0], 0, 64), W=(A[1], 0, 64), target=A[2], loss=A[3],
             lse=A[4], ws=A[5], n=1 << 40):
        return struct.pack("15q", type, M, V, D, *h, *W, target, loss, lse, ws, n)
    call = lambda **k: lib.xent_loss(args(**k), None)
    assert call(type=3) == INVALID and call(M=-1) == INVALID and call(V=0) == INVALID
    assert call(D=0) == INVALID and call(D=(1 << 20) + 1) == UNSUPPORTED
    assert call(V=1 << 31) == UNSUPPORTED and call(M=1 << 31) == UNSUPPORTED
    assert call(V=1 << 30, D=128) == UNSUPPORTED
    for k in ("target", "loss", "lse"):
        assert call(**{k: 0}) == INVALID and call(**{k: A[6] + 2}) == INVALID, k
    assert call(h=(0, 0, 64)) == INVALID and call(W=(A[1] + 1, 0, 64)) == INVALID
    assert call(h=(A[0], 0, -1)) == INVALID
    assert call(loss=A[4]) == INVALID and call(lse=A[0]) == INVALID
    assert call(ws=0) == WORKSPACE and call(ws=A[5] + 128) == WORKSPACE and call(n=100) == WORKSPACE
    assert call(M=0, h=(0, 0, 0), target=0, loss=0, lse=0, ws=0) == 0


def test_loss_backward_refusals(lib):
    def args(M=10, h=(A[0], 0, 64), W=(A[1], 0, 64), target=A[2], lse=A[3], dloss=A[4],
             dh=(A[5], 0, 64), dW=(A[6], 0, 64), ws=A[7], n=1 << 40):
        return struct.pack("21q", 1, M, 100, 64, *h, *W, target, lse, dloss, *dh, *dW, ws, n)
    call = lambda **k: lib.xent_loss_backward(args(**k), None)
    for k in ("target", "lse", "dloss"):
        assert call(**{k: 0}) == INVALID, k
    assert call(dh=(A[0], 0, 64)) == INVALID and call(dW=(A[1], 0, 64)) == INVALID
    assert call(dh=(A[6], 0, 64)) == INVALID and call(dh=(A[5], 0, 63)) == INVALID
    assert call(dW=(A[6], 0, 63)) == INVALID and call(dW=(A[6] + 1, 0, 64)) == INVALID
    assert call(dW=(A[7], 0, 64)) == INVALID
    assert call(ws=0) == WORKSPACE and call(n=64) == WORKSPACE
    assert call(dh=(0, 0, 0), dW=(0, 0, 0)) == 0                   # nothing wanted
    assert call(M=0, dW=(0, 0, 0)) == 0
