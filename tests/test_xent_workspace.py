"""The loss's workspaces without a GPU: rows that are read as they lie need no room, a call is held to what
its own rows need, and rows that are laid out anew are not let into less."""
import struct

import pytest

from state_space_sequence_gb300 import build as dlr_build
from state_space_sequence_gb300 import xent

INVALID, WORKSPACE = 1, 5
A = [k << 40 for k in range(1, 20)]  # never followed: every call below is refused on the host
M, V, D = 16, 131072, 4096
H_IN, W_IN = 16, 32


@pytest.fixture(scope="module")
def lib():
    dlr_build.build()
    return xent._load()


def test_sizes_of_rows_in_place(lib):
    f, b = lib.xent_loss_workspace_size, lib.xent_loss_backward_workspace_size
    w, h = 2 * V * D, 2 * M * D
    for t in (1, 2):
        assert f(t, M, V, D) - f(t + W_IN, M, V, D) == w
        assert f(t, M, V, D) - f(t + H_IN, M, V, D) == h
        assert f(t, M, V, D) - f(t + H_IN + W_IN, M, V, D) == w + h
        assert b(t, M, V, D) - b(t + W_IN, M, V, D) == w
        assert b(t + H_IN, M, V, D) == b(t, M, V, D)      # it lays h out in any case
        assert f(t + H_IN + W_IN, M, V, D) < 1 << 20      # 16 rows: statistics alone
    for bad in (16, 32, 48, 3 + 16, 64 + 1, -1, -1 + 16):  # float32's rows are never read as they lie
        assert f(bad, M, V, D) == b(bad, M, V, D) == 0


def loss(n, h=(A[0], 0, D), W=(A[1], 0, D), type=1):
    return struct.pack("15q", type, M, V, D, *h, *W, A[2], A[3], A[4], A[5], n)


def back(n, W=(A[1], 0, D), type=1):
    return struct.pack("21q", type, M, V, D, A[0], 0, D, *W, A[2], A[3], A[4], A[5], 0, D, A[6], 0, D, A[7], n)


@pytest.mark.parametrize("ptr,step", [(A[1] + 2, D), (A[1] + 8, D), (A[1], D + 4), (A[1], 0), (A[1], D - 8)])
def test_rows_that_are_laid_out_need_their_room(lib, ptr, step):
    """Off 16 bytes, steps of no multiple of 8, one row for all, rows that overlap."""
    f, b = lib.xent_loss_workspace_size, lib.xent_loss_backward_workspace_size
    n = f(1 + H_IN, M, V, D)
    assert lib.xent_loss(loss(n - 1, W=(ptr, 0, step)), None) == WORKSPACE
    assert lib.xent_loss(loss(f(1 + W_IN, M, V, D) - 1, h=(ptr - A[1] + A[0], 0, step)), None) == WORKSPACE
    assert lib.xent_loss_backward(back(b(1, M, V, D) - 1, W=(ptr, 0, step)), None) == WORKSPACE


def test_a_byte_less_is_refused(lib):
    assert lib.xent_loss(loss(lib.xent_loss_workspace_size(1 + 48, M, V, D) - 1), None) == WORKSPACE
    assert lib.xent_loss_backward(back(lib.xent_loss_backward_workspace_size(1 + 32, M, V, D) - 1),
                                  None) == WORKSPACE
    assert lib.xent_loss(loss(lib.xent_loss_workspace_size(0, M, V, D) - 1, type=0), None) == WORKSPACE
    # a call's own type has no flags
    assert lib.xent_loss(loss(1 << 40, type=1 + W_IN), None) == INVALID
