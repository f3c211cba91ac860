"""Sizes that the 8-bit checkpoints (include/glr.h) take and refuse. No GPU is needed and no address
is followed: every call below is refused on the host."""

import pytest

from state_space_sequence_gb300 import build as dlr_build
from state_space_sequence_gb300 import glr

INVALID, UNSUPPORTED = 1, 2
T, CODES, SCALES = (k << 44 for k in (1, 2, 3))
MOST = 2 ** 34 - 8  # groups: 2^31 - 1 blocks of 256 threads


@pytest.fixture(scope="module")
def lib():
    dlr_build.build()
    return glr._load()


@pytest.mark.parametrize("type", [0, 1, 2])
@pytest.mark.parametrize("M,H", [
    (2 ** 34, 1), (2 ** 34, 31), (2 ** 34, 32), (MOST + 1, 1), (MOST // 2 + 1, 33),
    (2 ** 35 + 64, 1),       # 2^32 + 8 blocks, which an unsigned int holds as 8
    (2 ** 35 + 8, 31),
    (1, 2 ** 31 - 31), (1, 2 ** 31 - 1),   # whose last group passes 2^31
    (2 ** 62, 1), (2 ** 62, 2 ** 31 - 32), (1, 2 ** 62),
])
def test_more_groups_than_a_launch_takes_are_refused(lib, type, M, H):
    assert lib.glr_ckpt_pack(type, M, H, T, H, CODES, SCALES, None) == UNSUPPORTED
    assert lib.glr_ckpt_unpack(type, M, H, CODES, SCALES, T, H, None) == UNSUPPORTED


@pytest.mark.parametrize("M,H", [(MOST, 1), (MOST, 32), (MOST // 2, 33), (8, 2 ** 31 - 32), (1, 2 ** 31 - 32)])
def test_the_largest_sizes_pass_that_check(lib, M, H):
    """They are refused for an address that is missing, not for their size."""
    assert lib.glr_ckpt_pack(0, M, H, T, H, 0, SCALES, None) == INVALID
    assert lib.glr_ckpt_unpack(0, M, H, 0, SCALES, T, H, None) == INVALID
