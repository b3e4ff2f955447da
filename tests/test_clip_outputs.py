"""Clipping refuses outputs that overlap; host checks only, no GPU is touched."""
import ctypes

import pytest

from gated_delta_rule_42_gb300 import _lib, build

A = 0x100000  # a well-aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def clip(lib, at, sizes, kinds):
    n = len(at)
    p, z, k = (ctypes.c_void_p * n)(*at), (ctypes.c_int64 * n)(*sizes), (ctypes.c_int * n)(*kinds)
    return lib.kda_clip_grad_norm(n, p, p, z, k, 1.0, A, A, 1 << 40, None)


@pytest.mark.parametrize("at,sizes,kinds", [
    ([A, A + 64, A], [4, 4, 4], [0, 0, 0]),                    # listed twice
    ([A, A + 12], [4, 4], [0, 0]),                             # the last element of one is the first of the other
    ([A + 12, A], [4, 4], [0, 0]),
    ([A + 100, A, A + 40], [4, 11, 4], [0, 0, 0]),
    ([A, A + 4], [3, 4], [1, 0]),                              # bf16 and fp32
    ([A, A + 8], [100, 1], [0, 0]),                            # one inside the other
    ([A, A + 64, A + 16, A + 80], [4, 4, 32, 4], [0, 1, 0, 1]),  # each type ascends, the two meet
    ([A + 64, A, A + 80, A + 8], [4, 4, 4, 100], [0, 1, 0, 1]),
])
def test_overlapping_outputs(lib, at, sizes, kinds):
    assert clip(lib, at, sizes, kinds) == _lib.KDA_ERR_INVALID_ARG
    assert b"overlap" in lib.kda_last_error()
