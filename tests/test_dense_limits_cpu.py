"""Sizes of the dense product that its tiles would round past 2^31 are refused before
anything is launched."""
import ctypes

import pytest

GOOD = 0x10000  # an aligned fake address; never dereferenced by a rejected call
MOST = 2 ** 31 - 4096


def vp(v):
    return ctypes.c_void_p(v)


@pytest.fixture(scope="module")
def lib():
    from sparse_moe_expert_gb300 import _build
    _build.build()
    import sparse_moe_expert_gb300 as m
    return m.lib()


# each size alone, in each form: a few rows, tiles, pairs
@pytest.mark.parametrize("T,K,N", [(1, 2 ** 31 - 8, 1), (32, MOST + 8, 16), (2 ** 31 - 1, 8, 1),
                                   (MOST + 1, 64, 4096), (1, 8, 2 ** 31 - 1), (200, 64, MOST + 2),
                                   (40, 2 ** 31 - 8, 64), (4, 8, 2 ** 31 - 2)])
def test_linear(lib, T, K, N):
    for act in (0, 3):
        if act == 3 and N % 2:
            continue
        assert lib.moe_linear(vp(GOOD), K, vp(GOOD), None, None, T, K, N, act, 1, vp(GOOD), None, None) == 1
        cols = N // 2 if act == 3 else N
        ld = (N + 7) // 8 * 8
        for d_x, d_w in ((vp(GOOD), None), (None, vp(GOOD)), (vp(GOOD), vp(GOOD))):
            assert lib.moe_linear_backward(vp(GOOD), 1, cols, vp(GOOD), K, vp(GOOD), vp(GOOD), T, K, N, act,
                                           vp(GOOD), ld, d_x, d_w, 0, 0, None, None, 0, None) == 1
