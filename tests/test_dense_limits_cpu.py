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


def test_adamw_refuses_buffers_that_tensors_share_across_their_kinds(lib):
    from sparse_moe_expert_gb300._lib import AdamWTensor
    MB = 1 << 20
    names = ["param", "grad", "master", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"]
    n = 1000
    size = dict(param=2 * n, grad=2 * n, master=4 * n, exp_avg=n, exp_avg_sq=n, exp_avg_scale=16,
                exp_avg_sq_scale=16)

    def call(ts):  # bf16 params with masters, 8-bit states
        arr = (AdamWTensor * len(ts))(*[AdamWTensor(**t) for t in ts])
        return lib.moe_adamw_step(arr, len(ts), 1, 1, 8, 1e-3, None, 0.9, 0.99, 1e-8, None, vp(MB), None)
    for order in ((0, 1, 2), (2, 0, 1)):  # in the order of their addresses, and not
        for k in names:
            for other in names:
                if k == other:
                    continue
                for i, j in ((0, 2), (2, 0), (1, 2)):
                    ts = [dict({m: MB * (1 + o * 8 + c) for c, m in enumerate(names)}, n=n, weight_decay=0.0)
                          for o in order]
                    ts[i][k] = ts[j][other] + (size[other] - 4)
                    assert call(ts) == 1, (k, other, i, j)
                    ts[i][k] = ts[j][other] - (size[k] - 4)
                    assert call(ts) == 1, (k, other, i, j)
