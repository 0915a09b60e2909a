"""Refusals of the norms, the dense product and AdamW that need no GPU: the C
calls return a status before anything is launched, and the Python calls refuse
tensors that are not on a device."""
import ctypes

import pytest
import torch

GOOD = 0x10000  # an aligned fake address; never dereferenced by a rejected call


def vp(v):
    return ctypes.c_void_p(v)


@pytest.fixture(scope="module")
def moe():
    from sparse_moe_expert_gb300 import _build
    _build.build()
    import sparse_moe_expert_gb300 as m
    m.lib()
    return m


def check(f, names, good, cases):
    """Each case: (status, changed arguments)."""
    assert len(names) == len(f.argtypes), "argument list"
    for want, over in cases:
        a = dict(good, **over)
        assert set(over) <= set(names), over
        assert f(*(a[n] for n in names)) == want, over


def test_layer_norm(moe):
    f = moe.lib().moe_layer_norm
    names = ("x xt ldx r ldr w b wt T H kind eps ot out s mean rstd st").split()
    good = dict(x=vp(GOOD), xt=1, ldx=64, r=None, ldr=0, w=vp(GOOD), b=None, wt=0, T=4, H=64, kind=0,
                eps=1e-6, ot=1, out=vp(GOOD), s=None, mean=None, rstd=None, st=None)
    check(f, names, good, [
        (1, dict(T=-1)), (1, dict(H=0)), (1, dict(H=8193)), (1, dict(kind=2)), (1, dict(xt=2)),
        (1, dict(ot=5)), (1, dict(wt=-1)), (1, dict(eps=-1e-3)), (1, dict(eps=float("nan"))),
        (1, dict(eps=float("inf"))), (1, dict(x=None)), (1, dict(out=None)), (1, dict(ldx=63)),
        (1, dict(x=vp(GOOD + 1))), (1, dict(w=vp(GOOD + 2))), (1, dict(out=vp(GOOD + 1))),
        (1, dict(r=vp(GOOD), ldr=64)),                    # a residual needs summed
        (1, dict(r=vp(GOOD), ldr=8, s=vp(GOOD))), (1, dict(mean=vp(GOOD + 2))),
        (0, dict(T=0, x=None, out=None)),
    ])


def test_layer_norm_backward(moe):
    f = moe.lib().moe_layer_norm_backward
    names = ("d dt ldd x xt ldx mean rstd w wt ds lds T H dx dw db ws wsb st").split()
    good = dict(d=vp(GOOD), dt=1, ldd=64, x=vp(GOOD), xt=1, ldx=64, mean=vp(GOOD), rstd=vp(GOOD),
                w=vp(GOOD), wt=0, ds=None, lds=0, T=4, H=64, dx=vp(GOOD), dw=vp(GOOD), db=None,
                ws=vp(GOOD), wsb=1 << 24, st=None)
    check(f, names, good, [
        (1, dict(H=8193)), (1, dict(T=-2)), (1, dict(dt=3)), (1, dict(rstd=None)), (1, dict(dx=None)),
        (1, dict(ldd=1)), (1, dict(ds=vp(GOOD), lds=0)), (1, dict(ws=None)), (1, dict(wsb=16)),
        (1, dict(ws=vp(GOOD + 4))), (1, dict(dw=vp(GOOD + 1))), (1, dict(d=vp(GOOD + 1))),
    ])
    assert moe.moe_layer_norm_workspace_size(0, 64) == 16
    assert moe.moe_layer_norm_workspace_size(4, 64) >= 2 * 64 * 4
    assert moe.moe_layer_norm_workspace_size(4, 10 ** 6) == 16


def test_linear(moe):
    f = moe.lib().moe_linear
    names = "x ldx w b r T K N act ot out pre st".split()
    good = dict(x=vp(GOOD), ldx=64, w=vp(GOOD), b=None, r=None, T=4, K=64, N=32, act=0, ot=1,
                out=vp(GOOD), pre=None, st=None)
    check(f, names, good, [
        (1, dict(T=-1)), (1, dict(K=0)), (1, dict(K=60)), (1, dict(N=0)), (1, dict(act=4)),
        (1, dict(act=-1)), (1, dict(act=3, N=33)), (1, dict(ot=2)), (1, dict(x=None)),
        (1, dict(w=None)), (1, dict(out=None)), (1, dict(x=vp(GOOD + 8))), (1, dict(w=vp(GOOD + 2))),
        (1, dict(ldx=68)), (1, dict(ldx=56)), (1, dict(out=vp(GOOD + 1))), (1, dict(b=vp(GOOD + 2))),
        (1, dict(pre=vp(GOOD + 1))), (1, dict(r=vp(GOOD + 1))), (0, dict(T=0, x=None)),
    ])


def test_linear_backward(moe):
    f = moe.lib().moe_linear_backward
    names = "d dt ldd x ldx w pre T K N act dz ldz dx dw wt acc db ws wsb st".split()
    good = dict(d=vp(GOOD), dt=1, ldd=32, x=vp(GOOD), ldx=64, w=vp(GOOD), pre=None, T=4, K=64, N=32,
                act=0, dz=None, ldz=0, dx=vp(GOOD), dw=vp(GOOD), wt=0, acc=0, db=None, ws=None, wsb=0,
                st=None)
    check(f, names, good, [
        (1, dict(K=12)), (1, dict(N=0)), (1, dict(act=3, N=31)), (1, dict(dt=2)), (1, dict(wt=2)),
        (1, dict(d=None)), (1, dict(ldd=31)), (1, dict(act=1, dz=vp(GOOD), ldz=32)),  # no preact
        (1, dict(dt=0)),                                       # fp32 needs d_preact
        (1, dict(ldd=33)),                                     # and so do rows off their boundary
        (1, dict(dt=0, dz=vp(GOOD), ldz=31)), (1, dict(dt=0, dz=vp(GOOD), ldz=36)),
        (1, dict(dt=0, dz=vp(GOOD + 2), ldz=32)), (1, dict(w=None)), (1, dict(x=None)),
        (1, dict(ldx=66)), (1, dict(db=vp(GOOD))), (1, dict(db=vp(GOOD), ws=vp(GOOD), wsb=8)),
        (1, dict(dw=vp(GOOD + 4))), (1, dict(dx=vp(GOOD + 2))),
    ])
    assert moe.moe_linear_backward_workspace_size(0, 5) == 16
    assert moe.moe_linear_backward_workspace_size(100, 32) >= 32 * 4


def test_adamw(moe):
    from sparse_moe_expert_gb300._lib import AdamWTensor
    f = moe.lib().moe_adamw_step

    def tensor(**over):
        a = dict(param=GOOD, grad=GOOD, master=None, exp_avg=GOOD, exp_avg_sq=GOOD,
                 exp_avg_scale=GOOD, exp_avg_sq_scale=GOOD, n=4, weight_decay=0.0)
        a.update(over)
        return AdamWTensor(**a)

    def call(tensors, pt=0, gt=0, bits=32, lr=1e-3, lr_dev=None, b1=0.9, b2=0.99, eps=1e-8, gs=None,
             step=GOOD, count=None):
        arr = (AdamWTensor * max(1, len(tensors)))(*tensors)
        return f(arr, len(tensors) if count is None else count, pt, gt, bits, lr, lr_dev, b1, b2, eps,
                 gs, vp(step) if step else None, None)
    for kw in (dict(pt=2), dict(gt=-1), dict(b1=1.0), dict(b1=-0.1), dict(b2=1.0), dict(eps=-1.0),
               dict(eps=float("inf")), dict(lr=float("nan")), dict(step=None), dict(step=GOOD + 2),
               dict(count=-1)):
        assert call([tensor()], **kw) == 1, kw
    assert call([tensor()], bits=4) == 2
    for over in (dict(param=None), dict(grad=None), dict(exp_avg=None), dict(exp_avg_sq=None),
                 dict(n=-1), dict(param=GOOD + 2), dict(weight_decay=float("nan")),
                 dict(exp_avg=GOOD + 1)):
        assert call([tensor(**over)]) == 1, over
    assert call([tensor(exp_avg_scale=None)], bits=8) == 1
    assert call([tensor(exp_avg_sq_scale=GOOD + 1)], bits=8) == 1
    assert call([tensor(master=GOOD)]) == 2                       # a master beside fp32
    assert call([tensor(master=GOOD), tensor(param=2 * GOOD)], pt=1) == 2  # for some only
    assert call([tensor(), tensor()]) == 1                        # the same tensor twice
    g = moe.lib().moe_adamw_values
    assert g((AdamWTensor * 1)(tensor()), 1, None, vp(GOOD), None) == 1
    assert g((AdamWTensor * 1)(tensor(n=0)), 1, None, None, None) == 0


def test_adamw_refuses_buffers_that_share_memory(moe):
    from sparse_moe_expert_gb300._lib import AdamWTensor
    f = moe.lib().moe_adamw_step
    MB = 1 << 20
    names = ["param", "grad", "master", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"]
    n = 1000
    size = dict(param=2 * n, grad=2 * n, master=4 * n, exp_avg=n, exp_avg_sq=n, exp_avg_scale=16,
                exp_avg_sq_scale=16)

    def tensors(count=3):
        return [dict({k: MB * (1 + i * 8 + j) for j, k in enumerate(names)}, n=n, weight_decay=0.0)
                for i in range(count)]

    def call(ts):  # bf16 params with masters, 8-bit states
        arr = (AdamWTensor * len(ts))(*[AdamWTensor(**t) for t in ts])
        return f(arr, len(ts), 1, 1, 8, 1e-3, None, 0.9, 0.99, 1e-8, None, vp(MB), None)
    for k in names:  # within a tensor: by its last bytes, by its first
        for other in names:
            if other == k:
                continue
            ts = tensors()
            ts[1][k] = ts[1][other] + (size[other] - 4)
            assert call(ts) == 1, (k, other)
    for k in names:
        if k == "grad":  # only read
            continue
        for i, j in ((0, 2), (2, 0)):
            ts = tensors()
            ts[i][k] = ts[j][k] + (size[k] - 4)
            assert call(ts) == 1, (k, i, j)
            ts = tensors()
            ts[i][k] = ts[j][k]
            assert call(ts) == 1, (k, i, j)


def test_optimizer_refuses_decay_of_unknown_names(moe):
    with pytest.raises(ValueError):
        moe.AdamW({"w": torch.zeros(4)}, weight_decay={"v": 0.1})


def test_python_calls_refuse_tensors_of_the_host(moe):
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(32, 64, dtype=torch.bfloat16)
    f = torch.zeros(4)
    for call in (lambda: moe.moe_layer_norm(x), lambda: moe.moe_linear(x, w),
                 lambda: moe.moe_layer_norm_backward(x, x, f, f),
                 lambda: moe.moe_linear_backward(x[:, :32], x, w),
                 lambda: moe.moe_adamw_step([f], [f], [f], [f], torch.zeros(2, dtype=torch.int32)),
                 lambda: moe.moe_adamw_values([f.to(torch.int8)], [f.to(torch.uint8)], [f], [f]),
                 lambda: moe.moe_adamw_step(f, [f], [f], [f], torch.zeros(2, dtype=torch.int32)),
                 lambda: moe.moe_linear(x, w, out_dtype=torch.float16),
                 lambda: moe.moe_layer_norm(x, out_dtype=torch.int32),
                 lambda: moe.moe_adamw_values([], [], [], [])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        moe.moe_linear("x", w)
