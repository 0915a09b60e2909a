"""AdamW over many tensors against the formula in 64 bits, and the 8-bit states
code by code against the formula with every operation rounded to fp32.

Tolerances (u = 2^-24): beta, 1 - beta and each operation are rounded once, so
m is 4 u of beta1 |m| + (1 - beta1) |g| off and v 5 u of v; the quotient adds
half of that, the correction factors and four operations (16 u in all, of the
magnitudes that m was summed from); w adds 3 u of |w|.
"""
import math

import numpy as np
import pytest
import torch

from _parity import dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, B16 = torch.float32, torch.bfloat16
LR, B1, B2, EPS = 3e-3, 0.9, 0.995, 1e-7


def moe():
    import sparse_moe_expert_gb300 as m
    return m


def counter(t):
    return torch.tensor([t, 0], dtype=torch.int32, device=dev())


def make(sizes, param=F32, grad=F32, masters=False, seed=0, shift=0):
    """Lists of tensors; shift > 0 moves each off its 16-byte boundary."""
    g = torch.Generator().manual_seed(seed)

    def one(n, dtype, scale=1.0, positive=False):
        t = torch.randn(n + shift, generator=g) * scale * torch.exp(torch.randn(n + shift, generator=g))
        return (t.square() if positive else t).to(dtype).to(dev())[shift:]
    s = dict(grads=[one(n, grad, 0.01) for n in sizes], m=[one(n, F32, 0.01) for n in sizes],
             v=[one(n, F32, 0.01, True) for n in sizes])
    if masters:
        s["masters"] = [one(n, F32) for n in sizes]
        s["params"] = [t.to(param).clone() for t in s["masters"]]
    else:
        s["params"] = [one(n, param) for n in sizes]
    return s


def ref(w, g, m, v, t, decay, scale=1.0):
    w, g, m, v = (a.double().cpu() for a in (w, g, m, v))
    g = g * scale
    size = B1 * m.abs() + (1 - B1) * g.abs()
    m, v = B1 * m + (1 - B1) * g, B2 * v + (1 - B2) * g * g
    den = torch.sqrt(v / (1 - B2 ** t)) + EPS
    new = w * (1 - LR * decay) - LR * (m / (1 - B1 ** t)) / den
    return new, m, v, size, LR * size / (1 - B1 ** t) / den


SIZES = [1, 7, 8, 255, 256, 257, 2047, 2048, 2049, 5000, 0, 70001]


@pytest.mark.parametrize("param,masters", [(F32, False), (B16, True), (B16, False)])
@pytest.mark.parametrize("grad", [F32, B16])
@pytest.mark.parametrize("shift", [0, 1])
def test_32_bit_states(param, masters, grad, shift):
    m = moe()
    s = make(SIZES, param, grad, masters, shift=shift)
    decay = [0.0 if i % 2 else 0.2 for i in range(len(SIZES))]
    start = s["masters"] if masters else s["params"]
    scale = torch.tensor([0.25], device=dev())
    want = [ref(start[i], s["grads"][i], s["m"][i], s["v"][i], 8, decay[i], 0.25)
            for i in range(len(SIZES))]
    step = counter(7)
    assert m.moe_adamw_step(s["params"], s["grads"], s["m"], s["v"], step, lr=LR, beta1=B1, beta2=B2,
                            eps=EPS, weight_decay=decay, masters=s.get("masters"),
                            grad_scale=scale) is None
    assert step.tolist() == [8, 0]
    for i, (w, mm, vv, size, move) in enumerate(want):
        got = (s["masters"] if masters else s["params"])[i].double().cpu()
        tol = 3 * U * w.abs() + 16 * U * move
        if param == B16 and not masters:
            tol = tol + 2.0 ** -8 * w.abs() + 2.0 ** -133
        assert bool(((got - w).abs() <= tol).all()), i
        if masters:
            assert torch.equal(s["params"][i], s["masters"][i].to(B16))
        assert bool(((s["m"][i].double().cpu() - mm).abs() <= 4 * U * size + 1e-45).all())
        assert bool(((s["v"][i].double().cpu() - vv).abs() <= 5 * U * vv + 1e-45).all())


def blocks(a):
    n = a.size
    return np.pad(a, (0, -n % 256)).reshape(-1, 256)


f = np.float32


def decode(cm, sm, cv, sr):
    """Values of the states, each operation rounded to fp32."""
    a = blocks(cm.astype(f)) * f(1.0 / 127.0)
    r = blocks(cv.astype(f)) * f(1.0 / 255.0)
    m, r = (a * np.abs(a)) * sm[:, None], (r * r) * sr[:, None]
    n = cm.size
    return m.reshape(-1)[:n], r.reshape(-1)[:n]


def encode(m, r, v):
    n = m.size
    M, R, V = blocks(m), blocks(r), blocks(v)
    out = []
    for x, top in ((np.abs(M), 127.0), (R, 255.0)):
        s = x.max(1)
        with np.errstate(divide="ignore", over="ignore"):
            inv = np.where(s > 0, f(1.0) / s, f(0.0)).astype(f)
        s = np.where(np.isinf(inv), f(0.0), s)
        inv = np.where(np.isinf(inv), f(0.0), inv)
        out.append((np.rint(np.sqrt(x * inv[:, None]) * f(top)), s))
    cm = (out[0][0] * np.where(M < 0, -1, 1)).astype(np.int8)
    cv = np.where((V > 0) & (out[1][0] < 1), 1, out[1][0]).astype(np.uint8)
    return cm.reshape(-1)[:n], out[0][1], cv.reshape(-1)[:n], out[1][1]


def eight(s):
    """8-bit states of the fp32 ones in s."""
    cols = [[], [], [], []]
    for m, v in zip(s["m"], s["v"]):
        v = v.cpu().numpy()
        for c, t in zip(cols, encode(m.cpu().numpy(), np.sqrt(v), v)):
            c.append(torch.from_numpy(np.ascontiguousarray(t)).to(dev()))
    return cols


@pytest.mark.parametrize("param,masters,grad", [(F32, False, F32), (B16, True, B16), (B16, False, F32)])
@pytest.mark.parametrize("shift", [0, 3])
def test_8_bit_states_code_by_code(param, masters, grad, shift):
    m = moe()
    s = make(SIZES, param, grad, masters, seed=2, shift=shift)
    cm, sm, cv, sr = eight(s)
    if shift:  # codes off their boundary as well
        cm = [torch.cat([t[:1], t])[1:] for t in cm]
        cv = [torch.cat([t[:1], t])[1:] for t in cv]
    start = [t.clone() for t in (s["masters"] if masters else s["params"])]
    old = [[t.clone() for t in c] for c in (cm, sm, cv, sr)]
    step = counter(40)
    m.moe_adamw_step(s["params"], s["grads"], cm, cv, step, lr=LR, beta1=B1, beta2=B2, eps=EPS,
                     weight_decay=0.1, masters=s.get("masters"), exp_avg_scales=sm,
                     exp_avg_sq_scales=sr)
    flat_m, flat_v = m.moe_adamw_values(cm, cv, sm, sr)
    at = 0
    for i, n in enumerate(SIZES):
        if n == 0:
            continue
        mm, rr = decode(*(c[i].cpu().numpy() for c in old))
        vv = rr * rr
        g = s["grads"][i].float().cpu().numpy()
        m1 = mm * f(B1) + g * f(1 - B1)
        v1 = vv * f(B2) + (g * g) * f(1 - B2)
        want = encode(m1, np.sqrt(v1), v1)
        for got, w in zip((cm, sm, cv, sr), want):
            assert np.array_equal(got[i].cpu().numpy(), w), (i, n)
        em, er = decode(*want)
        assert np.array_equal(flat_m[at:at + n].cpu().numpy(), em)
        assert np.array_equal(flat_v[at:at + n].cpu().numpy(), er * er)
        at += n
        w, _, _, _, move = ref(start[i], s["grads"][i], torch.from_numpy(mm), torch.from_numpy(vv), 41, 0.1)
        got = (s["masters"] if masters else s["params"])[i].double().cpu()
        tol = 3 * U * w.abs() + 16 * U * move
        if param == B16 and not masters:
            tol = tol + 2.0 ** -8 * w.abs() + 2.0 ** -133
        assert bool(((got - w).abs() <= tol).all()), i
    assert at == flat_m.numel()


def test_codes_keep_small_values_and_zeros():
    m = moe()
    n = 600
    g = torch.zeros(n, device=dev())
    g[0], g[1], g[300] = 1.0, 1e-6, 1e-30  # the last's square is zero in fp32
    p = torch.zeros(n, device=dev())
    cm, cv = torch.zeros(n, dtype=torch.int8, device=dev()), torch.zeros(n, dtype=torch.uint8, device=dev())
    sm, sr = torch.zeros(3, device=dev()), torch.zeros(3, device=dev())
    step = counter(0)
    m.moe_adamw_step([p], [g], [cm], [cv], step, lr=1.0, beta1=0.5, beta2=0.5, eps=1e-8,
                     exp_avg_scales=[sm], exp_avg_sq_scales=[sr])
    # the first step moves by the gradient's sign where the gradient is not lost
    assert abs(float(p[0]) + 1.0) < 1e-6 and abs(float(p[1]) + 1.0 / 1.01) < 1e-4
    assert not p[2:300].any() and torch.isfinite(p).all()
    assert int(cv[0]) == 255 and int(cv[1]) == 1 and not cv[2:300].any()
    assert int(cm[0]) == 127 and int(cm[1]) == 0
    assert float(sr[1]) == 0.0 and not cv[256:512].any() and float(sm[2]) == 0.0
    for _ in range(5):  # no gradient: nothing grows, nothing becomes NaN
        g.zero_()
        before = p.clone()
        m.moe_adamw_step([p], [g], [cm], [cv], step, lr=1.0, beta1=0.5, beta2=0.5, eps=1e-8,
                         exp_avg_scales=[sm], exp_avg_sq_scales=[sr])
        assert torch.isfinite(p).all() and float((p - before).abs().max()) <= 1.0
    assert step.tolist() == [6, 0]


def test_not_finite_gradients():
    m = moe()
    for bad in (float("nan"), float("inf")):
        n = 520
        g = torch.full((n,), 0.1, device=dev())
        g[3] = bad
        p = torch.ones(n, device=dev())
        cm, cv = torch.zeros(n, dtype=torch.int8, device=dev()), torch.zeros(n, dtype=torch.uint8, device=dev())
        sm, sr = torch.zeros(3, device=dev()), torch.zeros(3, device=dev())
        m.moe_adamw_step([p], [g], [cm], [cv], counter(0), exp_avg_scales=[sm], exp_avg_sq_scales=[sr])
        a, b = m.moe_adamw_values([cm], [cv], [sm], [sr])
        assert torch.isnan(a[:256]).all() and torch.isnan(b[:256]).all()  # the block says so
        assert torch.isfinite(a[256:]).all() and torch.isfinite(b[256:]).all()
        assert torch.isnan(p[3]) and torch.isfinite(p[4:]).all()


def test_scale_that_is_not_finite_skips_the_step():
    m = moe()
    for bits in (32, 8):
        s = make([300, 5000])
        states = eight(s) if bits == 8 else None
        keep = [t.clone() for t in s["params"] + s["m"] + s["v"]]
        for bad in (float("inf"), float("nan")):
            step = counter(5)
            scale = torch.tensor([bad], device=dev())
            if bits == 8:
                kept = [[t.clone() for t in c] for c in states]
                m.moe_adamw_step(s["params"], s["grads"], states[0], states[2], step,
                                 exp_avg_scales=states[1], exp_avg_sq_scales=states[3], grad_scale=scale)
                assert all(torch.equal(a, b) for x, y in zip(states, kept) for a, b in zip(x, y))
            else:
                m.moe_adamw_step(s["params"], s["grads"], s["m"], s["v"], step, grad_scale=scale)
            assert step.tolist() == [5, 0]
            assert all(torch.equal(a, b) for a, b in zip(keep, s["params"] + s["m"] + s["v"]))


def test_more_tensors_than_a_table_holds():
    m = moe()
    sizes = [1 + (i * 37) % 900 for i in range(1000)]
    s = make(sizes)
    want = [ref(*(s[k][i] for k in ("params", "grads", "m", "v")), 1, 0.0) for i in range(len(sizes))]
    step = counter(0)
    m.moe_adamw_step(s["params"], s["grads"], s["m"], s["v"], step, lr=LR, beta1=B1, beta2=B2, eps=EPS)
    assert step.tolist() == [1, 0]
    for i, (w, _, _, _, move) in enumerate(want):
        assert bool(((s["params"][i].double().cpu() - w).abs() <= 3 * U * w.abs() + 16 * U * move).all())
    m.moe_adamw_step([], [], [], [], step)
    assert step.tolist() == [2, 0]


def test_late_steps_and_large_counts():
    m = moe()
    for t in (0, 1, 999, 10 ** 6, 2 ** 31 - 3):
        s = make([777], seed=3)
        want = ref(s["params"][0], s["grads"][0], s["m"][0], s["v"][0], t + 1, 0.0)
        step = counter(t)
        m.moe_adamw_step(s["params"], s["grads"], s["m"], s["v"], step, lr=LR, beta1=B1, beta2=B2, eps=EPS)
        w, move = want[0], want[4]
        assert bool(((s["params"][0].double().cpu() - w).abs() <= 3 * U * w.abs() + 16 * U * move).all())
        assert step.tolist() == [t + 1, 0]


def test_captured_step_counts_and_follows_the_schedule():
    m = moe()
    a, b = make([5000, 33], seed=4), make([5000, 33], seed=4)
    lr = torch.tensor([1e-2], device=dev())
    step, other = counter(0), counter(0)

    def go(s, c):
        m.moe_adamw_step(s["params"], s["grads"], s["m"], s["v"], c, lr=lr, weight_decay=0.1)
    for i in range(4):
        lr.fill_(1e-2 / (i + 1))
        go(b, other)
    graph = torch.cuda.CUDAGraph()
    lr.fill_(0.0)
    with torch.cuda.graph(graph):
        go(a, step)
    assert step.tolist() == [0, 0]
    for i in range(4):
        lr.fill_(1e-2 / (i + 1))
        graph.replay()
    torch.cuda.synchronize()
    assert step.tolist() == [4, 0]
    for k in ("params", "m", "v"):
        assert all(torch.equal(x, y) for x, y in zip(a[k], b[k]))


def test_refusals():
    m = moe()
    s = make([300, 40])
    step = counter(0)
    args = [s["params"], s["grads"], s["m"], s["v"], step]

    def bad(exc, over=None, **kw):
        a = list(args)
        for i, v in (over or {}).items():
            a[i] = v
        with pytest.raises(exc):
            m.moe_adamw_step(*a, **kw)
    bad(ValueError, {1: s["grads"][:1]})
    bad(ValueError, {1: [s["grads"][1], s["grads"][0]]})
    bad(ValueError, {0: [s["params"][0].half(), s["params"][1]]})
    bad(ValueError, {1: [s["grads"][0].to(B16), s["grads"][1]]})
    bad(ValueError, {0: s["params"][0]})
    bad(ValueError, {2: [t.to(B16) for t in s["m"]]})
    bad(ValueError, {2: [t.to(torch.int8) for t in s["m"]]})
    bad(ValueError, {4: step[:1]})
    bad(ValueError, {4: step.long()})
    bad(ValueError, {4: step.cpu()})
    bad(ValueError, {0: [torch.zeros(600, device=dev())[::2], s["params"][1]]})
    bad(ValueError, weight_decay=[0.1])
    bad(ValueError, grad_scale=torch.ones(2, device=dev()))
    bad(ValueError, masters=s["params"][:1])
    bad(m.MoEError, masters=[t.clone() for t in s["params"]])   # beside fp32 params
    bad(m.MoEError, {0: [s["params"][0]] * 2, 1: [s["grads"][0]] * 2, 2: [s["m"][0]] * 2,
                     3: [s["v"][0]] * 2})
    for kw in (dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0), dict(lr=float("nan")),
               dict(weight_decay=float("inf"))):
        bad(m.MoEError, **kw)
    assert step.tolist() == [0, 0]
    assert math.isfinite(float(s["params"][0].sum()))
