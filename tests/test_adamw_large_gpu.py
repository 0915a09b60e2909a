"""AdamW where a CTA takes several units of 2048 elements, of different tensors, against the
references and tolerances of test_adamw_gpu.py."""
import numpy as np
import pytest
import torch

from _parity import dev
from test_adamw_gpu import (B1, B16, B2, EPS, F32, LR, U, counter, decode, eight, encode, f, make, ref)

pytestmark = pytest.mark.gpu


def sizes(count, most):
    """From one element on, whole units among them; some 3 to 4 units each."""
    return [2048 if i % 9 == 0 else 1 + (i * 7919) % most for i in range(count)]


@pytest.mark.parametrize("param,masters,grad", [(F32, False, B16), (B16, True, F32), (B16, False, B16)])
def test_32_bit_states_of_many_units(param, masters, grad):
    import sparse_moe_expert_gb300 as m
    ns = sizes(400, 16000)
    assert sum(-(-n // 2048) for n in ns) > 1216  # eight CTAs of each of 152 SMs
    s = make(ns, param, grad, masters, seed=6)
    decay = [0.1 * (i % 3) for i in range(len(ns))]
    start = s["masters"] if masters else s["params"]
    want = [ref(start[i], s["grads"][i], s["m"][i], s["v"][i], 3, decay[i]) for i in range(len(ns))]
    step = counter(2)
    m.moe_adamw_step(s["params"], s["grads"], s["m"], s["v"], step, lr=LR, beta1=B1, beta2=B2, eps=EPS,
                     weight_decay=decay, masters=s.get("masters"))
    assert step.tolist() == [3, 0]
    for i, (w, mm, vv, size, move) in enumerate(want):
        got = (s["masters"] if masters else s["params"])[i].double().cpu()
        tol = 3 * U * w.abs() + 16 * U * move
        if param == B16 and not masters:
            tol = tol + 2.0 ** -8 * w.abs() + 2.0 ** -133
        assert bool(((got - w).abs() <= tol).all()), i
        if masters:
            assert torch.equal(s["params"][i], s["masters"][i].to(B16))
        assert bool(((s["m"][i].double().cpu() - mm).abs() <= 4 * U * size + 1e-45).all()), i
        assert bool(((s["v"][i].double().cpu() - vv).abs() <= 5 * U * vv + 1e-45).all()), i


@pytest.mark.parametrize("param,masters,grad,shift", [(F32, False, F32, 0), (B16, True, B16, 0),
                                                      (B16, False, F32, 1)])
def test_8_bit_states_of_many_units(param, masters, grad, shift):
    import sparse_moe_expert_gb300 as m
    ns = sizes(400, 16000)
    assert sum(-(-n // 2048) for n in ns) > 3 * 456  # three CTAs of each SM, three turns
    s = make(ns, param, grad, masters, seed=7, shift=shift)
    cm, sm, cv, sr = eight(s)
    start = [t.clone() for t in (s["masters"] if masters else s["params"])]
    old = [[t.clone() for t in c] for c in (cm, sm, cv, sr)]
    step = counter(40)
    m.moe_adamw_step(s["params"], s["grads"], cm, cv, step, lr=LR, beta1=B1, beta2=B2, eps=EPS,
                     weight_decay=0.1, masters=s.get("masters"), exp_avg_scales=sm, exp_avg_sq_scales=sr)
    flat_m, flat_v = m.moe_adamw_values(cm, cv, sm, sr)
    assert step.tolist() == [41, 0]
    at = 0
    for i, n in enumerate(ns):
        mm, rr = decode(*(c[i].cpu().numpy() for c in old))
        vv = rr * rr
        g = s["grads"][i].float().cpu().numpy()
        m1 = mm * f(B1) + g * f(1 - B1)
        v1 = vv * f(B2) + (g * g) * f(1 - B2)
        want = encode(m1, np.sqrt(v1), v1)
        for got, w in zip((cm, sm, cv, sr), want):
            assert np.array_equal(got[i].cpu().numpy(), w), (i, n)
        em, er = decode(*want)
        assert np.array_equal(flat_m[at:at + n].cpu().numpy(), em), i
        assert np.array_equal(flat_v[at:at + n].cpu().numpy(), er * er), i
        at += n
        w, _, _, _, move = ref(start[i], s["grads"][i], torch.from_numpy(mm), torch.from_numpy(vv), 41, 0.1)
        got = (s["masters"] if masters else s["params"])[i].double().cpu()
        tol = 3 * U * w.abs() + 16 * U * move
        if param == B16 and not masters:
            tol = tol + 2.0 ** -8 * w.abs() + 2.0 ** -133
        assert bool(((got - w).abs() <= tol).all()), i
    assert at == flat_m.numel()


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_of_many_tensors(bits):
    """Tables of a few tensors, of hundreds and of more than one launch holds."""
    import sparse_moe_expert_gb300 as m
    for count in (3, 60, 500):
        ns = sizes(count, 5000)
        sets = []
        for _ in range(2):
            s = make(ns, B16, B16, True, seed=8)
            states = eight(s) if bits == 8 else (s["m"], [], s["v"], [])
            sets.append((s, states, counter(0)))

        def go(s, c, step):
            kw = dict(exp_avg_scales=c[1], exp_avg_sq_scales=c[3]) if bits == 8 else {}
            m.moe_adamw_step(s["params"], s["grads"], c[0], c[2], step, lr=LR, weight_decay=0.1,
                             masters=s["masters"], **kw)
        for _ in range(3):
            go(*sets[0])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            go(*sets[1])
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        (a, ca, sa), (b, cb, sb) = sets
        assert sa.tolist() == sb.tolist() == [3, 0]
        for x, y in zip([*a["params"], *a["masters"], *(t for c in ca for t in c)],
                        [*b["params"], *b["masters"], *(t for c in cb for t in c)]):
            assert torch.equal(x, y)
