"""The 8-bit second moments' codes where values come near the smallest that fp32 holds."""
import numpy as np
import pytest
import torch

from _parity import dev
from test_adamw_gpu import counter, encode, f

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shift", [0, 1])
def test_codes_of_blocks_with_subnormal_second_moments(shift):
    """From states of zero one step makes v = (1 - beta2) g^2: its largest value of a
    block runs from 2^-104 to 2^-92, the others down to zero.  The codes are those of the
    formula with every operation rounded to fp32."""
    import sparse_moe_expert_gb300 as m
    b1, b2 = 0.9, 0.5
    rng = np.random.default_rng(5)
    tops = np.repeat(np.arange(-104.0, -91.75, 0.25), 8)
    low = rng.uniform(-150.0, tops[:, None], (len(tops), 256))
    low[:, 0] = tops
    low[:, 1:40] = rng.uniform(-127.5, -125.5, (len(tops), 39))  # around the last normal values
    g = np.exp2((np.concatenate([row[rng.permutation(256)] for row in low]) + 1.0) / 2.0).astype(f)
    n = g.size
    v = (g * g) * f(1 - b2)
    mm = g * f(1 - b1)
    want = encode(mm, np.sqrt(v), v)
    assert (want[2][(v > 0) & (v < 2.0 ** -126)] > 1).any()  # such values have codes of their own

    def make(a):
        return torch.cat([torch.zeros(shift, dtype=a.dtype), a]).to(dev())[shift:]
    p, grad = make(torch.zeros(n)), make(torch.from_numpy(g))
    cm, cv = make(torch.zeros(n, dtype=torch.int8)), make(torch.zeros(n, dtype=torch.uint8))
    sm, sr = torch.zeros(n // 256, device=dev()), torch.zeros(n // 256, device=dev())
    m.moe_adamw_step([p], [grad], [cm], [cv], counter(0), beta1=b1, beta2=b2, exp_avg_scales=[sm],
                     exp_avg_sq_scales=[sr])
    for got, w, what in zip((cm, sm, cv, sr), want, ("m", "m's scale", "v", "v's scale")):
        got = got.cpu().numpy()
        assert np.array_equal(got, w), (what, int((got != w).sum()))


@pytest.mark.parametrize("eps", [1e-10, 2e-11, 1e-12, 1e-14, 1e-16])
@pytest.mark.parametrize("b2", [0.5, 0.999, 0.99999])
def test_steps_of_subnormal_second_moments_beside_a_small_eps(eps, b2):
    """m is one product (1 u), its correction another; the divisor's terms are 2^-23 of eps
    and 6 u of the root off: 16 u of the move, with v as fp32 holds it."""
    import sparse_moe_expert_gb300 as m
    n, lr, b1 = 2000, 0.5, 0.9
    g = torch.Generator().manual_seed(3)
    p, grad = torch.zeros(n, device=dev()), torch.zeros(n, device=dev())
    avg = (torch.randn(n, generator=g) * eps).to(dev())
    sq = torch.exp2(-132.0 + 12.0 * torch.rand(n, generator=g)).to(dev())
    first = avg.double()
    m.moe_adamw_step([p], [grad], [avg], [sq], counter(0), lr=lr, beta1=b1, beta2=b2, eps=eps)
    want = -lr * (b1 * first / (1 - b1)) / (torch.sqrt(sq.double() / (1 - b2)) + eps)
    assert bool(((p.double() - want).abs() <= 16 * 2.0 ** -24 * want.abs()).all())


def test_gradients_may_overlap_each_other():
    import sparse_moe_expert_gb300 as m
    flat = torch.randn(3000, device=dev())
    grads = [flat[i:i + 1000] for i in (1000, 0, 500, 1000, 2000)]
    sets = []
    for gs in (grads, [g.clone() for g in grads]):
        p, a, b = ([torch.zeros(1000, device=dev()) for _ in grads] for _ in range(3))
        m.moe_adamw_step(p, gs, a, b, counter(0))
        sets.append(p + a + b)
    assert all(torch.equal(x, y) for x, y in zip(*sets))
    params = [flat[2000:]] + [torch.zeros(1000, device=dev()) for _ in range(4)]
    with pytest.raises(m.MoEError):  # the last tensor's gradient
        m.moe_adamw_step(params, grads, a, b, counter(0))


@pytest.mark.parametrize("bits", [32, 8])
def test_refused_gradients_leave_every_tensor_as_it_was(bits):
    """The fp32 and the bf16 tensors are a launch each; neither runs if one is refused."""
    import sparse_moe_expert_gb300 as m

    def normal(n, dtype=torch.float32):
        return torch.randn(n, device=dev()).to(dtype)
    B16 = torch.bfloat16
    p = {"a": normal(300), "b": normal(77, B16), "c": normal(1000, B16)}
    opt = m.AdamW(p, lr=0.1, state_bits=bits)
    good = {n: normal(t.numel()) for n, t in p.items()}
    opt.step(good)
    keep = {n: t.clone() for n, t in p.items()}
    states = {n: {k: t.clone() for k, t in s.items()} for n, s in opt.state_dict().items()}
    for wrong in (dict(b=normal(76)), dict(c=normal(1000, B16)), dict(c=normal(2000)[::2]), dict(b=normal(77).cpu()),
                  dict(b=normal(77).half(), c=normal(1000).half()), dict(b=None), dict(a=normal(299)),
                  dict(a=normal(300).half())):
        with pytest.raises(ValueError):
            opt.step(dict(good, **wrong))
    assert all(torch.equal(t, keep[n]) for n, t in p.items())
    for n, s in opt.state_dict().items():
        assert all(torch.equal(t, states[n][k]) for k, t in s.items())
    opt.step(good)
    assert all(int(s["step"][0]) == 2 for s in opt.state_dict().values())
    assert not any(torch.equal(t, keep[n]) for n, t in p.items())
