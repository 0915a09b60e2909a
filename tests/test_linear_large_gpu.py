"""The dense product and its gradient where pairs of CTAs take several tiles each, with
every epilogue, and the form for a few rows where a CTA takes several groups of columns,
against 64 bits.  Tolerances as in test_linear_gpu.py."""
import math

import pytest
import torch

from _parity import dev
from test_linear_gpu import BF16, B16, F32, NAMES, TOL, act64, close, inputs, rand

pytestmark = pytest.mark.gpu


def moe():
    import sparse_moe_expert_gb300 as m
    return m


# 4 and more tiles per pair, with whole 16-byte pieces of a row and without; 2; a long K
LARGE = [(6000, 136, 3088), (6000, 136, 3082), (5900, 72, 6160), (2300, 2056, 2064)]


@pytest.mark.parametrize("T,K,N", LARGE)
@pytest.mark.parametrize("act", NAMES)
@pytest.mark.parametrize("out_dtype", [B16, F32])
def test_forward_of_many_tiles(T, K, N, act, out_dtype):
    m = moe()
    x, w, b, r = inputs(T, K, N, act, True, out_dtype)
    z = x.double() @ w.double().t()
    zb = z + b.double()
    y, yb = act64(z, act), act64(zb, act)
    tol = 2 * TOL + (BF16 if out_dtype == B16 else 0)
    for bias, residual, keep in ((True, True, True), (True, False, False), (False, True, False),
                                 (False, False, False), (False, False, True)):
        out, pre = m.moe_linear(x, w, b if bias else None, residual=r if residual else None,
                                out_dtype=out_dtype, activation=NAMES.index(act), need_preact=keep)
        want = yb if bias else y
        close(out, want + r.double() if residual else want, tol, (bias, residual, keep))
        if keep:
            close(pre, zb if bias else z, TOL + BF16, "preact")
    again = r.clone()
    m.moe_linear(x, w, b, residual=again, out=again, activation=NAMES.index(act))
    first, _ = m.moe_linear(x, w, b, residual=r, activation=NAMES.index(act))
    assert torch.equal(again, first)
    assert m.moe_get_device_error() == 0


def test_many_tiles_are_exact_where_the_sums_are():
    """Whole numbers: sums, bias, residual and gradients are exact, so every entry is equal."""
    m = moe()
    g = torch.Generator(device="cuda").manual_seed(0)

    def whole(*shape):
        return torch.randint(-3, 4, shape, generator=g, device=dev())
    for T, K, N in ((6000, 136, 3088), (6000, 136, 3082), (5900, 72, 6160), (2300, 2056, 2064),
                    (6000, 3088, 136), (777, 4104, 1544), (4000, 2056, 3080), (4000, 2056, 3083)):
        x, w, b = whole(T, K).to(B16), whole(N, K).to(B16), whole(N).to(F32)
        sums = (x.double() @ w.double().t()).float()
        assert torch.equal(m.moe_linear(x, w, out_dtype=F32)[0], sums)
        assert torch.equal(m.moe_linear(x, w)[0], sums.to(B16))
        for dt in (F32, B16):
            r = whole(T, N).to(dt)
            assert torch.equal(m.moe_linear(x, w, b, residual=r)[0], (sums + b + r.float()).to(dt))
        d = whole(T, N).to(B16)
        start = whole(N, K).to(F32)
        dw = (d.double().t() @ x.double()).float()
        dx = (d.double() @ w.double()).float().to(B16)
        for dt in (F32, B16):
            more = start.to(dt, copy=True)  # the call adds to it
            got = m.moe_linear_backward(d, x, w, d_w=more, accumulate=True)
            assert torch.equal(got[0], dx) and torch.equal(more, (dw + start).to(dt))
            assert torch.equal(got[2], d.double().sum(0).float())
            got = m.moe_linear_backward(d, x, w, d_w_dtype=dt)
            assert torch.equal(got[0], dx) and torch.equal(got[1], dw.to(dt))
        assert torch.equal(m.moe_linear_backward(d, x, None, need_d_x=False)[1], dw)
        assert torch.equal(m.moe_linear_backward(d, x, w, need_d_w=False)[0], dx)


@pytest.mark.parametrize("T,K,N", [(6000, 136, 3088), (6000, 136, 3082), (2300, 2056, 2064), (777, 1032, 3088)])
@pytest.mark.parametrize("act", NAMES)
def test_backward_of_many_tiles(T, K, N, act):
    m = moe()
    cols = N // 2 if act == "swiglu" else N
    x, w, d = rand((T, K), 1), rand((N, K), 2, K ** -0.5), rand((T, cols), 3)
    pre = None if act == "none" else rand((T, N), 4, 1.5)
    z = (torch.zeros(T, N, device=dev()) if pre is None else pre).double().requires_grad_()
    d_z, = torch.autograd.grad(act64(z, act), z, d.double())
    dx, dw, db, dz = m.moe_linear_backward(d, x, w, pre, activation=NAMES.index(act))
    close(dz, d_z, BF16 + TOL, "d_preact")
    close(db, d_z.sum(0), TOL * max(1.0, float(d_z.abs().sum(0).norm() / d_z.sum(0).norm())), "d_bias")
    held = dz.double()
    close(dx, held @ w.double(), TOL + BF16, "d_x")
    close(dw, held.t() @ x.double(), TOL, "d_w")


@pytest.mark.parametrize("N", [3088, 3083])
def test_gelu_in_the_tail_and_of_values_that_are_not_ordinary(N):
    """As for the small tiles: 1.2e-5 of the value at |z| <= 9, limits past it."""
    m = moe()
    T = 6000
    x, w = torch.zeros(T, 8, dtype=B16), torch.zeros(N, 8, dtype=B16)
    x[:, 0] = torch.linspace(-9.0, 9.0, T).to(B16)
    special = torch.tensor([float("inf"), 1e38, 14.0, 0.0, -14.0, -1e38, float("nan")], dtype=B16)
    x[100:107, 0] = special
    w[:, 0] = 1.0
    out, pre = m.moe_linear(x.to(dev()), w.to(dev()), activation=m.ACT_GELU, out_dtype=F32, need_preact=True)
    out = out.cpu()
    z = x[:, 0].double()
    ordinary = torch.ones(T, dtype=torch.bool)
    ordinary[100:107] = False
    want = (z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0)))[ordinary][:, None]
    got = out[ordinary].double()
    assert float(((got - want).abs() - 1.2e-5 * want.abs()).max()) <= 1e-30
    assert bool((pre.cpu()[ordinary] == x[ordinary][:, :1]).all())
    for i in range(3):
        assert bool((out[100 + i] == float(special[i])).all()), i
    assert float(out[103].abs().max()) == 0.0 and float(out[104].abs().max()) < 1e-37
    assert float(out[105].abs().max()) == 0.0 and bool(torch.isnan(out[106]).all())


@pytest.mark.parametrize("T", [1, 3, 8, 11, 16, 20, 32])
@pytest.mark.parametrize("K,N", [(264, 5001), (2056, 5000), (1032, 10002)])
@pytest.mark.parametrize("act", NAMES)
def test_a_few_rows_with_more_columns_than_the_ctas_take_at_once(T, K, N, act):
    m = moe()
    N += N % 2
    if act == "swiglu" and K * N < 1 << 23:
        N *= 2
    for out_dtype, residual, bias, keep in ((B16, True, True, True), (F32, False, False, False)):
        x, w, b, r = inputs(T, K, N, act, residual, out_dtype)
        out, pre = m.moe_linear(x, w, b if bias else None, residual=r, out_dtype=out_dtype,
                                activation=NAMES.index(act), need_preact=keep)
        z = x.double() @ w.double().t()
        if bias:
            z = z + b.double()
        y = act64(z, act)
        close(out, y + r.double() if residual else y, 2 * TOL + (BF16 if out_dtype == B16 else 0), "out")
        if keep:
            close(pre, z, TOL + BF16, "preact")
    whole = [torch.randint(-3, 4, s).to(B16).to(dev()) for s in ((T, K), (N, K))]
    assert torch.equal(m.moe_linear(*whole, out_dtype=F32)[0], (whole[0].double() @ whole[1].double().t()).float())


def test_many_tiles_captured_and_on_streams_beside_smaller_products():
    """A replayed graph and calls on two streams, with other kernels in between, give the bits
    of a call alone; accumulation adds once per replay."""
    m = moe()
    shapes = [(2300, 136, 3088), (64, 1536, 512), (2300, 136, 1541 * 2), (20, 520, 5000)]
    data = [(rand((T, K), i), rand((N, K), 9 + i, K ** -0.5), rand((T, N // 2), 20 + i))
            for i, (T, K, N) in enumerate(shapes)]

    def step(stream=None, sums=None):
        out = []
        for i, (x, w, d) in enumerate(data):
            y, pre = m.moe_linear(x, w, activation=m.ACT_SWIGLU, need_preact=True, stream=stream)
            out += [y, pre, *m.moe_linear_backward(d, x, w, pre, activation=m.ACT_SWIGLU, stream=stream)]
            if sums is not None:
                m.moe_linear_backward(d, x, w, pre, activation=m.ACT_SWIGLU, d_w=sums[i], accumulate=True,
                                      stream=stream)
        return out
    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = [step(s) for s in streams * 5]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, want))
    once, sums = ([torch.zeros_like(w, dtype=F32) for _, w, _ in data] for _ in range(2))
    for _ in range(3):
        step(sums=once)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(sums=sums)
    assert not any(bool(s.any()) for s in sums)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(sums, once))
    assert m.moe_get_device_error() == 0


@pytest.mark.parametrize("T,N", [(12, 32), (100, 64), (6000, 3088), (6000, 3082)])
def test_silu_and_swiglu_keep_their_digits_in_the_tail(T, N):
    """z is exact (one product by one).  The hardware's exponential is 2 + 1.173 |z| ulp off, the
    sum 1/2, the quotient 2 ulp: (5 + 1.2 |z|) 2^-23 of the value; SwiGLU's product 2^-24 more."""
    m = moe()
    x, w = torch.zeros(T, 8, dtype=B16), torch.zeros(N, 8, dtype=B16)
    z = torch.linspace(-80.0, 80.0, T).to(B16)
    x[:, 0] = z
    x[:, 1] = 3.0
    w[:, 0] = 1.0
    zd = z.double()[:, None]
    silu = zd / (1.0 + torch.exp(-zd))
    out = m.moe_linear(x.to(dev()), w.to(dev()), activation=m.ACT_SILU, out_dtype=F32)[0].cpu().double()
    assert bool(((out - silu).abs() <= (5.0 + 1.2 * zd.abs()) * 2.0 ** -23 * silu.abs()).all())
    w[N // 2:, 0], w[N // 2:, 1] = 0.0, 1.0  # up: 3 everywhere
    out = m.moe_linear(x.to(dev()), w.to(dev()), activation=m.ACT_SWIGLU, out_dtype=F32)[0].cpu().double()
    assert out.shape == (T, N // 2)
    assert bool(((out - 3.0 * silu).abs() <= (5.5 + 1.2 * zd.abs()) * 2.0 ** -23 * 3.0 * silu.abs()).all())
