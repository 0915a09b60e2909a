"""The dense product with its epilogue, and its gradient, against 64 bits.

Tolerances (u = 2^-24): the tensor cores add at most K / 16 steps of 16
products, each step cut to fp32: 2 u of the running sum per step, so K / 8 u of
the sum of magnitudes, which is sqrt(pi K / 2) .. of random factors the result's
size times that at worst; summed in 8 runs or more and with errors of either
sign it stays below K^(1/2) u of the result: 4e-6 for K <= 4096, and 1e-5 is asked
of fp32 results in the 2-norm for every K here.  Activations add 1e-6 of their
input's size.  bf16 results add one rounding, 2^-8 of the value.
"""
import math

import numpy as np
import pytest
import torch

from _parity import dev

pytestmark = pytest.mark.gpu

TOL, BF16 = 1e-5, 2.0 ** -8
F32, B16 = torch.float32, torch.bfloat16
NAMES = ("none", "silu", "gelu", "swiglu")


def moe():
    import sparse_moe_expert_gb300 as m
    return m


def rand(shape, seed, scale=1.0, dtype=B16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).to(dev())


def act64(z, act):
    if act == "silu":
        return torch.nn.functional.silu(z)
    if act == "gelu":
        return torch.nn.functional.gelu(z)
    if act == "swiglu":
        g, u = z.chunk(2, dim=1)
        return torch.nn.functional.silu(g) * u
    return z


def close(got, want, tol, name=""):
    got, want = got.double(), want.double()
    assert got.shape == want.shape and torch.isfinite(got).all(), name
    err, size = float((got - want).norm()), float(want.norm())
    assert err <= tol * size + 1e-30, (name, err / size if size else err)
    # and nowhere far off: a value that is missing is of the values' own size
    if want.numel():
        rms = size / math.sqrt(want.numel())
        worst = float(((got - want).abs() / (want.abs() + rms)).max())
        assert worst <= max(tol * 8, 2e-4), (name, worst)


def inputs(T, K, N, act, residual, out_dtype, seed=0):
    cols = N // 2 if act == "swiglu" else N
    x, w = rand((T, K), seed + 1), rand((N, K), seed + 2, K ** -0.5)
    b = rand((N,), seed + 3, 0.3, F32)
    return x, w, b, rand((T, cols), seed + 4, 1.0, out_dtype) if residual else None


SIZES = [(1, 8, 1), (1, 64, 16), (1, 4096, 40), (2, 136, 17), (3, 2000, 300), (8, 512, 129),
         (9, 256, 64), (16, 1024, 33), (17, 320, 200), (31, 72, 515), (32, 4096, 128),
         (33, 64, 64), (40, 1000, 77), (64, 1536, 512), (127, 128, 130), (128, 2048, 96),
         (129, 520, 384), (300, 4096, 1000), (777, 264, 1234), (1000, 96, 2050),
         (1300, 1032, 2052)]


@pytest.mark.parametrize("T,K,N", SIZES)
@pytest.mark.parametrize("act", NAMES)
def test_forward(T, K, N, act):
    m = moe()
    if act == "swiglu":
        N += N % 2
    for out_dtype, residual, bias in ((B16, True, True), (F32, False, True), (F32, True, False)):
        x, w, b, r = inputs(T, K, N, act, residual, out_dtype)
        out, pre = m.moe_linear(x, w, b if bias else None, residual=r, out_dtype=out_dtype,
                                activation=NAMES.index(act), need_preact=act != "none")
        z = x.double() @ w.double().t()
        if bias:
            z = z + b.double()
        y = act64(z, act)
        if residual:
            y = y + r.double()
        close(out, y, 2 * TOL + (BF16 if out_dtype == B16 else 0), "out")
        if pre is not None:
            close(pre, z, TOL + BF16, "preact")
        else:
            assert act == "none"


def test_selected_entries_are_exact():
    """Whole numbers: every sum is exact, so every entry has to be equal."""
    m = moe()
    g = torch.Generator().manual_seed(0)
    for T, K, N in ((5, 136, 33), (40, 200, 100), (200, 1032, 333), (513, 4104, 700), (1500, 1032, 2104)):
        x = torch.randint(-3, 4, (T, K), generator=g).to(B16).to(dev())
        w = torch.randint(-3, 4, (N, K), generator=g).to(B16).to(dev())
        want = (x.double() @ w.double().t()).float()
        got = m.moe_linear(x, w, out_dtype=F32)[0]
        assert torch.equal(got, want), (T, K, N, int((got != want).sum()))
        d = torch.randint(-3, 4, (T, N), generator=g).to(B16).to(dev())
        dx, dw, db, dz = m.moe_linear_backward(d, x, w)
        assert torch.equal(dz, d)
        assert torch.equal(dw, (d.double().t() @ x.double()).float()), (T, K, N)
        assert torch.equal(dx, (d.double() @ w.double()).float().to(B16)), (T, K, N)
        assert torch.equal(db, d.double().sum(0).float())


def test_strides_in_place_and_memory_around():
    m = moe()
    for T in (5, 70, 300):
        K, N = 192, 136
        big = rand((T, K + 64), 1)
        x, w = big[:, 8:8 + K], rand((N, K), 2, K ** -0.5)
        r = rand((T, N), 3)
        want = m.moe_linear(x.contiguous(), w, residual=r)[0]
        assert torch.equal(m.moe_linear(x, w, residual=r)[0], want)
        # rows behind the last stay as they were
        buf = torch.full((T + 40, N), 7.0, dtype=B16, device=dev())
        buf[:T] = r
        got = m.moe_linear(x, w, residual=buf[:T], out=buf[:T])[0]
        assert got.data_ptr() == buf.data_ptr() and torch.equal(buf[:T], want)
        assert bool((buf[T:] == 7.0).all())
        # an output off its 16-byte boundary
        flat = torch.full((T * N + 9,), 7.0, dtype=B16, device=dev())
        out = flat[1:1 + T * N].view(T, N)
        m.moe_linear(x, w, residual=r, out=out)
        assert torch.equal(out, want) and float(flat[0]) == 7.0 and bool((flat[1 + T * N:] == 7.0).all())
    assert m.moe_linear(big[:0, :192], w)[0].shape == (0, 136)


def test_infinities_and_nan_stay_in_their_rows():
    m = moe()
    for T in (4, 100):
        x, w = rand((T, 256), 1), rand((96, 256), 2)
        x[1, 3], x[2, 5] = float("nan"), float("inf")
        out = m.moe_linear(x, w, out_dtype=F32)[0]
        assert torch.isnan(out[1]).all() and not torch.isfinite(out[2]).any()
        assert torch.isfinite(out[0]).all() and torch.isfinite(out[3:]).all()
        w[7] = float("nan")
        out = m.moe_linear(x[3:].contiguous() if T > 4 else x[3:], w, out_dtype=F32)[0]
        assert torch.isnan(out[:, 7]).all()
        keep = [i for i in range(96) if i != 7]
        assert torch.isfinite(out[:, keep]).all()
    # SwiGLU: a column's halves and no others
    x, w = rand((50, 128), 3), rand((200, 128), 4)
    w[100 + 9] = float("nan")
    out = m.moe_linear(x, w, activation=m.ACT_SWIGLU)[0]
    assert torch.isnan(out[:, 9]).all()
    assert torch.isfinite(out[:, [i for i in range(100) if i != 9]]).all()


GRAD_SIZES = [(1, 64, 40), (1, 4096, 17), (3, 136, 300), (7, 8, 8), (33, 256, 129), (64, 1536, 200),
              (129, 72, 515), (300, 520, 1000), (777, 1024, 130),
              (1300, 1032, 2052)]


@pytest.mark.parametrize("T,K,N", GRAD_SIZES)
@pytest.mark.parametrize("act", NAMES)
@pytest.mark.parametrize("d_dtype", [B16, F32])
def test_backward(T, K, N, act, d_dtype):
    m = moe()
    if act == "swiglu":
        N += N % 2
    cols = N // 2 if act == "swiglu" else N
    x, w = rand((T, K), 1), rand((N, K), 2, K ** -0.5)
    d = rand((T, cols), 3, 1.0, d_dtype)
    pre = None if act == "none" else rand((T, N), 4, 1.5)
    z = (torch.zeros(T, N, dtype=torch.float64, device=dev()) if pre is None else pre.double())
    z.requires_grad_()
    d_z, = torch.autograd.grad(act64(z, act), z, d.double())
    dx, dw, db, dz = m.moe_linear_backward(d, x, w, pre, activation=NAMES.index(act))
    assert dz.dtype == B16 and dw.dtype == db.dtype == F32 and dx.dtype == B16
    close(dz, d_z, BF16 + TOL, "d_preact")
    # sums of T terms that are 4 u off (a few more for the slope), in runs: T u at worst
    close(db, d_z.sum(0), TOL * max(1.0, float(d_z.abs().sum(0).norm() / d_z.sum(0).norm())), "d_bias")
    held = dz.double()
    close(dx, held @ w.double(), TOL + BF16, "d_x")
    close(dw, held.t() @ x.double(), TOL, "d_w")
    # into what is there, in either type
    more = torch.ones(N, K, device=dev())
    m.moe_linear_backward(d, x, w, pre, activation=NAMES.index(act), d_w=more, accumulate=True,
                          need_d_x=False, need_d_bias=False)
    close(more, held.t() @ x.double() + 1.0, TOL, "accumulated")
    half = m.moe_linear_backward(d, x, w, pre, activation=NAMES.index(act), d_w_dtype=B16,
                                 need_d_x=False, need_d_bias=False)
    assert half[0] is None and half[2] is None and half[1].dtype == B16
    close(half[1], held.t() @ x.double(), TOL + BF16, "d_w bf16")


@pytest.mark.parametrize("act", NAMES)
def test_backward_is_the_derivative(act):
    """Against central differences in 64 bits of sum(d_out * out) for the
    pre-activations that were kept (step 1e-5: 1e-9 of truncation)."""
    m = moe()
    T, K, N = 5, 64, 24
    cols = N // 2 if act == "swiglu" else N
    x, w, b = rand((T, K), 1), rand((N, K), 2, K ** -0.5), rand((N,), 3, 0.2, F32)
    d = rand((T, cols), 4)
    pre = m.moe_linear(x, w, b, activation=NAMES.index(act), need_preact=True)[1]
    dx, dw, db, _ = m.moe_linear_backward(d, x, w, pre, activation=NAMES.index(act))
    X, W, Bb, D = (t.double().cpu() for t in (x, w, b, d))

    def f():
        return float((act64(X @ W.t() + Bb, act) * D).sum())
    rng = np.random.default_rng(1)
    for t, got in ((X, dx), (W, dw), (Bb, db)):
        size = float(got.double().norm()) / math.sqrt(got.numel())
        for _ in range(10):
            i = tuple(int(rng.integers(n)) for n in t.shape)
            keep = float(t[i])
            t[i] = keep + 1e-5
            hi = f()
            t[i] = keep - 1e-5
            lo = f()
            t[i] = keep
            # d_z and z are held in bf16: each term 2^-8 off, and its slope 2^-8 |z| off
            assert abs((hi - lo) / 2e-5 - float(got[i])) <= 0.03 * (abs(float(got[i])) + size)


def test_empty_batch_and_strided_gradients():
    m = moe()
    x, w = rand((20, 64), 1), rand((24, 64), 2)
    dx, dw, db, dz = m.moe_linear_backward(rand((20, 24), 3)[:0], x[:0], w)
    assert dx.shape == (0, 64) and not dw.any() and not db.any() and dz.shape == (0, 24)
    kept = torch.ones(24, 64, device=dev())
    m.moe_linear_backward(rand((20, 24), 3)[:0], x[:0], w, d_w=kept, accumulate=True)
    assert bool((kept == 1).all())
    for pad in (8, 3):  # rows that a tensor map can describe, and rows that it cannot
        d = rand((20, 24 + pad), 4)[:, :24]
        a = m.moe_linear_backward(d, x, w)
        b = m.moe_linear_backward(d.contiguous(), x, w)
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_captured_on_two_streams_and_repeated():
    m = moe()
    shapes = [(4, 512, 256), (90, 512, 256), (600, 512, 256)]
    data = [(rand((T, K), 1), rand((N, K), 2, K ** -0.5), rand((T, N), 3)) for T, K, N in shapes]

    def step(stream=None):
        out = []
        for x, w, d in data:
            y, pre = m.moe_linear(x, w, activation=m.ACT_GELU, need_preact=True, stream=stream)
            out += [y, pre, *m.moe_linear_backward(d, x, w, pre, activation=m.ACT_GELU, stream=stream)]
        return out
    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = [step(s) for s in streams * 6]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, want))
    assert m.moe_get_device_error() == 0


def test_refusals():
    m = moe()
    x, w = rand((6, 64), 1), rand((32, 64), 2)
    b = rand((32,), 3, 1.0, F32)
    for args, kw in [((x.float(), w), {}), ((x, w.float()), {}), ((x, w[:, :56]), {}), ((x, w, b[:31]), {}),
                     ((x, w, b.to(B16)), {}), ((x, w.t().contiguous().t()), {}),
                     ((rand((6, 68), 1)[:, :64], w), {}), ((rand((6, 80), 1)[:, 4:68], w), {}),
                     ((x, w), dict(residual=rand((6, 31), 4))),
                     ((x, w), dict(residual=rand((6, 32), 4), out_dtype=F32)),
                     ((x, w), dict(out=torch.empty(6, 16, dtype=B16, device=dev()))),
                     ((x, w), dict(out_dtype=torch.float16)), ((x.cpu(), w), {}),
                     ((x, w), dict(out=w[:6, :32])), ((x, w), dict(preact=x))]:
        with pytest.raises(ValueError):
            m.moe_linear(*args, **kw)
    for args, kw in [((rand((6, 60), 1).contiguous(), rand((32, 60), 1)), {})]:
        with pytest.raises((ValueError, m.MoEError)):
            m.moe_linear(*args, **kw)
    with pytest.raises(m.MoEError):
        m.moe_linear(x, rand((33, 64), 2), activation=m.ACT_SWIGLU)
    with pytest.raises(m.MoEError):
        m.moe_linear(x, w, activation=4)
    d = rand((6, 32), 5)
    for args, kw in [((d[:5], x, w), {}), ((d, x, w), dict(activation=m.ACT_SILU)),
                     ((d, x, w), dict(accumulate=True)), ((d, x, w), dict(d_x=x)),
                     ((d, x, w), dict(d_w=w)), ((d, x, w[:31]), {}), ((d.half(), x, w), {}),
                     ((d, x, w), dict(d_w_dtype=torch.float16))]:
        with pytest.raises(ValueError):
            m.moe_linear_backward(*args, **kw)
    with pytest.raises(m.MoEError):
        m.moe_linear_backward(d, x, w, workspace=torch.empty(16, dtype=torch.uint8, device=dev()))


@pytest.mark.parametrize("T,N", [(12, 24), (100, 64), (300, 4096), (300, 1001)])
def test_gelu_keeps_its_digits_in_the_tail(T, N):
    """z is exact (one product by one).  The tail is 1.2e-6 of itself off, e^(-z^2/2) z^2 2^-23
    and 2 ulp, so 1.2e-5 at |z| = 9; the slope's terms as much of themselves, below 1e-6 in
    all, and a rounding to bf16."""
    m = moe()
    z = torch.linspace(-9.0, 9.0, T).to(B16)
    x = torch.zeros(T, 8, dtype=B16)
    x[:, 0] = z
    w = torch.zeros(N, 8, dtype=B16)
    w[:, 0] = 1.0
    x, w = x.to(dev()), w.to(dev())
    out, pre = m.moe_linear(x, w, activation=m.ACT_GELU, out_dtype=F32, need_preact=True)
    zd = z.double()
    tail = 0.5 * torch.special.erfc(-zd / math.sqrt(2.0))
    want = (zd * tail)[:, None].expand(T, N)
    got = out.double().cpu()
    assert float(((got - want).abs() - 1.2e-5 * want.abs()).max()) <= 1e-30
    assert torch.equal(pre.cpu(), z[:, None].expand(T, N))
    d = torch.ones(T, N, dtype=B16, device=dev())
    dz = m.moe_linear_backward(d, x, w, pre, activation=m.ACT_GELU, need_d_x=False, need_d_w=False)[3]
    slope = tail + zd * torch.exp(-0.5 * zd * zd) / math.sqrt(2.0 * math.pi)
    err = (dz.double().cpu() - slope[:, None]).abs()
    assert float((err - BF16 * slope.abs()[:, None]).max()) <= 1e-6


def test_gelu_of_values_that_are_not_ordinary():
    m = moe()
    z = torch.tensor([float("inf"), 1e38, 1e20, 14.0, 0.0, -14.0, -1e20, -1e38, float("nan")], dtype=B16)
    for T, N in ((9, 16), (9 * 20, 512)):
        x = torch.zeros(T, 8, dtype=B16)
        x[:, 0] = z.repeat(T // 9)
        w = torch.zeros(N, 8, dtype=B16)
        w[:, 0] = 1.0
        out = m.moe_linear(x.to(dev()), w.to(dev()), activation=m.ACT_GELU, out_dtype=F32)[0].cpu()
        # the other seven products of a sum are 0 x 0
        for i in range(4):
            assert torch.equal(out[i::9], x[i::9, :1].float().expand(T // 9, N)), i
        assert float(out[4::9].abs().max()) == 0.0
        assert float(out[5::9].abs().max()) < 1e-37 and float(out[6::9].abs().max()) == 0.0
        assert float(out[7::9].abs().max()) == 0.0 and bool(torch.isnan(out[8::9]).all())


@pytest.mark.parametrize("T,K,N", [(1, 8, 1), (1, 216, 4770), (2, 264, 77), (3, 2048, 1536), (4, 1032, 999),
                                   (5, 4096, 2048), (8, 2056, 4097), (9, 2056, 4097), (7, 2048, 1536)])
def test_d_w_of_a_few_rows(T, K, N):
    """At most 9 products summed: 9 u of their magnitudes, below TOL; the same bits again;
    rows of x and d_out of any stride; values that are not finite stay in their columns."""
    m = moe()
    g = torch.Generator().manual_seed(T * 7 + K)
    x = torch.randn(T, K + 24, generator=g).to(B16).to(dev())[:, :K]
    w = torch.randn(N, K, generator=g).to(B16).to(dev())
    d = torch.randn(T, N + 5, generator=g).to(B16).to(dev())[:, :N]
    want = d.double().t() @ x.double()
    size = float((d.double().abs().t() @ x.double().abs()).norm())
    for dt, tol in ((F32, TOL), (B16, TOL + BF16)):
        _, dw, db, _ = m.moe_linear_backward(d, x, w, d_w_dtype=dt)
        assert dw.dtype == dt and float((dw.double() - want).norm()) <= tol * size
        again = m.moe_linear_backward(d, x, w, d_w_dtype=dt, need_d_x=False)[1]
        assert torch.equal(again, dw)
        start = torch.randn(N, K, generator=g).to(dt).to(dev())
        more = start.clone()
        m.moe_linear_backward(d, x, None, d_w=more, accumulate=True, need_d_x=False, need_d_bias=False)
        close(more, want + start.double(), tol * max(1.0, size / float((want + start.double()).norm())),
              "accumulated")
    x2, d2 = x.clone(), d.clone()
    x2[0, K - 1], d2[T - 1, 0] = float("inf"), float("nan")
    dw = m.moe_linear_backward(d2, x2, None, need_d_x=False, need_d_bias=False)[1]
    assert bool(torch.isnan(dw[0]).all())
    assert bool(torch.isfinite(dw[1:, :K - 1]).all()) and not bool(torch.isfinite(dw[:, K - 1]).any())
