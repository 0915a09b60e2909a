"""Layer and RMS norm and their gradient against the formulas in 64 bits.

Tolerances (u = 2^-24): a row's sums are trees of at most 16 serial adds, 5
shuffles and 5 more, 26 u of the sum of magnitudes.  With rows whose mean is at
most 3 of their deviations, the centred values are 104 u of the deviation off,
rstd 20 u, the products 3 u: below 130 u = 7.8e-6 of the row's size; 1e-5 in
the 2-norm.  bf16 results add one rounding, 2^-8 relative.  d_weight and d_bias
add T / (2 SMs) serial terms, 16 runs and the error of their factors: below 256
u of the sum of magnitudes for the T here, 1.6e-5.
"""
import numpy as np
import pytest
import torch

from _parity import dev

pytestmark = pytest.mark.gpu

TOL, SUM_TOL, BF16 = 1e-5, 1.6e-5, 2.0 ** -8
F32, B16 = torch.float32, torch.bfloat16


def moe():
    import sparse_moe_expert_gb300 as m
    return m


def make(T, H, dtype, seed=0, pad=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H + pad, generator=g) * scale * torch.exp(torch.randn(T, 1, generator=g))
    return (x + torch.randn(T, 1, generator=g)).to(dtype).to(dev())[:, :H]


def vec(H, seed, dtype=F32, centre=0.0):
    g = torch.Generator().manual_seed(seed)
    return (centre + 0.3 * torch.randn(H, generator=g)).to(dtype).to(dev())


def ref(x, w, b, eps, rms):
    x = x.double().cpu()
    mu = torch.zeros(x.shape[0], dtype=torch.float64) if rms else x.mean(1)
    d = x - mu[:, None]
    rstd = 1.0 / torch.sqrt((d * d).mean(1) + eps)
    y = d * rstd[:, None]
    if w is not None:
        y = y * w.double().cpu()
    if b is not None:
        y = y + b.double().cpu()
    return y, mu, rstd


def close(got, want, tol, size=None):
    got, want = got.double().cpu(), want.double().cpu()
    assert got.shape == want.shape
    size = want if size is None else size
    assert torch.isfinite(got).all()
    assert float((got - want).norm()) <= tol * float(size.norm()) + 1e-30


SHAPES = [(1, 4096), (3, 8), (5, 1), (7, 53), (2, 257), (9, 511), (4, 512), (3, 520), (33, 1000),
          (2, 4099), (6, 8192), (1, 8191), (400, 2048), (700, 64)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype,out_dtype", [(F32, F32), (B16, B16), (F32, B16), (B16, F32)])
def test_forward(T, H, kind, dtype, out_dtype):
    m = moe()
    x, r = make(T, H, dtype, 1), make(T, H, dtype, 2)
    w, b = vec(H, 3, centre=1.0), vec(H, 4)
    rms = kind == "rms"
    out, s, mean, rstd = m.moe_layer_norm(
        x, w, None if rms else b, residual=r, eps=1e-5, out_dtype=out_dtype, need_stats=True,
        kind=m.NORM_RMS if rms else m.NORM_LAYER)
    want_s = (x.float() + r.float()).to(dtype)
    assert torch.equal(s, want_s)
    y, mu, rs = ref(s, w, None if rms else b, 1e-5, rms)
    assert out.dtype == out_dtype
    close(out, y, TOL + (BF16 if out_dtype == B16 else 0.0), y if H > 1 else torch.ones_like(y))
    close(rstd, rs, TOL)
    if rms:
        assert mean is None
    else:
        close(mean, mu, 26 * 2 ** -24, s.double().abs().mean(1).cpu())
    # the sum and the norm in one call are the two calls, bit for bit
    two = m.moe_layer_norm(s, w, None if rms else b, eps=1e-5, out_dtype=out_dtype,
                           kind=m.NORM_RMS if rms else m.NORM_LAYER)
    assert torch.equal(two[0], out) and two[1] is None and two[3] is None


@pytest.mark.parametrize("H", [64, 77, 2048])
def test_strided_rows_in_place_and_bf16_weights(H):
    m = moe()
    x, r = make(12, H, B16, 5, pad=8), make(12, H, B16, 6, pad=3)
    w, b = vec(H, 7, B16, 1.0), vec(H, 8, B16)
    dense = m.moe_layer_norm(x.contiguous(), w, b, residual=r.contiguous())
    got = m.moe_layer_norm(x, w, b, residual=r)
    close(got[0], dense[0], 2 * BF16)  # another load path may add in another order
    assert torch.equal(got[1], dense[1])
    y = ref(dense[1], w, b, 1e-6, False)[0]
    close(got[0], y, TOL + BF16)
    xs, rr = x.contiguous(), r.contiguous()
    o, s, _, _ = m.moe_layer_norm(xs, w, b, residual=rr, out=xs, summed=rr)
    assert o.data_ptr() == xs.data_ptr() and s.data_ptr() == rr.data_ptr()
    assert torch.equal(o, dense[0]) and torch.equal(s, dense[1])
    assert m.moe_layer_norm(x)[0].shape == (12, H)  # no weight, no bias
    assert m.moe_layer_norm(x[:0])[0].shape == (0, H)


def test_constant_rows_and_infinities():
    m = moe()
    x = torch.full((3, 256), 2.5, device=dev())
    x[1, 7] = float("inf")
    x[2] = 0.0
    out = m.moe_layer_norm(x, eps=1e-6)[0]
    assert torch.equal(out[0], torch.zeros(256, device=dev()))
    assert torch.isnan(out[1]).all() and torch.equal(out[2], torch.zeros(256, device=dev()))
    # a deviation of 1e-3 around a mean of 100 is not lost in squares
    big = 100.0 + 1e-3 * torch.randn(2, 4096, device=dev())
    y, _, _ = ref(big, None, None, 0.0, False)
    # the mean is 26 u * 100 off, 1.6e-1 of the deviation at worst; in the mean far less
    close(m.moe_layer_norm(big, eps=0.0)[0], y, 0.16)


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("d_dtype,dtype", [(F32, F32), (B16, B16), (F32, B16), (B16, F32)])
def test_backward(T, H, kind, d_dtype, dtype):
    m = moe()
    rms = kind == "rms"
    k = m.NORM_RMS if rms else m.NORM_LAYER
    x, d, ds = make(T, H, dtype, 1), make(T, H, d_dtype, 2), make(T, H, dtype, 3)
    w = vec(H, 4, centre=1.0)
    _, _, mean, rstd = m.moe_layer_norm(x, w, eps=1e-5, kind=k, need_stats=True)
    dx, dw, db = m.moe_layer_norm_backward(d, x, rstd, mean, w, d_sum=ds, kind=k)
    assert dx.dtype == dtype and dw.dtype == db.dtype == F32
    # the formula in 64 bits, with the statistics as given
    X, D, R = x.double().cpu(), d.double().cpu(), rstd.double().cpu()[:, None]
    M = 0.0 if rms else mean.double().cpu()[:, None]
    xh, c = (X - M) * R, D * w.double().cpu()
    m1 = (c * xh).mean(1, keepdim=True)
    m0 = torch.zeros_like(m1) if rms else c.mean(1, keepdim=True)
    want = R * (c - m0 - xh * m1) + ds.double().cpu()
    size = R * (c.abs() + m0.abs() + (xh * m1).abs()) + ds.double().cpu().abs()
    close(dx, want, TOL + (BF16 if dtype == B16 else 0.0), size)
    close(dw, (D * xh).sum(0), SUM_TOL, (D * xh).abs().sum(0))
    close(db, D.sum(0), SUM_TOL, D.abs().sum(0))
    again = m.moe_layer_norm_backward(d, x, rstd, mean, w, d_sum=ds, kind=k)
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, dw, db)))


@pytest.mark.parametrize("rms", [False, True])
def test_backward_is_the_derivative(rms):
    """Against central differences of the 64-bit formula (step 1e-6 of a
    function of size 1: the quotient is 1e-9 off)."""
    m = moe()
    T, H = 3, 72
    k = m.NORM_RMS if rms else m.NORM_LAYER
    x, d, w, b = make(T, H, F32, 1), make(T, H, F32, 2), vec(H, 3, centre=1.0), vec(H, 4)
    _, _, mean, rstd = m.moe_layer_norm(x, w, b, kind=k, need_stats=True)
    dx, dw, db = m.moe_layer_norm_backward(d, x, rstd, mean, w, kind=k)

    def f(X, W, Bb):
        return float((ref(X, W, Bb, 1e-6, rms)[0] * d.double().cpu()).sum())
    X, W, Bb = x.double().cpu(), w.double().cpu(), b.double().cpu()
    rng = np.random.default_rng(0)
    for t, got, which in ((X, dx, 0), (W, dw, 1), (Bb, db, 2)):
        for _ in range(12):
            i = tuple(int(rng.integers(n)) for n in t.shape)
            keep = float(t[i])
            t[i] = keep + 1e-5
            hi = f(X, W, Bb)
            t[i] = keep - 1e-5
            lo = f(X, W, Bb)
            t[i] = keep
            assert abs((hi - lo) / 2e-5 - float(got[i])) <= 1e-4 * (1.0 + abs(float(got[i])))


def test_backward_parts_strides_in_place_and_empty():
    m = moe()
    x, d = make(50, 200, B16, 1, pad=8), make(50, 200, B16, 2, pad=5)
    w = vec(200, 3, centre=1.0)
    _, _, mean, rstd = m.moe_layer_norm(x, w, need_stats=True)
    dx, dw, db = m.moe_layer_norm_backward(d, x, rstd, mean, w)
    dense = m.moe_layer_norm_backward(d.contiguous(), x.contiguous(), rstd, mean, w)
    close(dx, dense[0], 2 * BF16)
    close(dw, dense[1], 2 * SUM_TOL)
    only = m.moe_layer_norm_backward(d, x, rstd, mean, w, need_d_weight=False, need_d_bias=False)
    assert only[1] is None and only[2] is None and torch.equal(only[0], dx)
    dd = d.contiguous()
    got = m.moe_layer_norm_backward(dd, x.contiguous(), rstd, mean, w, d_x=dd)
    assert got[0].data_ptr() == dd.data_ptr() and torch.equal(got[0], dense[0])
    none = m.moe_layer_norm_backward(d[:0], x[:0], rstd[:0], mean[:0], w)
    assert none[0].shape == (0, 200) and not none[1].any() and not none[2].any()


def test_captured_and_on_two_streams():
    m = moe()
    x, d = make(300, 1024, B16, 1), make(300, 1024, B16, 2)
    w = vec(1024, 3, centre=1.0)

    def step(stream=None):
        o, _, mean, rstd = m.moe_layer_norm(x, w, need_stats=True, stream=stream)
        return (o, *m.moe_layer_norm_backward(d, x, rstd, mean, w, stream=stream))
    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    a.wait_stream(torch.cuda.current_stream())
    b.wait_stream(torch.cuda.current_stream())
    outs = [step(s) for s in (a, b) * 10]
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for o in outs for p, q in zip(o, want))


def test_refusals():
    m = moe()
    x = make(4, 64, B16)
    w = vec(64, 1)
    bad = [dict(weight=w[:63]), dict(residual=x.float()), dict(residual=x[:3]),
           dict(summed=torch.empty_like(x)), dict(out=torch.empty(4, 64, device=dev()).t()),
           dict(weight=w, bias=w.to(B16)), dict(weight=w.half()), dict(weight=w.cpu())]
    for kw in bad:
        with pytest.raises(ValueError):
            m.moe_layer_norm(x, **kw)
    for args, kw in [((x.half(),), {}), ((x[0],), {}), ((x.t(),), {}),
                     ((x.expand(4, 64)[:1].expand(4, 64),), {})]:
        with pytest.raises(ValueError):
            m.moe_layer_norm(*args, **kw)
    for kw in (dict(eps=-1.0), dict(eps=float("nan")), dict(kind=2)):
        with pytest.raises(m.MoEError):
            m.moe_layer_norm(x, **kw)
    with pytest.raises(m.MoEError):
        m.moe_layer_norm(torch.empty(2, 8193, device=dev()))
    flat = torch.empty(4 * 64 + 64, dtype=B16, device=dev())
    with pytest.raises(ValueError):  # one row further on: rows would be read after they are written
        m.moe_layer_norm(flat[:256].view(4, 64), out=flat[64:].view(4, 64))
    o, _, mean, rstd = m.moe_layer_norm(x, w, need_stats=True)
    with pytest.raises(ValueError):
        m.moe_layer_norm_backward(o, x, rstd, None, w)
    with pytest.raises(ValueError):
        m.moe_layer_norm_backward(o, x, rstd, mean, w, kind=m.NORM_RMS)
    with pytest.raises(ValueError):
        m.moe_layer_norm_backward(o[:3], x, rstd, mean, w)
    with pytest.raises(m.MoEError):
        m.moe_layer_norm_backward(o, x, rstd, mean, w,
                                  workspace=torch.empty(16, dtype=torch.uint8, device=dev()))


@pytest.mark.parametrize("T,H", [(1, 8), (16, 8), (255, 64), (513, 64), (128, 264), (257, 512),
                                 (33, 520), (127, 1024), (129, 1024), (32, 2048), (64, 2048),
                                 (65, 2048), (31, 4096), (33, 4096)])
@pytest.mark.parametrize("d_dtype,dtype", [(F32, F32), (B16, B16), (B16, F32)])
def test_backward_around_the_form_for_few_rows(T, H, d_dtype, dtype):
    """At most 4 rows of a group, 16 groups and 16 CTAs one after the other, or what the
    other forms add: below the 256 u of the sums' tolerance."""
    m = moe()
    x, d, ds = make(T, H, dtype, 11), make(T, H, d_dtype, 12, pad=8), make(T, H, dtype, 13, pad=16)
    for w in (vec(H, 14, centre=1.0), None):
        for rms in (False, True):
            k = m.NORM_RMS if rms else m.NORM_LAYER
            _, _, mean, rstd = m.moe_layer_norm(x, w, eps=1e-5, kind=k, need_stats=True)
            args = dict(mean=None if rms else mean, weight=w, d_sum=ds, kind=k)
            d_x, d_w, d_b = m.moe_layer_norm_backward(d, x, rstd, **args)
            xd = x.double().cpu()
            mu = torch.zeros(T, 1, dtype=torch.float64) if rms else xd.mean(1, keepdim=True)
            r = 1.0 / torch.sqrt(((xd - mu) ** 2).mean(1, keepdim=True) + 1e-5)
            xh, dd = (xd - mu) * r, d.double().cpu()
            c = dd if w is None else dd * w.double().cpu()
            core = c - xh * (c * xh).mean(1, keepdim=True)
            if not rms:
                core = core - c.mean(1, keepdim=True)
            want = r * core + ds.double().cpu()
            size = r * (c.abs() + 1.0 * xh.abs() * (c * xh).abs().mean(1, keepdim=True)
                        + c.abs().mean(1, keepdim=True)) + ds.double().cpu().abs()
            close(d_x, want, TOL + (BF16 if dtype is B16 else 0.0), size)
            close(d_w, (dd * xh).sum(0), SUM_TOL, (dd * xh).abs().sum(0))
            close(d_b, dd.sum(0), SUM_TOL, dd.abs().sum(0))
            # the same bits again, and each output alone
            again = m.moe_layer_norm_backward(d, x, rstd, **args)
            assert all(torch.equal(a, b) for a, b in zip(again, (d_x, d_w, d_b)))
            only = m.moe_layer_norm_backward(d, x, rstd, need_d_weight=False, **args)
            assert only[1] is None and torch.equal(only[2], d_b) and torch.equal(only[0], d_x)
            only = m.moe_layer_norm_backward(d, x, rstd, need_d_bias=False, **args)
            assert only[2] is None and torch.equal(only[1], d_w)


@pytest.mark.parametrize("T,H", [(20, 64), (20, 2048), (20, 4096)])
def test_few_rows_on_streams_at_once_and_captured(T, H):
    """Calls on two streams and a replayed graph give the bits of a call alone."""
    m = moe()
    w = vec(H, 14, centre=1.0)
    sets = [(make(T, H, B16, 20 + i), make(T, H, B16, 30 + i)) for i in range(4)]
    rstd, mean = vec(T, 1, centre=1.0), vec(T, 2)
    want = [m.moe_layer_norm_backward(d, x, rstd, mean, w) for x, d in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i, (x, d) in enumerate(sets * 8):
        got.append(m.moe_layer_norm_backward(d, x, rstd, mean, w, stream=streams[i % 2]))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 4]))
    x, d = sets[0][0].clone(), sets[0][1].clone()
    m.moe_layer_norm_backward(d, x, rstd, mean, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = m.moe_layer_norm_backward(d, x, rstd, mean, w)
    for i in (1, 3):
        x.copy_(sets[i][0])
        d.copy_(sets[i][1])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i]))


def test_outputs_over_the_weights_are_refused():
    m = moe()
    x, w = make(4, 64, F32, 1), vec(64, 2)
    both = torch.zeros(5, 64, device=dev())
    for call in (lambda: m.moe_layer_norm(x, both[0], out=both[:4]),
                 lambda: m.moe_layer_norm(x, w, both[3], out=both[:4]),
                 lambda: m.moe_layer_norm(x, both[2], residual=x.clone(), summed=both[:4]),
                 lambda: m.moe_layer_norm_backward(x, x, w[:4], w[:4].clone(), both[1], d_x=both[:4]),
                 lambda: m.moe_layer_norm_backward(x, x, w[:4], w[:4].clone(), both[1],
                                                   d_weight=both[1])):
        with pytest.raises(ValueError):
            call()
