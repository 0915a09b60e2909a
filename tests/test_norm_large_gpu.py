"""The norms and their gradient where they are many rows, in the kernels that serve
those, against the formulas in 64 bits, row by row.

Tolerances (u = 2^-24): forward, a warp per row: a lane adds 16 times, a pair, and 5 shuffles
more, so a mean is 26 u of the row's mean magnitude off; the squares are 64 serial sums and
7 more, 71 u, so rstd is 38 u off.  Rows here have means of at most 2.2 of their deviations
(mean magnitudes of at most 2.4): centred values 63 u, products 3 u, below 110 u of the
row's size, 1e-5 asked.  bf16 results add one rounding, 2^-8 of the value.
Gradient, with the statistics as given: sums of 8 serial terms per thread, 2 and 10 more, 30 u
of the magnitudes; 1e-5 of them asked.  d_weight and d_bias: 33 rows of a CTA, 5 CTAs of a run,
32 runs and 4 u of the terms, 74 u of the magnitudes; 1.6e-5 asked.
"""
import pytest
import torch

from _parity import dev

pytestmark = pytest.mark.gpu

TOL, SUM_TOL, BF16 = 1e-5, 1.6e-5, 2.0 ** -8
F32, B16 = torch.float32, torch.bfloat16


def moe():
    import sparse_moe_expert_gb300 as m
    return m


class Draw:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(self, *shape):
        return torch.randn(shape, generator=self.g, device=dev())

    def rows(self, T, H, dtype, size, pad=0):
        shift = 3.0 * torch.rand(T, 1, generator=self.g, device=dev()) - 1.5
        return ((self.normal(T, H + pad) + shift) * size).to(dtype)[:, :H]


def rows_close(got, want, tol, size, rounding=0.0, what=""):
    """Every row: tol of its `size` and `rounding` of its values."""
    got = got.double()
    assert got.shape == want.shape and bool(torch.isfinite(got).all()), what
    err = (got - want).norm(dim=-1)
    allowed = tol * size.norm(dim=-1) + rounding * want.norm(dim=-1) + 1e-30
    assert bool((err <= allowed).all()), (what, float((err / allowed).max()))


WIDTHS = [(1024, 520), (3001, 520), (5000, 1024), (1024, 1032), (3001, 2056), (5000, 2048), (1500, 4096),
          (3001, 4088), (1024, 8192), (3001, 8184)]


@pytest.mark.parametrize("T,H", WIDTHS)
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype,out_dtype", [(F32, F32), (B16, B16), (F32, B16), (B16, F32)])
def test_forward_of_many_rows(T, H, kind, dtype, out_dtype):
    m = moe()
    d = Draw(T + H)
    rms = kind == "rms"
    size = torch.exp(0.5 * d.normal(T, 1))
    x, r = d.rows(T, H, dtype, size, pad=8), d.rows(T, H, dtype, size, pad=16)
    for residual, wt, bias in ((r, F32, True), (None, B16, True), (r, B16, False), (None, None, False)):
        w = None if wt is None else (1.0 + 0.3 * d.normal(H)).to(wt)
        b = (0.3 * d.normal(H)).to(wt) if bias else None
        args = dict(eps=1e-5, kind=m.NORM_RMS if rms else m.NORM_LAYER, out_dtype=out_dtype, need_stats=True)
        out, s, mean, rstd = m.moe_layer_norm(x, w, b, residual=residual, **args)
        total = x
        if residual is not None:
            total = (x.float() + r.float()).to(dtype)
            assert torch.equal(s, total)
        X = total.double()
        mu = torch.zeros(T, dtype=torch.float64, device=dev()) if rms else X.mean(1)
        R = 1.0 / torch.sqrt((X - mu[:, None]).square().mean(1) + 1e-5)
        y = (X - mu[:, None]) * R[:, None]
        if w is not None:
            y = y * w.double()
        size_y = y.abs()
        if b is not None:
            y = y + b.double()
            size_y = size_y + b.double().abs()
        rows_close(out, y, TOL, size_y, BF16 if out_dtype == B16 else 0.0, "out")
        assert bool(((rstd.double() - R).abs() <= 73 * 2.0 ** -24 * R).all())
        if rms:
            assert mean is None
        else:
            assert bool(((mean.double() - mu).abs() <= 26 * 2.0 ** -24 * X.abs().mean(1) + 1e-30).all())
    # in place: the sum over the residual, the result over the input
    if dtype == out_dtype:
        a, c = x.contiguous(), r.contiguous()
        want = m.moe_layer_norm(a, w, residual=c, kind=m.NORM_RMS if rms else m.NORM_LAYER)
        got = m.moe_layer_norm(a, w, residual=c, kind=m.NORM_RMS if rms else m.NORM_LAYER, out=a, summed=c)
        assert got[0] is a and got[1] is c and torch.equal(a, want[0]) and torch.equal(c, want[1])
    assert m.moe_get_device_error() == 0


@pytest.mark.parametrize("T,H", WIDTHS + [(5000, 64), (5000, 512), (3001, 2047), (2000, 4099), (1024, 8191)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("d_dtype,dtype", [(F32, F32), (B16, B16), (F32, B16), (B16, F32)])
def test_backward_of_many_rows(T, H, kind, d_dtype, dtype):
    m = moe()
    g = Draw(T + H)
    rms = kind == "rms"
    size = torch.exp(0.5 * g.normal(T, 1))
    x = g.rows(T, H, dtype, size, pad=8)
    X = x.double()
    M = torch.zeros(T, 1, dtype=F32, device=dev()) if rms else X.mean(1, keepdim=True).float()
    R = (1.0 / torch.sqrt((X - M.double()).square().mean(1, keepdim=True) + 1e-5)).float()
    d, ds = g.normal(T, H + 8).to(d_dtype)[:, :H], g.normal(T, H).to(dtype)
    for w, d_sum in (((1.0 + 0.3 * g.normal(H)), ds), ((1.0 + 0.3 * g.normal(H)).to(B16), None), (None, ds)):
        args = dict(mean=None if rms else M.view(-1), weight=w, d_sum=d_sum,
                    kind=m.NORM_RMS if rms else m.NORM_LAYER)
        dx, dw, db = m.moe_layer_norm_backward(d, x, R.view(-1), **args)
        D, r = d.double(), R.double()
        xh = (X - M.double()) * r
        c = D if w is None else D * w.double()
        m0 = 0.0 if rms else c.mean(1, keepdim=True)
        m1 = (c * xh).mean(1, keepdim=True)
        want = r * (c - m0 - xh * m1)
        size_x = r * (c.abs() + c.abs().mean(1, keepdim=True)
                      + xh.abs() * (c * xh).abs().mean(1, keepdim=True))
        if d_sum is not None:
            want, size_x = want + d_sum.double(), size_x + d_sum.double().abs()
        rows_close(dx, want, TOL, size_x, BF16 if dtype == B16 else 0.0, "d_x")
        for got, terms, what in ((dw, D * xh, "d_weight"), (db, D, "d_bias")):
            err, allowed = (got.double() - terms.sum(0)).abs(), SUM_TOL * terms.abs().sum(0)
            assert bool((err <= allowed).all()), (what, float((err / allowed).max()))
        again = m.moe_layer_norm_backward(d, x, R.view(-1), **args)
        assert all(torch.equal(p, q) for p, q in zip(again, (dx, dw, db)))
        only = m.moe_layer_norm_backward(d, x, R.view(-1), need_d_weight=False, need_d_bias=False, **args)
        assert torch.equal(only[0], dx) and only[1] is None and only[2] is None
    assert m.moe_get_device_error() == 0
