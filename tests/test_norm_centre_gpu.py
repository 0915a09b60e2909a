"""The norms' gradient of rows far from zero, in each of its forms, against the formula
in 64 bits with the statistics as given.

Tolerances (u = 2^-24): x - mean is rounded once, its product with rstd once, so the normed
value is 2 u of itself off whatever the mean.  The sums and products that follow are those
of the other tests of this gradient: below 130 u of a row's magnitudes (1e-5), 256 u of a
column's (1.6e-5), and a rounding of bf16 results, 2^-8.
"""
import pytest
import torch

from _parity import dev

pytestmark = pytest.mark.gpu

TOL, SUM_TOL, BF16 = 1e-5, 1.6e-5, 2.0 ** -8
F32, B16 = torch.float32, torch.bfloat16


def close(got, want, tol, size, what):
    got = got.double()
    assert got.shape == want.shape and bool(torch.isfinite(got).all()), what
    err, size = float((got - want).norm()), float(size.norm())
    assert err <= tol * size + 1e-30, (what, err / max(size, 1e-300))


# few rows in a cluster, the ring with one vector and two, narrow rows, rows off their boundary
@pytest.mark.parametrize("T,H,pad", [(20, 2048, 0), (64, 64, 0), (700, 2048, 0), (700, 1000, 8),
                                     (40, 8192, 0), (1500, 64, 0), (50, 77, 0), (700, 2047, 0),
                                     (700, 2048, 1)])
@pytest.mark.parametrize("d_dtype,dtype", [(F32, F32), (B16, F32), (B16, B16)])
def test_rows_far_from_zero(T, H, pad, d_dtype, dtype):
    import sparse_moe_expert_gb300 as m
    g = torch.Generator(device="cuda").manual_seed(H + T)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev())
    w = 1.0 + 0.3 * normal(H)
    for far in (1e3, 1e5, None):
        if far is None:  # constant rows
            x = (100.3 * normal(T, 1)).expand(T, H + pad).clone()
        else:
            x = normal(T, H + pad) + far * (1.0 + 0.1 * normal(T, 1))
        x = x.to(dtype)[:, :H]
        d = normal(T, H + pad).to(d_dtype)[:, :H]
        _, _, mean, rstd = m.moe_layer_norm(x, w, need_stats=True)
        dx, dw, db = m.moe_layer_norm_backward(d, x, rstd, mean, w)
        X, D, R, M = x.double(), d.double(), rstd.double()[:, None], mean.double()[:, None]
        xh, c = (X - M) * R, D * w.double()
        m0, m1 = c.mean(1, keepdim=True), (c * xh).mean(1, keepdim=True)
        close(dx, R * (c - m0 - xh * m1), TOL + (BF16 if dtype == B16 else 0.0),
              R * (c.abs() + c.abs().mean(1, keepdim=True) + xh.abs() * (c * xh).abs().mean(1, keepdim=True)),
              (far, "d_x"))
        close(dw, (D * xh).sum(0), SUM_TOL, (D * xh).abs().sum(0), (far, "d_weight"))
        close(db, D.sum(0), SUM_TOL, D.abs().sum(0), (far, "d_bias"))
