"""Results and workspaces of the norms and the dense product in memory that another
argument or result takes are refused."""
import pytest
import torch

from _parity import dev

pytestmark = pytest.mark.gpu

B16 = torch.bfloat16


def test_norm():
    import sparse_moe_expert_gb300 as m
    T, H = 64, 64
    flat = torch.randn(8 * T * H, device=dev())
    x, w, b = flat[:T * H].view(T, H), flat[T * H:T * H + H].clone(), flat[T * H:T * H + H].clone()
    r, stat = x.clone(), torch.zeros(T, device=dev())
    out = torch.empty_like(x)
    for mean, rstd in ((stat, stat), (x[3], None), (None, x[3]), (r[0], None), (None, w), (b, None),
                       (None, out[0])):
        with pytest.raises(ValueError):
            m.moe_layer_norm(x, w, b, residual=r, mean=mean, rstd=rstd, out=out)
    _, s, mean, rstd = m.moe_layer_norm(x, w, b, residual=r, need_stats=True)
    with pytest.raises(ValueError):
        m.moe_layer_norm(x, w, b, residual=r, summed=s, mean=s[5])
    d, ds = torch.randn_like(x), torch.randn_like(x)
    own = torch.zeros(H, device=dev())
    bytes_of = flat[T * H:].view(torch.uint8)
    for kw in (dict(d_weight=own, d_bias=own), dict(d_weight=d[1]), dict(d_bias=s[1]), dict(d_weight=ds[1]),
               dict(d_bias=w), dict(d_weight=mean), dict(d_bias=rstd),
               dict(d_x=d, d_bias=d[0]),
               dict(workspace=bytes_of, d_weight=flat[T * H:T * H + H]),
               dict(workspace=bytes_of, d_x=flat[T * H:2 * T * H].view(T, H)),
               dict(workspace=flat.view(torch.uint8), d_bias=flat[:H])):
        with pytest.raises(ValueError):
            m.moe_layer_norm_backward(d, s, rstd, mean, w, d_sum=ds, **kw)
    big = torch.zeros(T + 1, T, device=dev())  # 64 rows of 64: a row is as long as the statistics
    with pytest.raises(ValueError):
        m.moe_layer_norm_backward(d, s, big[2], mean, w, d_x=big[:T])
    with pytest.raises(ValueError):
        m.moe_layer_norm_backward(d, s, rstd, big[2], w, d_x=big[:T])
    got = m.moe_layer_norm_backward(d, s, rstd, mean, w, d_sum=ds, d_weight=own, workspace=bytes_of)
    want = m.moe_layer_norm_backward(d, s, rstd, mean, w, d_sum=ds)
    assert got[1] is own and all(torch.equal(p, q) for p, q in zip(got, want))


def test_linear():
    import sparse_moe_expert_gb300 as m
    T, K, N = 64, 64, 64
    x, w, d = (torch.randn(64, 64, device=dev()).to(B16) for _ in range(3))
    d_w, d_x = torch.empty(N, K, device=dev()), torch.empty(T, K, dtype=B16, device=dev())
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=dev())
    for kw in (dict(d_w=d_w, d_bias=d_w[3]), dict(d_x=d_x, d_bias=d_x.view(torch.float32)[0:2].view(-1)),
               dict(d_bias=ws[:4 * N].view(torch.float32), workspace=ws),
               dict(d_w=ws[:4 * N * K].view(torch.float32).view(N, K), workspace=ws),
               dict(d_x=ws[:2 * T * K].view(B16).view(T, K), workspace=ws)):
        with pytest.raises(ValueError):
            m.moe_linear_backward(d, x, w, **kw)
    for name in ("d", "x", "w"):
        args = dict(d=d, x=x, w=w)
        args[name] = ws[:2 * 64 * 64].view(B16).view(64, 64)
        with pytest.raises(ValueError):
            m.moe_linear_backward(args["d"], args["x"], args["w"], workspace=ws)
    pre = ws[:2 * 64 * 64].view(B16).view(64, 64)
    with pytest.raises(ValueError):
        m.moe_linear_backward(d, x, w, pre, activation=m.ACT_SILU, workspace=ws)
    got = m.moe_linear_backward(d, x, w, d_w=d_w, d_x=d_x, workspace=ws)
    want = m.moe_linear_backward(d, x, w)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
