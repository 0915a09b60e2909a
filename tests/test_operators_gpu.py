"""Score routing, its gradient and losses, the combine's gradient and the
adapters against plain implementations in 64 bits (numpy), at the sizes and
masks where they can go wrong.

Tolerances (u = 2^-24, fp32 unit roundoff):
- routing weights: a score is a handful of roundings (exponential <= 2 ulp,
  sum over E <= 1024 by a tree of depth 10, a division, a sum of <= 16 terms,
  a division, a product): < 40 u = 2.4e-6 relative;
- d_logits fp32: differences of terms of the row's own size, each with
  relative error <= 100 u; measured against the row's largest term, 1e-5;
- bf16 results: one rounding, 2^-9 relative per value, so 2^-8 in the 2-norm
  leaves room for the fp32 error in front of it;
- adapters: fp32 sums over K <= 4096 products accumulated by the tensor core
  in at most K / 16 / 8 truncating steps of 2 u plus 8 adds: 100 u worst case
  for K = 4096 relative to the sum of magnitudes (about sqrt(K) times the
  result's size in the worst, a few times in the mean): 1e-5 in the 2-norm.
"""
import math

import numpy as np
import pytest
import torch

from _parity import dev, to_np

pytestmark = pytest.mark.gpu

W_TOL, D_TOL, BF16_TOL, LORA_TOL = 2.4e-6, 1e-5, 2.0 ** -8, 1e-5


def rel(a, b):
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    n = np.linalg.norm(b)
    return float(np.linalg.norm(a - b) / n) if n else float(np.linalg.norm(a - b))


# ---------------------------------------------------------------- plain forms


def scores64(l, score):
    """l float64 [T, E] -> (scores, available)."""
    on = np.isfinite(l)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == 1:
            s = np.where(on, 1.0 / (1.0 + np.exp(-np.where(on, l, 0.0))), 0.0)
        else:
            m = np.max(np.where(on, l, -np.inf), axis=1, keepdims=True)
            e = np.where(on, np.exp(np.where(on, l, 0.0) - np.where(np.isfinite(m), m, 0.0)), 0.0)
            d = e.sum(axis=1, keepdims=True)
            s = np.where(d > 0, e / np.where(d > 0, d, 1.0), 0.0)
    return s, on


def choices64(l, score, bias):
    s, on = scores64(l, score)
    c = s if bias is None else s + bias.astype(np.float64)
    c = np.where(on & ~np.isnan(c), c, -np.inf)
    return s, c


def route64(l, k, score, bias, G, topk_groups, group_top, renorm, scale):
    """Brute force, token by token; also the smallest gap that a decision had."""
    s, c = choices64(l, score, bias)
    T, E = l.shape
    ids = np.full((T, k), -1)
    w = np.zeros((T, k))
    gap = np.full(T, np.inf)

    def order(values):
        return sorted(range(len(values)), key=lambda i: (-values[i], i))

    def margin(values, upto):
        got = sorted((v for v in values if v > -np.inf), reverse=True)
        pairs = [got[i] - got[i + 1] for i in range(min(upto, len(got) - 1))]
        pairs = [p for p in pairs if p > 0]  # exact ties go to the lower index
        return min(pairs, default=np.inf)

    for t in range(T):
        row = c[t].copy()
        if G > 1:
            n = E // G
            val = []
            for g in range(G):
                top = sorted(row[g * n:(g + 1) * n], reverse=True)
                top = [v for v in top[:group_top] if v > -np.inf]
                val.append(sum(top) if top else -np.inf)
            keep = order(val)[:topk_groups]
            gap[t] = min(gap[t], margin(val, topk_groups))
            for g in range(G):
                if g not in keep:
                    row[g * n:(g + 1) * n] = -np.inf
        gap[t] = min(gap[t], margin(row, k))
        best = [e for e in order(row)[:k] if row[e] > -np.inf]
        ids[t, :len(best)] = best
        w[t, :len(best)] = s[t, best]
        if renorm:
            tot = w[t].sum()
            w[t] = w[t] / tot if tot > 0 else 0.0
    return ids, w * scale, gap


def grad64(l, ids, dw, counts, k, score, renorm, scale, a, z):
    T, E = l.shape
    s, on = scores64(l, score)
    out = np.zeros_like(l)
    bal = zl = 0.0
    for t in range(T):
        sel = [(j, e) for j, e in enumerate(ids[t]) if e >= 0]
        ds = np.zeros(E)
        tot = sum(s[t, e] for _, e in sel)
        if dw is not None:
            if renorm and tot > 0:
                dot = sum(scale * dw[t, j] * s[t, e] for j, e in sel) / tot
                for j, e in sel:
                    ds[e] += (scale * dw[t, j] - dot) / tot
            elif not renorm:
                for j, e in sel:
                    ds[e] += scale * dw[t, j]
        S = s[t].sum()
        if S > 0 and counts is not None and a:
            q = s[t] / S
            ce = a * E / (k * T) * counts / T
            bal += (ce * q).sum()
            ds += (ce - (ce * q).sum()) / S
        if score == 1:
            out[t] = ds * s[t] * (1 - s[t])
        else:
            out[t] = s[t] * (ds - (ds * s[t]).sum())
        if on[t].any():
            m = l[t][on[t]].max()
            e = np.where(on[t], np.exp(np.where(on[t], l[t], 0) - m), 0.0)
            lse = m + math.log(e.sum())
            zl += z * lse * lse / T
            out[t] += 2 * z / T * lse * e / e.sum()
        out[t][~on[t]] = 0.0
    return out, np.array([bal, zl])


def lora64(x, row_token, row_slot, x_row, A, B, scales, base, swiglu):
    """x [.., K], A [S, R, K], B [S, N, R] float64; slot = adapter * E + expert or -1."""
    z = base.copy()
    E = A.shape[0] // len(scales)
    for r, s in enumerate(row_slot):
        if s >= 0:
            z[r] += scales[s // E] * (B[s] @ (A[s] @ x[x_row[r]]))
    if not swiglu:
        return z
    h = z.shape[1] // 2
    g, u = z[:, :h], z[:, h:]
    return g / (1 + np.exp(-g)) * u


# -------------------------------------------------------------------- routing


def check_route(moe, l_t, k, score, bias=None, G=1, topk_groups=1, group_top=2, renorm=True,
                scale=1.0, **kw):
    bias_t = None if bias is None else torch.tensor(bias, dtype=torch.float32, device=dev())
    ids, w, kd = moe.moe_route_scored(l_t, k, score=score, select_bias=bias_t, n_groups=G,
                                      topk_groups=topk_groups, group_top=group_top,
                                      renormalize=renorm, scale=scale, **kw)
    assert int(kd.item()) == k
    ids, w = to_np(ids), to_np(w)
    assert (ids[:, k:] == -1).all() and (w[:, k:] == 0).all()
    l = l_t.double().cpu().numpy()
    rid, rw, gap = route64(l, k, score, None if bias is None else np.float32(bias), G, topk_groups,
                           group_top, renorm, scale)
    # decisions closer than the fp32 error of a choice (relative to the row's
    # largest, 1e-6 at most) may go either way
    _, c64 = choices64(l, score, None if bias is None else np.float32(bias))
    top = np.abs(np.where(np.isfinite(c64), c64, 0.0)).max(axis=1)
    clear = gap > np.minimum(1e-6, W_TOL * top)
    assert clear.mean() > 0.95
    assert np.array_equal(ids[clear][:, :k], rid[clear])
    assert np.allclose(w[clear][:, :k], rw[clear], rtol=W_TOL, atol=1e-30)
    return ids, w


SHAPES = [  # T, E, k
    (1, 8, 2), (1, 256, 8), (3, 1, 1), (5, 33, 4), (64, 60, 6), (17, 64, 16), (129, 96, 8),
    (40, 384, 8), (9, 1024, 16), (1300, 128, 8), (2, 31, 3), (7, 511, 5),
]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_scored_shapes(cuda_lib, T, E, k, score, dtype):
    g = np.random.default_rng(T * 1000 + E)
    l = torch.tensor(g.normal(0, 2, (T, E)), dtype=torch.float32, device=dev()).to(dtype)
    check_route(cuda_lib, l, k, score, renorm=True, scale=2.5)
    bias = np.round(g.normal(0, 20, E)) * 0.001
    check_route(cuda_lib, l, k, score, bias=bias, renorm=False)


@pytest.mark.parametrize("E,G,tg,gt,k", [(256, 8, 4, 2, 8), (64, 4, 2, 1, 4), (60, 4, 2, 2, 6),
                                         (96, 32, 5, 2, 8), (160, 8, 3, 2, 6), (24, 3, 1, 2, 8),
                                         (32, 32, 8, 1, 8), (1024, 4, 1, 2, 16), (26, 2, 2, 2, 3)])
@pytest.mark.parametrize("score", [0, 1])
def test_route_scored_groups(cuda_lib, E, G, tg, gt, k, score):
    g = np.random.default_rng(E + G)
    l = torch.tensor(g.normal(0, 1.5, (70, E)), dtype=torch.float32, device=dev())
    l[3, : E // G] = -math.inf          # a group without any expert
    l[4] = -math.inf                    # a row without any
    l[5, 1:] = -math.inf                # one expert left
    if E // G > 1:
        l[6, 1:: E // G] = -math.inf
    bias = np.round(g.normal(0, 20, E)) * 0.001
    for b in (None, bias):
        ids, w = check_route(cuda_lib, l, k, score, bias=b, G=G, topk_groups=tg, group_top=gt)
        assert (ids[4] == -1).all() and (w[4] == 0).all()
        assert ids[5, 0] == 0 and (ids[5, 1:] == -1).all()


def test_route_scored_ties_go_to_the_lower_id(cuda_lib):
    d = dev()
    for E, k in ((8, 3), (64, 8), (256, 8), (100, 16)):
        for score in (0, 1):
            l = torch.zeros((4, E), device=d)
            l[1, E // 2:] = 1.0
            l[2, -1] = 1.0
            ids, w, _ = cuda_lib.moe_route_scored(l, k, score=score)
            ids, w = to_np(ids), to_np(w)
            assert ids[0].tolist() == list(range(k))
            hi = list(range(E // 2, E))[:k]
            assert ids[1].tolist() == (hi + list(range(k)))[:k]
            assert ids[2].tolist() == [E - 1] + list(range(k - 1))
            assert np.allclose(w[0], 1.0 / k, rtol=W_TOL)
    # equal groups: the lower ones
    ids, _, _ = cuda_lib.moe_route_scored(torch.zeros((1, 64), device=d), 4, score=1, n_groups=8,
                                          topk_groups=2, group_top=2)
    assert to_np(ids)[0].tolist() == [0, 1, 2, 3]
    # scores that saturate at 1 tie although the logits differ
    l = torch.full((1, 8), 40.0, device=d)
    l[0, 5] = 60.0
    ids, _, _ = cuda_lib.moe_route_scored(l, 2, score=1)
    assert to_np(ids)[0].tolist() == [0, 1]


def test_route_scored_masks_and_bad_values(cuda_lib):
    d = dev()
    cuda_lib.moe_get_device_error(clear=True)
    big = torch.finfo(torch.float32).max
    l = torch.zeros((6, 16), device=d)
    l[0, :14] = -math.inf                 # two left of four
    l[1] = -big                           # masked with the type's lowest value: still finite
    l[2] = -big
    l[2, 3] = 5.0
    l[3] = -200.0                         # sigmoid underflows to 0
    for score in (0, 1):
        ids, w, _ = cuda_lib.moe_route_scored(l, 4, score=score, scale=2.0)
        ids, w = to_np(ids), to_np(w)
        assert ids[0].tolist() == [14, 15, -1, -1]
        assert np.allclose(w[0], [1.0, 1.0, 0, 0], rtol=W_TOL)
        assert ids[1].tolist() == [0, 1, 2, 3]
        assert ids[2].tolist() == [3, 0, 1, 2] and w[2].tolist() == [2.0, 0.0, 0.0, 0.0]
        assert np.isfinite(w).all()
        # all scores 0 (sigmoid of the lowest value): weights 0, not NaN
        assert np.allclose(w[1], 0.0 if score else 0.5, rtol=W_TOL)
    bias = torch.zeros(16, device=d)
    bias[:8] = -math.inf                  # experts taken out by their bias
    ids, _, _ = cuda_lib.moe_route_scored(torch.zeros((2, 16), device=d), 8, score=1,
                                          select_bias=bias)
    assert to_np(ids)[0].tolist() == list(range(8, 16))
    ids, _, _ = cuda_lib.moe_route_scored(torch.zeros((2, 16), device=d), 10, score=1,
                                          select_bias=bias)
    assert to_np(ids)[1].tolist() == list(range(8, 16)) + [-1, -1]
    assert cuda_lib.moe_get_device_error(clear=True) == 0
    for bad in (math.nan, math.inf):
        for score in (0, 1):
            l = torch.zeros((3, 40), device=d)
            l[1, 0] = bad
            ids, w, _ = cuda_lib.moe_route_scored(l, 3, score=score)
            assert to_np(ids).tolist() == [[0, 1, 2], [1, 2, 3], [0, 1, 2]]
            assert np.isfinite(to_np(w)).all()
            assert cuda_lib.moe_get_device_error(clear=True) == cuda_lib.DEVERR_BAD_SCORE
    # a bias of +inf puts an expert ahead of all others, within the chosen groups
    up = torch.zeros(64, device=d)
    up[[9, 40, 41]] = math.inf
    for E, G in ((64, 1), (64, 8)):
        l = torch.linspace(-1, 1, E, device=d).repeat(3, 1)
        ids, w, _ = cuda_lib.moe_route_scored(l, 3, score=1, select_bias=up, n_groups=G,
                                              topk_groups=1 if G == 8 else G, group_top=2)
        want = [9, 40, 41] if G == 1 else [9, 15, 14]  # equal groups: the lower one
        assert to_np(ids).tolist() == [want] * 3 and np.isfinite(to_np(w)).all()
    bias[9] = math.nan
    ids, _, _ = cuda_lib.moe_route_scored(torch.zeros((1, 16), device=d), 2, score=0,
                                          select_bias=bias)
    assert to_np(ids)[0].tolist() == [8, 10]
    assert cuda_lib.moe_get_device_error(clear=True) == cuda_lib.DEVERR_BAD_SCORE


def test_route_scored_strides_kmax_and_empty(cuda_lib):
    d = dev()
    g = np.random.default_rng(5)
    for dtype in (torch.float32, torch.bfloat16):
        for off, pad in ((0, 0), (0, 8), (1, 3), (5, 64), (8, 8)):
            wide = torch.tensor(g.normal(0, 2, (33, off + 64 + pad)), dtype=torch.float32,
                                device=d).to(dtype)
            check_route(cuda_lib, wide[:, off:off + 64], 5, 1, kmax=9)
    ids, w, kd = cuda_lib.moe_route_scored(torch.empty((0, 64), device=d), 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4) and int(kd.item()) == 4
    # the same call twice gives the same bits
    l = torch.tensor(g.normal(0, 1, (500, 256)), dtype=torch.float32, device=d)
    a = cuda_lib.moe_route_scored(l, 8, n_groups=8, topk_groups=4)
    b = cuda_lib.moe_route_scored(l, 8, n_groups=8, topk_groups=4)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("E,G,tg,gt,k", [(256, 8, 4, 2, 8), (128, 1, 1, 1, 8), (60, 1, 1, 1, 5),
                                         (64, 4, 2, 1, 4), (33, 1, 1, 1, 16), (512, 32, 9, 2, 12),
                                         (8, 1, 1, 1, 8), (1000, 1, 1, 1, 3), (60, 4, 2, 2, 6)])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_scored_many_tokens_as_few(cuda_lib, E, G, tg, gt, k, score, dtype):
    """A call of many tokens gives each token what a call of few gives it, bit
    for bit, with masks, ties, empty rows and odd strides among them."""
    T = 16384 + 37
    g = torch.Generator(device=dev())
    g.manual_seed(E + G)
    wide = torch.randn((T, E + 5), generator=g, device=dev()) * 1.5
    wide[::7] = torch.round(wide[::7])                    # ties
    wide[torch.rand((T, E + 5), generator=g, device=dev()) < 0.05] = -math.inf
    wide[100] = -math.inf
    wide[101] = 0.0
    wide[102, 1:] = -math.inf
    wide = wide.to(dtype)
    bias = torch.round(torch.randn(E, generator=g, device=dev()) * 20) * 0.001
    for l, b in ((wide[:, :E].contiguous(), bias), (wide[:, :E].contiguous(), None),
                 (wide[:, 3:3 + E], bias)):
        kw = dict(k=k, score=score, select_bias=b, n_groups=G, topk_groups=tg, group_top=gt,
                  scale=2.5, kmax=k + 1 if k < 16 else k)
        ids, w, kd = cuda_lib.moe_route_scored(l, **kw)
        assert int(kd.item()) == k
        few = [cuda_lib.moe_route_scored(l[i:i + 4000], **kw) for i in range(0, T, 4000)]
        assert torch.equal(ids, torch.cat([f[0] for f in few]))
        fw = torch.cat([f[1] for f in few])
        # the weights' sum runs in another order: two roundings of <= 16 terms
        assert torch.allclose(w, fw, rtol=W_TOL, atol=0)
    cuda_lib.moe_get_device_error(clear=True)
    l = wide[:, :E].contiguous()
    l[T - 1, E - 1] = math.nan
    ids, _, _ = cuda_lib.moe_route_scored(l, k, score=score)
    assert cuda_lib.moe_get_device_error(clear=True) == cuda_lib.DEVERR_BAD_SCORE
    assert not (ids[T - 1] == E - 1).any()


def test_route_scored_refusals(cuda_lib):
    d = dev()
    l = torch.zeros((4, 64), device=d)
    f = cuda_lib.moe_route_scored
    for kw in (dict(k=0), dict(k=17), dict(k=65), dict(k=4, kmax=3), dict(k=4, n_groups=5),
               dict(k=4, n_groups=0), dict(k=4, n_groups=64), dict(k=4, n_groups=4, topk_groups=5),
               dict(k=4, n_groups=4, topk_groups=0), dict(k=4, group_top=3), dict(k=4, score=2),
               dict(k=9, n_groups=8, topk_groups=1), dict(k=4, scale=0.0), dict(k=4, scale=math.inf),
               dict(k=4, scale=math.nan)):
        with pytest.raises(cuda_lib.MoEError) as e:
            f(l, **kw)
        assert e.value.status == 1, kw
    for bad in (l.cpu(), l.double(), l.t(), l[0], l.expand(4, 64)[:, ::2]):
        with pytest.raises(ValueError):
            f(bad, 4)
    with pytest.raises(ValueError):
        f(l, 4, select_bias=torch.zeros(63, device=d))
    with pytest.raises(ValueError):
        f(l, 4, topk_ids=torch.zeros((4, 5), dtype=torch.int32, device=d))
    with pytest.raises(cuda_lib.MoEError):
        f(torch.zeros((2, 1025), device=d), 4)


def test_route_scored_on_another_stream(cuda_lib):
    d = dev()
    l = torch.randn((4096, 128), device=d)
    ref = cuda_lib.moe_route_scored(l, 8, score=1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = cuda_lib.moe_route_scored(l, 8, score=1, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])


# ------------------------------------------------------------ routing gradient


def make_grad(T, E, k, dtype, seed, masked=True):
    g = np.random.default_rng(seed)
    l = torch.tensor(g.normal(0, 1.5, (T, E)), dtype=torch.float32, device=dev()).to(dtype)
    if masked and T > 3 and E > 4:
        l[1, ::2] = -math.inf
        l[2] = -math.inf
    ids = np.argsort(-l.float().cpu().numpy(), axis=1, kind="stable")[:, :k].astype(np.int32)
    if masked and T > 3 and E > 4:
        ids[2] = -1
        ids[0, -1] = -1
        avail = np.isfinite(l[1].float().cpu().numpy())
        ids[1] = np.where(avail[ids[1]], ids[1], -1)
    dw = g.normal(0, 1, (T, k)).astype(np.float32)
    counts = np.bincount(ids[ids >= 0].ravel(), minlength=E).astype(np.int32)
    return l, ids, dw, counts


@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (5, 33, 4), (64, 60, 6), (30, 256, 8), (9, 1024, 16),
                                   (700, 128, 8), (3, 1, 1), (50, 384, 8)])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_formula(cuda_lib, T, E, k, score, renorm):
    for dtype in (torch.float32, torch.bfloat16):
        l, ids, dw, counts = make_grad(T, E, k, dtype, T + E)
        d = dev()
        a, z, scale = 0.3, 0.05, 2.5
        dl, loss = cuda_lib.moe_route_scored_backward(
            l, torch.tensor(ids, device=d), torch.tensor(dw, device=d),
            torch.tensor(counts, device=d), score=score, renormalize=renorm, scale=scale,
            balance_coef=a, z_coef=z)
        ref, rl = grad64(l.double().cpu().numpy(), ids, dw.astype(np.float64),
                         counts.astype(np.float64), k, score, renorm, scale, a, z)
        got = dl.double().cpu().numpy()
        top = np.abs(ref).max(axis=1, keepdims=True) + np.abs(scale * dw).max(axis=1, keepdims=True)
        if dtype == torch.float32:
            assert (np.abs(got - ref) <= D_TOL * top).all()
        else:
            assert (np.abs(got - ref) <= np.abs(ref) * BF16_TOL + D_TOL * top).all()
        assert np.allclose(to_np(loss), rl, rtol=1e-5, atol=1e-12)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_against_differences(cuda_lib, score, renorm):
    """Central differences of the 64-bit objective in every logit."""
    T, E, k = 4, 9, 3
    l, ids, dw, counts = make_grad(T, E, k, torch.float32, 77, masked=False)
    a, z, scale = 0.4, 0.1, 1.5
    l64 = l.double().cpu().numpy()

    def objective(x):
        s, _ = scores64(x, score)
        tot = 0.0
        for t in range(T):
            w = s[t, ids[t]]
            w = scale * (w / w.sum() if renorm else w)
            tot += (dw[t] * w).sum()
        q = s / s.sum(axis=1, keepdims=True)
        tot += a * E / (k * T) * (counts * q.mean(axis=0)).sum()
        m = x.max(axis=1)
        lse = m + np.log(np.exp(x - m[:, None]).sum(axis=1))
        return tot + z * (lse ** 2).mean()

    num = np.zeros_like(l64)
    h = 1e-5
    for t in range(T):
        for e in range(E):
            hi, lo = l64.copy(), l64.copy()
            hi[t, e] += h
            lo[t, e] -= h
            num[t, e] = (objective(hi) - objective(lo)) / (2 * h)
    d = dev()
    dl, _ = cuda_lib.moe_route_scored_backward(
        l, torch.tensor(ids, device=d), torch.tensor(dw, device=d), torch.tensor(counts, device=d),
        score=score, renormalize=renorm, scale=scale, balance_coef=a, z_coef=z)
    # differences are good to h^2 and 2^-52 / h: 1e-9; fp32 results to D_TOL
    assert np.abs(to_np(dl) - num).max() <= D_TOL * np.abs(num).max() * 4


def test_route_backward_parts_strides_and_empty(cuda_lib):
    d = dev()
    l, ids, dw, counts = make_grad(40, 64, 4, torch.float32, 3)
    ids_t, dw_t, c_t = (torch.tensor(v, device=d) for v in (ids, dw, counts))
    # the losses alone (no weights' gradient), and none at all
    dl, loss = cuda_lib.moe_route_scored_backward(l, ids_t, None, c_t, balance_coef=0.2, z_coef=0.0)
    ref, rl = grad64(l.double().cpu().numpy(), ids, None, counts, 4, 0, True, 1.0, 0.2, 0.0)
    assert np.abs(to_np(dl) - ref).max() <= D_TOL * np.abs(ref).max()
    assert np.allclose(to_np(loss), rl, rtol=1e-5)
    dl, loss = cuda_lib.moe_route_scored_backward(l, ids_t, None)
    assert not to_np(dl).any() and not to_np(loss).any()
    # strided rows in and out; the gap between rows is not written
    wide = torch.zeros((40, 80), device=d)
    wide[:, 8:72] = l
    out = torch.full((40, 70), 7.0, device=d)
    cuda_lib.moe_route_scored_backward(wide[:, 8:72], ids_t, dw_t, d_logits=out[:, 3:67])
    ref, _ = grad64(l.double().cpu().numpy(), ids, dw, None, 4, 0, True, 1.0, 0.0, 0.0)
    assert np.abs(to_np(out)[:, 3:67] - ref).max() <= D_TOL * np.abs(dw).max()
    assert (to_np(out)[:, :3] == 7).all() and (to_np(out)[:, 67:] == 7).all()
    dl, loss = cuda_lib.moe_route_scored_backward(torch.empty((0, 64), device=d),
                                                  torch.empty((0, 4), dtype=torch.int32, device=d))
    assert dl.shape == (0, 64) and to_np(loss).tolist() == [0.0, 0.0]
    # fixed order: the same bits again
    big, bi, bw, bc = make_grad(3000, 128, 8, torch.float32, 9)
    a = [cuda_lib.moe_route_scored_backward(big, torch.tensor(bi, device=d),
                                            torch.tensor(bw, device=d), torch.tensor(bc, device=d),
                                            balance_coef=0.1, z_coef=0.1) for _ in range(2)]
    assert torch.equal(a[0][0], a[1][0]) and torch.equal(a[0][1], a[1][1])
    # one chosen expert has a constant weight: exactly no gradient
    for score in (0, 1):
        one = ids_t.clone()
        one[:, 1:] = -1
        dl, _ = cuda_lib.moe_route_scored_backward(l, one, dw_t, score=score, scale=2.5)
        assert not to_np(dl).any()
    # a bad id is reported and skipped
    cuda_lib.moe_get_device_error(clear=True)
    ids_t[5, 0] = 64
    cuda_lib.moe_route_scored_backward(l, ids_t, dw_t)
    assert cuda_lib.moe_get_device_error(clear=True) == cuda_lib.DEVERR_BAD_EXPERT


def test_route_backward_refusals(cuda_lib):
    d = dev()
    l = torch.zeros((4, 64), device=d)
    ids = torch.zeros((4, 2), dtype=torch.int32, device=d)
    f = cuda_lib.moe_route_scored_backward
    for kw in (dict(balance_coef=0.1), dict(z_coef=math.nan), dict(scale=-1.0), dict(k=3),
               dict(score=5), dict(workspace=torch.empty(16, dtype=torch.uint8, device=d)),
               dict(d_logits=l)):
        with pytest.raises(cuda_lib.MoEError) as e:
            f(l, ids, **kw)
        assert e.value.status == 1, kw
    for kw in (dict(d_topk_w=torch.zeros((4, 3), device=d)),
               dict(d_logits=torch.zeros((4, 64), dtype=torch.bfloat16, device=d)),
               dict(expert_counts=torch.zeros(63, dtype=torch.int32, device=d))):
        with pytest.raises(ValueError):
            f(l, ids, **kw)


# ------------------------------------------------------------- masked grouping


def test_permute_masked(cuda_lib):
    d = dev()
    g = np.random.default_rng(1)
    for T, k, E, cap in ((1, 1, 4, None), (7, 4, 16, None), (700, 4, 60, None), (300, 8, 128, 5),
                         (5, 2, 8, 0)):
        ids = np.argsort(g.normal(size=(T, E)), axis=1)[:, :k].astype(np.int32)
        ids[g.random((T, k)) < 0.3] = -1
        cuda_lib.moe_get_device_error(clear=True)
        kd = torch.tensor([k], dtype=torch.int32, device=d)
        cnt, off, srt, inv = (to_np(v) for v in cuda_lib.moe_permute_masked(
            torch.tensor(ids, device=d), kd, E, capacity=cap))
        flat = ids.ravel()
        want, where = [], np.full(T * k, -2)
        for e in range(E):
            mine = np.nonzero(flat == e)[0][:cap]
            where[mine] = len(want) + np.arange(len(mine))
            assert cnt[e] == len(mine) and off[e] == len(want)
            want += mine.tolist()
        assert off[E] == len(want)
        assert srt[:len(want)].tolist() == want and not srt[len(want):T * k].any()
        assert np.array_equal(inv[:T * k], where)
        assert cuda_lib.moe_get_device_error(clear=True) == 0


# ------------------------------------------------------------ combine gradient


@pytest.mark.parametrize("T,k,H", [(1, 1, 64), (1, 8, 4096), (3, 2, 192), (64, 4, 1088), (33, 16, 64),
                                   (500, 8, 2048), (7, 9, 8128)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_combine_backward(cuda_lib, T, k, H, dtype):
    d = dev()
    g = np.random.default_rng(T + H)
    A = T * k
    d_out = torch.tensor(g.normal(size=(T, H)), dtype=torch.float32, device=d).bfloat16()
    y = torch.tensor(g.normal(size=(A, H)), dtype=torch.float32, device=d).to(dtype)
    inv = g.permutation(A).astype(np.int32)
    inv[g.random(A) < 0.2] = -2
    w = g.random((T, k)).astype(np.float32)
    kd = torch.tensor([k], dtype=torch.int32, device=d)
    inv_t, w_t = torch.tensor(inv, device=d), torch.tensor(w, device=d)
    dw, dy = cuda_lib.moe_combine_backward(d_out, y, inv_t, w_t, kd)
    D, Y = d_out.double().cpu().numpy(), y.double().cpu().numpy()
    rw, ry = np.zeros((T, k)), np.zeros((A, H))
    mag = np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = inv[t * k + j]
            if r >= 0:
                rw[t, j] = D[t] @ Y[r]
                mag[t, j] = np.abs(D[t]) @ np.abs(Y[r])
                ry[r] = np.float64(w[t, j]) * D[t]
    # a fp32 sum of H terms in chains of at most H / 256 and trees after them
    assert (np.abs(to_np(dw) - rw) <= mag * (H / 256 + 24) * 2.0 ** -24).all()
    tol = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8
    assert (np.abs(dy.double().cpu().numpy() - ry) <= np.abs(ry) * tol).all()
    only, none = cuda_lib.moe_combine_backward(d_out, y, inv_t, w_t, kd, need_d_y=False)
    assert none is None and torch.equal(only, dw)


def test_combine_backward_k_below_kmax_and_differences(cuda_lib):
    """d_w and d_y are the differences of sum(d_out * combine); slots past k and
    dropped slots get nothing, their rows of d_y stay untouched."""
    d = dev()
    g = np.random.default_rng(2)
    T, kmax, k, H = 5, 4, 3, 64
    y = g.normal(size=(T * kmax, H)).astype(np.float32)
    inv = np.full((T, kmax), -1, np.int32)
    inv[:, :k] = g.permutation(T * k).reshape(T, k)
    inv[2, 1] = -2
    w = g.random((T, kmax)).astype(np.float32)
    d_out = torch.tensor(g.normal(size=(T, H)), dtype=torch.float32, device=d).bfloat16()
    kd = torch.tensor([k], dtype=torch.int32, device=d)
    dy = torch.full((T * kmax, H), 3.0, device=d)
    cuda_lib.moe_get_device_error(clear=True)
    dw, dy = cuda_lib.moe_combine_backward(d_out, torch.tensor(y, device=d),
                                           torch.tensor(inv.ravel(), device=d),
                                           torch.tensor(w, device=d), kd, d_y=dy)
    assert cuda_lib.moe_get_device_error(clear=True) == 0
    D = d_out.double().cpu().numpy()

    def f(w_, y_):
        return sum(w_[t, j] * (D[t] @ y_[inv[t, j]]) for t in range(T) for j in range(k)
                   if inv[t, j] >= 0)

    w64, y64 = w.astype(np.float64), y.astype(np.float64)
    for t in range(T):
        for j in range(kmax):
            hi, lo = w64.copy(), w64.copy()
            hi[t, j] += 0.5
            lo[t, j] -= 0.5
            assert abs(float(dw[t, j]) - (f(hi, y64) - f(lo, y64))) < 1e-4
    used = set(inv[:, :k][inv[:, :k] >= 0].tolist())
    for r in range(T * kmax):
        if r not in used:
            assert (to_np(dy)[r] == 3.0).all()
            continue
        for m in (0, 63):
            hi, lo = y64.copy(), y64.copy()
            hi[r, m] += 0.5
            lo[r, m] -= 0.5
            assert abs(float(dy[r, m]) - (f(w64, hi) - f(w64, lo))) < 1e-5


def test_combine_backward_bad_rows_and_refusals(cuda_lib):
    d = dev()
    T, k, H = 3, 2, 64
    d_out = torch.ones((T, H), dtype=torch.bfloat16, device=d)
    y = torch.ones((T * k, H), device=d)
    inv = torch.arange(T * k, dtype=torch.int32, device=d)
    w = torch.ones((T, k), device=d)
    kd = torch.tensor([k], dtype=torch.int32, device=d)
    f = cuda_lib.moe_combine_backward
    cuda_lib.moe_get_device_error(clear=True)
    inv[0], inv[1] = 6, -1
    dw, _ = f(d_out, y, inv, w, kd)
    assert cuda_lib.moe_get_device_error(clear=True) == cuda_lib.DEVERR_BAD_INDEX
    assert to_np(dw)[0].tolist() == [0.0, 0.0] and (to_np(dw)[1:] == H).all()
    with pytest.raises(cuda_lib.MoEError):
        f(d_out, y, inv, w, kd, d_y=y)
    for bad in (dict(d_out=d_out.float()), dict(y=y.double()), dict(y=y[:, :32]), dict(w=w.t()),
                dict(kd=kd.long())):
        a = dict(d_out=d_out, y=y, inv=inv, w=w, kd=kd, **{})
        a.update(bad)
        with pytest.raises(ValueError):
            f(a["d_out"], a["y"], a["inv"], a["w"], a["kd"])
    dw, dy = f(torch.empty((0, H), dtype=torch.bfloat16, device=d), torch.empty((0, H), device=d),
               inv[:0], w[:0], kd)
    assert dw.shape == (0, k)


# -------------------------------------------------------------------- adapters


def make_lora(T, K, N, R, NA, seed, E=1, k=1, none=0.2, dtype=torch.float32):
    g = np.random.default_rng(seed)
    d = dev()

    def t(*shape, s=1.0, dt=torch.bfloat16):
        return torch.tensor(g.normal(0, s, shape), dtype=torch.float32, device=d).to(dt)

    ad = g.integers(0, NA, T).astype(np.int32)
    ad[g.random(T) < none] = -1
    o = dict(ad=ad, x=t(T, K), a=t(NA, E, R, K, s=K ** -0.5), b=t(NA, E, N, R, s=R ** -0.5),
             sc=(g.random(NA) + 0.5).astype(np.float32), base=t(T * k, N, dt=dtype))
    if E > 1:
        ids = np.argsort(g.normal(size=(T, E)), axis=1)[:, :k].astype(np.int32)
        order = np.argsort(ids.ravel(), kind="stable")
        o.update(ids=ids, sorted=order.astype(np.int32),
                 off=np.searchsorted(ids.ravel()[order], np.arange(E + 1)).astype(np.int32),
                 tok=order // k, slot=np.where(ad[order // k] < 0, -1,
                                               ad[order // k] * E + ids.ravel()[order]))
    else:
        o.update(tok=np.arange(T), slot=ad)
    return o


def lora_ref(o, swiglu=False, x_row=None, x=None):
    f = lambda v: v.double().cpu().numpy()  # noqa: E731
    A, B = f(o["a"]), f(o["b"])
    return lora64(f(o["x"]) if x is None else f(x), o["tok"], o["slot"],
                  o["tok"] if x_row is None else x_row, A.reshape(-1, *A.shape[2:]),
                  B.reshape(-1, *B.shape[2:]), o["sc"].astype(np.float64), f(o["base"]), swiglu)


def dense_args(o):
    d = dev()
    return (o["x"], torch.tensor(o["ad"], device=d), o["a"][:, 0], o["b"][:, 0],
            torch.tensor(o["sc"], device=d))


DENSE = [  # T, K, N, R, adapters
    (1, 64, 64, 8, 1), (1, 4096, 4096, 16, 8), (3, 128, 192, 24, 2), (33, 1088, 576, 16, 5),
    (64, 2048, 320, 32, 64), (130, 320, 1344, 64, 3), (257, 192, 64, 128, 4), (300, 704, 448, 48, 7),
    (2, 64, 11008, 104, 2), (600, 512, 704, 16, 1), (1500, 256, 128, 8, 300), (1111, 448, 192, 80, 9),
    (4100, 128, 64, 16, 3),
]


@pytest.mark.parametrize("T,K,N,R,NA", DENSE)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_lora_one_projection(cuda_lib, T, K, N, R, NA, dtype):
    o = make_lora(T, K, N, R, NA, T + K, dtype=dtype)
    ref = lora_ref(o)
    args = dense_args(o)
    out = cuda_lib.moe_lora_apply(*args, base=o["base"])
    assert out.dtype == dtype and out.data_ptr() != o["base"].data_ptr()
    tol = LORA_TOL if dtype == torch.float32 else BF16_TOL
    assert rel(out.double().cpu().numpy(), ref) <= tol
    none = o["slot"] < 0
    assert torch.equal(out[torch.tensor(none, device=dev())],
                       o["base"][torch.tensor(none, device=dev())])
    # in place, the same bits
    inp = o["base"].clone()
    assert cuda_lib.moe_lora_apply(*args, base=inp, out=inp).data_ptr() == inp.data_ptr()
    assert torch.equal(inp, out)
    # without a base: the correction alone
    delta = cuda_lib.moe_lora_apply(*args, out_dtype=torch.float32)
    o["base"] = torch.zeros_like(o["base"])
    assert rel(to_np(delta), lora_ref(o)) <= LORA_TOL
    assert not to_np(delta)[none].any()


EXPERTS = [  # T, k, E, adapters, K, N, R
    (1, 1, 4, 1, 64, 64, 8), (1, 8, 64, 16, 2048, 320, 16), (9, 2, 3, 2, 192, 128, 24),
    (64, 4, 64, 16, 320, 192, 16), (130, 3, 5, 3, 128, 448, 64), (700, 4, 8, 2, 192, 128, 32),
    (900, 8, 60, 5, 64, 64, 16),
]


@pytest.mark.parametrize("T,k,E,NA,K,N,R", EXPERTS)
@pytest.mark.parametrize("swiglu", [False, True])
def test_lora_expert_rows(cuda_lib, T, k, E, NA, K, N, R, swiglu):
    o = make_lora(T, K, N, R, NA, T + E, E=E, k=k)
    d = dev()
    route = dict(topk_ids=torch.tensor(o["ids"], device=d),
                 sorted_assign=torch.tensor(o["sorted"], device=d),
                 expert_offsets=torch.tensor(o["off"], device=d))
    args = (torch.tensor(o["ad"], device=d), o["a"], o["b"], torch.tensor(o["sc"], device=d))
    ep = cuda_lib.EPILOGUE_SWIGLU if swiglu else cuda_lib.EPILOGUE_RAW
    ref = lora_ref(o, swiglu)
    out = cuda_lib.moe_lora_apply(o["x"], *args, base=o["base"], epilogue=ep,
                                  out_dtype=torch.float32, **route)
    # SiLU * up multiplies the relative errors of both halves by at most a few
    assert rel(to_np(out), ref) <= LORA_TOL * (3 if swiglu else 1)
    # x already in sorted order gives the same bits
    xs = o["x"][torch.tensor(o["tok"], device=d)].contiguous()
    again = cuda_lib.moe_lora_apply(xs, *args, base=o["base"], epilogue=ep,
                                    out_dtype=torch.float32, x_by_token=False, **route)
    assert torch.equal(out, again)
    if swiglu:
        h = cuda_lib.moe_lora_apply(o["x"], *args, base=o["base"], epilogue=ep, **route)
        assert h.dtype == torch.bfloat16 and torch.equal(h, out.bfloat16())


def test_lora_rows_past_the_offsets_are_untouched(cuda_lib):
    """Empty and dropped slots leave fewer rows than T*k: the rest stays."""
    d = dev()
    for T in (6, 900):
        o = make_lora(T, 64, 64, 8, 2, 3, E=4, k=2)
        rows = T * 2 - 5
        off = np.minimum(o["off"], rows).astype(np.int32)
        out = torch.full((T * 2, 64), 9.0, device=d)
        cuda_lib.moe_lora_apply(o["x"], torch.tensor(o["ad"], device=d), o["a"], o["b"],
                                torch.tensor(o["sc"], device=d), base=o["base"], out=out,
                                topk_ids=torch.tensor(o["ids"], device=d),
                                sorted_assign=torch.tensor(o["sorted"], device=d),
                                expert_offsets=torch.tensor(off, device=d))
        assert rel(to_np(out)[:rows], lora_ref(o)[:rows]) <= LORA_TOL
        assert (to_np(out)[rows:] == 9.0).all()


def test_lora_all_without_adapter_nan_and_bad_ids(cuda_lib):
    d = dev()
    for T in (4, 800):
        o = make_lora(T, 128, 64, 16, 3, 8, none=0.0)
        args = list(dense_args(o))
        args[1] = torch.full((T,), -1, dtype=torch.int32, device=d)
        out = cuda_lib.moe_lora_apply(*args, base=o["base"])
        assert torch.equal(out, o["base"])
        # an adapter's NaN stays with its own rows
        args = list(dense_args(o))
        args[2] = args[2].clone()
        args[2][1] = math.nan
        mine = torch.tensor(o["ad"] == 1, device=d)
        out = cuda_lib.moe_lora_apply(*args, base=o["base"])
        assert torch.isnan(out[mine]).all() and not torch.isnan(out[~mine]).any()
        # a token's infinity stays with its own row
        args = list(dense_args(o))
        args[0] = args[0].clone()
        args[0][1] = math.inf
        out = cuda_lib.moe_lora_apply(*args, base=o["base"])
        assert not torch.isfinite(out[1]).all()
        assert torch.isfinite(out[0]).all() and torch.isfinite(out[2:]).all()
        # ids past the adapters: none, and reported
        cuda_lib.moe_get_device_error(clear=True)
        args = list(dense_args(o))
        args[1] = args[1].clone()
        args[1][2] = 3
        out = cuda_lib.moe_lora_apply(*args, base=o["base"])
        assert cuda_lib.moe_get_device_error(clear=True) == cuda_lib.DEVERR_BAD_ADAPTER
        assert torch.equal(out[2], o["base"][2])


def test_lora_deterministic_and_streams(cuda_lib):
    d = dev()
    o = make_lora(1024, 512, 256, 32, 6, 4)
    args = dense_args(o)
    a = cuda_lib.moe_lora_apply(*args, base=o["base"])
    b = cuda_lib.moe_lora_apply(*args, base=o["base"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c = cuda_lib.moe_lora_apply(*args, base=o["base"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, b) and torch.equal(a, c)
    g = torch.cuda.CUDAGraph()
    ws = torch.empty(cuda_lib.moe_lora_workspace_size(1024, 1, 1, 6, 32), dtype=torch.uint8,
                     device=d)
    out = torch.zeros_like(a)
    with torch.cuda.graph(g):
        cuda_lib.moe_lora_apply(*args, base=o["base"], out=out, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, a)


@pytest.mark.parametrize("T,NA", [(4200, 2100), (5000, 2048), (700, 60)])
def test_lora_many_adapters(cuda_lib, T, NA):
    """More adapters than the grouping counts (each row on its own), as many as
    it counts, and a batch that meets most of its adapters a few times."""
    o = make_lora(T, 64, 64, 8 if NA > 60 else 16, NA, NA)
    out = cuda_lib.moe_lora_apply(*dense_args(o), base=o["base"])
    assert rel(to_np(out), lora_ref(o)) <= LORA_TOL


def test_lora_expert_rows_in_a_graph_and_on_two_streams(cuda_lib):
    """The grouped form of expert rows replays, and calls on two streams at
    once (each with its own workspace) give what they give alone."""
    d = dev()
    cases = []
    for seed, T, E, n, K, N, R in ((1, 1200, 8, 3, 256, 256, 64), (2, 900, 6, 2, 512, 192, 128)):
        o = make_lora(T, K, N, R, n, seed, E=E, k=2)
        args = (o["x"], torch.tensor(o["ad"], device=d), o["a"], o["b"],
                torch.tensor(o["sc"], device=d), o["base"])
        kw = dict(topk_ids=torch.tensor(o["ids"], device=d),
                  sorted_assign=torch.tensor(o["sorted"], device=d),
                  expert_offsets=torch.tensor(o["off"], device=d),
                  workspace=torch.empty(cuda_lib.moe_lora_workspace_size(T, 2, E, n, R),
                                        dtype=torch.uint8, device=d))
        ref = cuda_lib.moe_lora_apply(*args, **kw)
        assert rel(to_np(ref), lora_ref(o)) <= LORA_TOL
        cases.append((args, kw, ref))
    args, kw, ref = cases[0]
    out = torch.zeros_like(ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cuda_lib.moe_lora_apply(*args, out=out, **kw)
    for _ in range(3):
        out.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[torch.empty_like(c[2]) for _ in range(20)] for c in cases]
    torch.cuda.synchronize()
    for i in range(20):
        for (args, kw, _), s, o in zip(cases, streams, outs):
            with torch.cuda.stream(s):
                cuda_lib.moe_lora_apply(*args, out=o[i], **kw)
    torch.cuda.synchronize()
    for (_, _, ref), o in zip(cases, outs):
        assert all(torch.equal(x, ref) for x in o)
    assert cuda_lib.moe_get_device_error(clear=True) == 0


def test_lora_refusals(cuda_lib):
    d = dev()
    o = make_lora(4, 128, 128, 16, 3, 8)
    x, ad, a, b, sc = dense_args(o)
    f = cuda_lib.moe_lora_apply
    base = o["base"]

    def z(*s, dt=torch.bfloat16):
        return torch.zeros(s, dtype=dt, device=d)

    for args, kw, status in (
            ((z(4, 96), ad, z(3, 16, 96), b, sc), dict(base=base), 1),          # K % 64
            ((x, ad, a, z(3, 96, 16), sc), {}, 1),                              # N % 64
            ((x, ad, z(3, 12, 128), z(3, 128, 12), sc), dict(base=base), 1),    # R % 8
            ((x, ad, z(3, 136, 128), z(3, 128, 136), sc), dict(base=base), 1),  # R > 128
            ((x, ad, a, b, sc), dict(base=base.bfloat16(), epilogue=1), 2),
            ((x, ad, a, b, sc), dict(epilogue=1), 1),                           # SWIGLU without base
            ((x, ad, a, b, sc), dict(base=base, epilogue=3), 1),
            ((x, ad, a, b, sc), dict(base=base, out=z(4, 128)), 2),             # mixed types
            ((x, ad, a, b, sc), dict(base=base, workspace=z(16, dt=torch.uint8)), 1)):
        with pytest.raises(cuda_lib.MoEError) as e:
            f(*args, **kw)
        assert e.value.status == status, kw
    for args, kw in (((x.float(), ad, a, b, sc), {}), ((x, ad.long(), a, b, sc), {}),
                     ((x, ad, a, b[:, :, :8], sc), {}), ((x, ad, a, b, sc[:2]), {}),
                     ((x, ad, a, b, sc), dict(base=base[:3])), ((x[:3], ad, a, b, sc), {}),
                     ((x, ad, a, b, sc), dict(topk_ids=torch.zeros((4, 1), dtype=torch.int32,
                                                                  device=d)))):
        with pytest.raises(ValueError):
            f(*args, **kw)
    out = f(x[:0], ad[:0], a, b, sc, base=base[:0])
    assert out.shape == (0, 128)


# -------------------------------------------------------------- logits alone


@pytest.mark.parametrize("T,H,E", [(1, 256, 8), (5, 1088, 60), (33, 576, 16), (200, 512, 128),
                                   (1300, 64, 256), (40, 128, 1024)])
def test_router_logits_match_the_fixed_order(cuda_lib, T, H, E):
    import oracle
    g = np.random.default_rng(T + E)
    x = torch.tensor(g.normal(size=(T, H)), dtype=torch.float32, device=dev()).bfloat16()
    w = g.normal(0, 0.05, (E, H)).astype(np.float32)
    bias = g.normal(size=E).astype(np.float32)
    bits = x.cpu().view(torch.int16).numpy().view(np.uint16)
    got = cuda_lib.moe_router_logits(x, torch.tensor(w, device=dev()),
                                     torch.tensor(bias, device=dev()), 0.75)
    ref = oracle.router_logits(bits, w, bias, 0.75)
    assert np.array_equal(to_np(got), ref)


# Ranks of 96 and more, whose CTAs take 128 columns at a time (64 with SwiGLU):
# column counts that are whole, and that leave half of the last unit.
@pytest.mark.parametrize("T,K,N,R,NA", [(700, 320, 192, 128, 2), (400, 128, 576, 96, 3),
                                        (1300, 64, 256, 120, 5), (350, 64, 64, 104, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_lora_wide_rank(cuda_lib, T, K, N, R, NA, dtype):
    test_lora_one_projection(cuda_lib, T, K, N, R, NA, dtype)


@pytest.mark.parametrize("T,k,E,NA,K,N,R", [(600, 2, 3, 2, 128, 192, 128), (500, 1, 2, 1, 64, 256, 96)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_lora_wide_rank_expert_rows(cuda_lib, T, k, E, NA, K, N, R, swiglu):
    test_lora_expert_rows(cuda_lib, T, k, E, NA, K, N, R, swiglu)


@pytest.mark.parametrize("pad", [0, 1])
def test_route_scored_groups_of_cancelling_biases(cuda_lib, pad):
    """Groups whose two best choices are large and of opposite sign: their sum
    is small, its rounding is the summands'.  The scores are taken from the
    call itself (every expert, no bias; checked in 64 bits), the choices and
    the group values from the definition in fp32.  One group's score runs over
    the floats around the points where score + 4096 rounds up, the other's
    stays inside the interval below."""
    step = 2.0 ** -11                        # an ulp of 4096 + s
    q = np.arange(80, 1960, dtype=np.float64)
    edge, inside = (q + 0.5) * step, q * step
    at = np.log(edge / (1 - edge)).astype(np.float32)
    near = np.stack([(at.view(np.int32) + d).view(np.float32) for d in range(-32, 33)], 1)
    other = np.log(inside / (1 - inside)).astype(np.float32)
    n = 2 + pad                              # experts of a group; the third one is masked
    l = np.full(near.shape + (2 * n,), -np.inf, np.float32)
    l[..., 0] = other[:, None]
    l[..., n] = near
    l[..., 1] = l[..., n + 1] = -0.3
    l = l.reshape(-1, 2 * n)
    bias = np.zeros(2 * n, np.float32)
    bias[[0, n]], bias[[1, n + 1]] = 4096.0, -4096.0
    l_t, d = torch.tensor(l, device=dev()), dev()
    on = np.isfinite(l)
    ids, w, _ = cuda_lib.moe_route_scored(l_t, 4, score=1, renormalize=False)
    s = np.zeros_like(l)
    np.put_along_axis(s, to_np(ids).astype(np.int64), to_np(w).astype(np.float32), 1)
    s64, _ = scores64(l.astype(np.float64), 1)
    assert np.allclose(s[on], s64[on], rtol=W_TOL, atol=0)
    c = (s + bias).astype(np.float32)
    value = np.stack([c[:, 0] + c[:, 1], c[:, n] + c[:, n + 1]], 1)
    assert (value[:, 0] == value[:, 1]).any() and (value[:, 0] < value[:, 1]).any()
    want = np.where(value[:, 1] > value[:, 0], n, 0)   # equal groups: the lower one
    ids, _, _ = cuda_lib.moe_route_scored(l_t, 2, score=1, select_bias=torch.tensor(bias, device=d),
                                          n_groups=2, topk_groups=1, group_top=2)
    assert np.array_equal(to_np(ids), np.stack([want, want + 1], 1))


def test_lora_rows_of_a_that_pass_32_bits(cuda_lib):
    """32 rows of A are 2^31 elements long: exact sums of single products at
    both ends of K, ranks past 32 among them."""
    T, K, N, R = 160, 1 << 26, 64, 40
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 30 GB")
    d = dev()
    x = torch.zeros((T, K), dtype=torch.bfloat16, device=d)
    a = torch.zeros((1, R, K), dtype=torch.bfloat16, device=d)
    rank = torch.arange(R, device=d)
    at = torch.where(rank % 2 == 0, rank * 7, K - 1 - rank * 3)  # different columns
    value = torch.randint(-8, 9, (T, R), device=d).bfloat16()
    x[:, at] = value
    a[0, rank, at] = 1.0
    b = torch.randint(-2, 3, (1, N, R), device=d).bfloat16()
    ids = torch.zeros(T, dtype=torch.int32, device=d)
    base = torch.randint(-4, 5, (T, N), device=d).float()
    got = cuda_lib.moe_lora_apply(x, ids, a, b, None, base)
    assert torch.equal(got.double(), base.double() + value.double() @ b[0].double().t())


@pytest.mark.parametrize("E,k", [(1, 1), (16, 4)])
def test_lora_calls_that_share_a_workspace(cuda_lib, E, k):
    """Calls one behind the other on one workspace, their adapters and tile
    lists different each time, eager and as a graph: each as when alone."""
    T, K, N, R, n = 1500, 512, 384, 32, 6
    d = dev()
    g = torch.Generator(device=d)
    g.manual_seed(E)
    a = (torch.randn((n, E, R, K), generator=g, device=d) * K ** -0.5).bfloat16()
    b = torch.randn((n, E, N, R), generator=g, device=d).bfloat16()
    if E == 1:
        a, b = a[:, 0], b[:, 0]
    x = torch.randn((T, K), generator=g, device=d).bfloat16()
    base = torch.randn((T * k, N), generator=g, device=d)
    ws = torch.empty(cuda_lib.moe_lora_workspace_size(T, k, E, n, R), dtype=torch.uint8, device=d)
    assert ws.numel() > 256                      # the grouped form
    calls = []
    for i in range(12):
        # none, one, few or all adapters, more or fewer tiles each time
        ids = torch.randint(-1, 1 + i % n, (T,), generator=g, device=d, dtype=torch.int32)
        ids[: (i * 331) % T] = -1
        kw = {}
        if E > 1:
            topk = torch.stack([torch.randperm(1 + (i % 4) * 5 if i % 4 else E, generator=g,
                                               device=d)[:k] for _ in range(T)]) \
                if i % 4 == 0 else torch.randint(0, 1 + (i % 4) * 5, (T, k), generator=g, device=d)
            topk = topk.int().contiguous()
            _, off, order, _ = cuda_lib.moe_permute_masked(
                topk, torch.full((1,), k, dtype=torch.int32, device=d), E)
            kw = dict(topk_ids=topk, sorted_assign=order, expert_offsets=off)
        out = torch.empty_like(base)
        calls.append((lambda ids=ids, kw=kw, out=out: cuda_lib.moe_lora_apply(
            x, ids, a, b, None, base, out, workspace=ws, **kw), out))
    want = []
    for call, out in calls:
        call()
        torch.cuda.synchronize()
        want.append(out.clone())

    def check():
        torch.cuda.synchronize()
        assert all(torch.equal(out, ref) for (_, out), ref in zip(calls, want))

    for _ in range(20):
        for call, out in calls:
            call()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call, out in calls:
            call()
    for _, out in calls:
        out.zero_()
    for _ in range(20):
        graph.replay()
    check()


@pytest.mark.parametrize("T,few", [(3, False), (20, False), (700, False), (110, True)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_lora_values_past_bf16_and_infinities(cuda_lib, T, few, dtype):
    """One entry of x A^T overflows to an infinity, is a NaN, or is finite and
    past bf16's largest number; the others are 0.  In every form (own rows,
    small and large tiles): infinities of B's signs, NaN, and the product; the
    other rows are as without them."""
    K, N, R, n = 256, 128, 64, 2
    d = dev()
    g = torch.Generator(device=d)
    g.manual_seed(T)
    top = 2.0 ** 127
    x = torch.zeros((T, K), device=d)
    a = torch.zeros((n, R, K), device=d)
    a[:, 0, :4] = 1.0
    a[:, 1, 4] = 255.0 / 128
    a[:, 1, 5] = 1.0
    x[0, :4] = top                         # 4 x 2^127: +inf
    x[1, :4] = -top                        # -inf
    x[2, 4], x[2, 5] = top, 2.0 ** 119     # finite, past 255 x 2^120
    if T > 3:
        x[5, 0] = math.nan
        x[4, 2] = 1.0
    b = torch.randint(1, 4, (n, N, R), generator=g, device=d) * 1.0
    b[:, ::3] *= -1.0
    b[:, :, 1] = 2.0 ** -126
    ids = torch.zeros(T, dtype=torch.int32, device=d)
    ids[6::1 if few else 2] = 1            # few: these rows are a small tile
    base = torch.randint(-3, 4, (T, N), generator=g, device=d).to(dtype)
    got = cuda_lib.moe_lora_apply(x.bfloat16(), ids, a.bfloat16(), b.bfloat16(), None,
                                  base).double()
    sign = torch.where(b[0, :, 0] > 0, 1.0, -1.0).double()
    assert torch.equal(got[0], sign * math.inf) and torch.equal(got[1], -sign * math.inf)
    want = base.double()
    want[2] += 255.0 / 64 + 2.0 ** -7
    if T > 3:
        assert got[5].isnan().all()
        want[4] += b[0, :, 0].double()
    rest = [i for i in range(T) if i not in (0, 1, 5)]
    want = want[rest].to(dtype).double()
    # exact sums of a few bits, but for the second product's own 2^-17 (bf16 base)
    assert torch.allclose(got[rest], want, rtol=0 if dtype == torch.float32 else 2.0 ** -8, atol=0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E", [32, 96, 256])
def test_route_backward_of_saturated_scores(cuda_lib, dtype, renorm, E):
    """Every chosen expert's derivative to its own relative accuracy, logits
    from -20 to 20.  Relative error of s (1 - s): e^-|l| has the roundings of
    the exponent (two of |l| log2 e <= 29, times ln 2: 2.4e-6) and of the
    hardware's exponential and reciprocal (2^-22 + 2^-23), then a few
    roundings: 4e-6; renormalized, sums and a difference of terms of one size
    on top: 1e-5.  bf16 logits: the fp32 result of the same numbers, rounded."""
    T, k, scale = 9, 16, 2.5
    g = np.random.default_rng(E)
    l = np.stack([g.permutation(np.linspace(-20, 20, E)) for _ in range(T)])
    l_t = torch.tensor(l, dtype=torch.float32, device=dev()).to(dtype).float()
    l = l_t.double().cpu().numpy()
    ids = np.stack([g.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    dw = np.float32(np.where(np.arange(k) % 2 == 0, 1.0, -1.0) * (1 + g.random((T, k))))

    def grad(logits):
        return cuda_lib.moe_route_scored_backward(
            logits, torch.tensor(ids, device=dev()), torch.tensor(dw, device=dev()), score=1,
            renormalize=renorm, scale=scale)[0]

    got = grad(l_t)
    if dtype == torch.bfloat16:
        assert torch.equal(grad(l_t.to(dtype)), got.to(dtype))
    s = 1 / (1 + np.exp(-l))
    ds = scale * dw.astype(np.float64)
    if renorm:
        p = np.take_along_axis(s, ids, 1)
        ds = (ds - (ds * p).sum(1, keepdims=True) / p.sum(1, keepdims=True)) / p.sum(1, keepdims=True)
        ds[np.abs(ds) < 0.1 * np.abs(ds).max(1, keepdims=True)] = np.nan  # differences near 0
    want = np.zeros_like(l)
    np.put_along_axis(want, ids, ds, 1)
    want *= s / (1 + np.exp(l))            # 1 - s without a difference
    got = got.double().cpu().numpy()
    on = ~np.isnan(want)
    assert on.mean() > 0.8 and (np.abs(want[on & (l > 17)]) > 0).any()
    assert np.allclose(got[on], want[on], rtol=1e-5 if renorm else 4e-6, atol=0)


@pytest.mark.parametrize("E,G,tg,k", [(256, 8, 4, 8), (60, 4, 2, 6), (33, 1, 1, 16)])
@pytest.mark.parametrize("score", [0, 1])
def test_route_scored_bits_do_not_depend_on_the_batch(cuda_lib, E, G, tg, k, score):
    """Ids and weights of one token per warp step (few tokens) and of two
    (many), bit for bit: a call of 8000 tokens against calls of 301."""
    g = torch.Generator(device=dev())
    g.manual_seed(E + score)
    l = torch.randn((8000, E), generator=g, device=dev()) * 1.5
    l[::7] = torch.round(l[::7])                              # ties
    l[torch.rand(l.shape, generator=g, device=dev()) < 0.05] = -math.inf
    l[100] = -math.inf
    bias = torch.round(torch.randn(E, generator=g, device=dev()) * 20) * 0.001
    kw = dict(k=k, score=score, select_bias=bias, n_groups=G, topk_groups=tg, scale=2.5)
    ids, w, _ = cuda_lib.moe_route_scored(l, **kw)
    few = [cuda_lib.moe_route_scored(l[i:i + 301], **kw) for i in range(0, 8000, 301)]
    assert torch.equal(ids, torch.cat([f[0] for f in few]))
    assert torch.equal(w, torch.cat([f[1] for f in few]))
