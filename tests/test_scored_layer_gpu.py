"""MoELayer with score routing and per-request adapters against a float64
evaluation, its router gradient against differences of the layer itself, and
the example that runs them together."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle
import workloads
from _parity import assert_layer_close, dev, rel_l2, to_np

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def make(moe, T, E, k, H, I, n, rank, path, bits=4, capacity=None, groups=4, seed=0):
    cfg = workloads.CONFIGS["tiny"].scaled(H=H, I=I, E=E, k=k, T=T, bits=bits)
    layer_np = workloads.make_layer(cfg)
    d = dev()
    g = np.random.default_rng(seed)

    def t(*shape, s):
        return torch.tensor(g.normal(0, s, shape), dtype=torch.float32, device=d).bfloat16()

    bias = np.float32(np.round(g.normal(0, 20, E)) * 0.001)
    scoring = moe.ScoredRouting(score=moe.SCORE_SIGMOID, select_bias=torch.tensor(bias, device=d),
                                n_groups=groups, topk_groups=max(1, groups // 2), scale=2.5)
    lora = moe.ExpertAdapters(t(n, E, rank, H, s=H ** -0.5), t(n, E, 2 * I, rank, s=0.2),
                              t(n, E, rank, I, s=I ** -0.5), t(n, E, H, rank, s=0.2),
                              torch.tensor(g.random(n) + 0.5, dtype=torch.float32, device=d))
    layer = moe.MoELayer.from_workload(layer_np, d, scoring=scoring, adapters=lora, path=path,
                                       capacity=capacity)
    x_bits = workloads.make_tokens(cfg)
    ids = g.integers(-1, n, T).astype(np.int32)
    return cfg, layer_np, layer, lora, x_bits, ids


def reference(layer_np, layer, lora, x_bits, ids, cfg, adapted):
    """float64 layer over the kernel's own routing."""
    b = layer.buffers(x_bits.shape[0])
    topk, w, inv = to_np(b["topk_ids"]), to_np(b["topk_w"]).astype(np.float64), to_np(b["inv_pos"])
    x = oracle.moe.bf16_to_f64(x_bits)
    f = lambda v: v.double().cpu().numpy()  # noqa: E731
    A1, B1, A2, B2 = f(lora.gate_up_a), f(lora.gate_up_b), f(lora.down_a), f(lora.down_b)
    sc = f(lora.scales)
    deq = {}
    for m in ("gate", "up", "down"):
        q = getattr(layer_np, m)
        cols = cfg.I if m == "down" else cfg.H
        deq[m] = [oracle.moe.dequant(q.q[e], q.s[e], q.b[e], q.bits, cols) for e in range(cfg.E)]
    out = np.zeros((x.shape[0], cfg.H))
    for t in range(x.shape[0]):
        for j, e in enumerate(topk[t]):
            if e < 0 or inv[t * topk.shape[1] + j] < 0:
                continue
            gu = np.concatenate([deq["gate"][e] @ x[t], deq["up"][e] @ x[t]])
            a = ids[t] if adapted else -1
            if a >= 0:
                gu = gu + sc[a] * (B1[a, e] @ (A1[a, e] @ x[t]))
            h = gu[:cfg.I] / (1 + np.exp(-gu[:cfg.I])) * gu[cfg.I:]
            y = deq["down"][e] @ h
            if a >= 0:
                y = y + sc[a] * (B2[a, e] @ (A2[a, e] @ h))
            out[t] += w[t, j] * y
    return out


CASES = [  # T, E, k, H, I, adapters, rank, path, bits, capacity
    (1, 8, 2, 256, 128, 3, 8, "auto", 4, None),
    (37, 16, 4, 512, 192, 5, 16, "auto", 4, None),
    (64, 16, 4, 256, 320, 2, 24, "auto", 8, 6),
    (48, 8, 3, 256, 256, 4, 16, "auto", 6, None),
    (300, 8, 2, 512, 256, 3, 32, "tc", 4, None),
]


@pytest.mark.parametrize("T,E,k,H,I,n,rank,path,bits,cap", CASES)
def test_layer_with_scores_and_adapters(cuda_lib, T, E, k, H, I, n, rank, path, bits, cap):
    p = {"auto": cuda_lib.PATH_AUTO, "tc": cuda_lib.PATH_TC}[path]
    cfg, layer_np, layer, lora, x_bits, ids = make(cuda_lib, T, E, k, H, I, n, rank, p, bits, cap)
    x = cuda_lib.bf16_from_bits(x_bits, dev())
    cuda_lib.moe_get_device_error(clear=True)
    plain = layer(x).clone()
    assert_layer_close(to_np(plain), reference(layer_np, layer, lora, x_bits, ids, cfg, False))
    ids_t = torch.tensor(ids, device=dev())
    got = layer(x, adapter_ids=ids_t).clone()
    ref = reference(layer_np, layer, lora, x_bits, ids, cfg, True)
    assert_layer_close(to_np(got), ref)
    none = torch.tensor(ids < 0, device=dev())
    # rows without an adapter: the activation is the same arithmetic on the
    # raw halves, so the same bits
    assert torch.equal(got[none], plain[none])
    again = layer(x, adapter_ids=ids_t)
    assert torch.equal(got, again)
    assert cuda_lib.moe_get_device_error(clear=True) == 0


def test_layer_masked_experts_and_refusals(cuda_lib):
    """Experts taken out by a -inf bias are not chosen; a layer whose experts
    are all out gives zeros; wrong combinations are refused."""
    cfg, layer_np, layer, lora, x_bits, ids = make(cuda_lib, 9, 8, 2, 256, 128, 2, 8,
                                                   cuda_lib.PATH_AUTO)
    x = cuda_lib.bf16_from_bits(x_bits, dev())
    layer.scoring.select_bias[4:] = -float("inf")
    layer.scoring.select_bias[:3] = -float("inf")   # one expert left for two slots
    cuda_lib.moe_get_device_error(clear=True)
    out = to_np(layer(x, adapter_ids=torch.tensor(ids, device=dev())))
    b = layer.buffers(9)
    assert (to_np(b["topk_ids"]) == [3, -1]).all() and int(to_np(b["offsets"])[8]) == 9
    assert_layer_close(out, reference(layer_np, layer, lora, x_bits, ids, cfg, True))
    layer.scoring.select_bias[:] = -float("inf")
    assert not to_np(layer(x)).any()
    assert cuda_lib.moe_get_device_error(clear=True) == 0
    with pytest.raises(ValueError):
        cuda_lib.MoELayer.from_workload(layer_np, dev(), adapters=lora, fuse_gate_up=False)
    with pytest.raises(ValueError):
        cuda_lib.MoELayer.from_workload(layer_np, dev(), scoring=layer.scoring, groups=2)
    bare = cuda_lib.MoELayer.from_workload(layer_np, dev())
    with pytest.raises(ValueError):
        bare(x, adapter_ids=torch.tensor(ids, device=dev()))
    with pytest.raises(ValueError):
        bare.router_grad(x)


def test_router_grad_is_the_difference_of_the_layer(cuda_lib):
    """Directional differences of sum(d_out * layer) plus the losses, in
    float64 over the kernel's experts' rows, against router_grad."""
    cfg, layer_np, layer, lora, x_bits, ids = make(cuda_lib, 40, 16, 4, 256, 128, 3, 8,
                                                   cuda_lib.PATH_AUTO)
    x = cuda_lib.bf16_from_bits(x_bits, dev())
    ids_t = torch.tensor(ids, device=dev())
    layer(x, adapter_ids=ids_t)
    g = np.random.default_rng(4)
    d_out = torch.tensor(g.normal(size=(40, 256)), dtype=torch.float32, device=dev()).bfloat16()
    d_logits, losses = layer.router_grad(d_out, balance_coef=0.5, z_coef=0.01)
    b = layer.buffers(40)
    y, topk, inv = b["y"].double().cpu().numpy(), to_np(b["topk_ids"]), to_np(b["inv_pos"])
    D, l0 = d_out.double().cpu().numpy(), b["logits"].double().cpu().numpy()
    counts = to_np(b["counts"]).astype(np.float64)
    proj = np.array([[D[t] @ y[inv[t * 4 + j]] for j in range(4)] for t in range(40)])

    def objective(l):
        s = 1 / (1 + np.exp(-l))
        w = np.take_along_axis(s, topk, 1)
        w = 2.5 * w / w.sum(1, keepdims=True)
        q = s / s.sum(1, keepdims=True)
        m = l.max(1, keepdims=True)
        lse = (m + np.log(np.exp(l - m).sum(1, keepdims=True)))[:, 0]
        return ((w * proj).sum(), 0.5 * 16 / (4 * 40) * (counts * q.mean(0)).sum(),
                0.01 * (lse ** 2).mean())

    assert np.allclose(to_np(losses), objective(l0)[1:], rtol=1e-5)
    num = np.zeros_like(l0)
    for t in range(40):
        for e in range(16):
            hi, lo = l0.copy(), l0.copy()
            hi[t, e] += 1e-5
            lo[t, e] -= 1e-5
            num[t, e] = (sum(objective(hi)) - sum(objective(lo))) / 2e-5
    # fp32 sums over H = 256 in d_w, then the gradient's own 1e-5
    assert rel_l2(to_np(d_logits), num) <= 2e-5


def test_example_runs_and_learns(cuda_lib):
    spec = importlib.util.spec_from_file_location(
        "score_routing_and_adapters", os.path.join(ROOT, "examples",
                                                   "score_routing_and_adapters.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    history, plain, adapted, none = ex.main(6)
    assert torch.equal(adapted[none], plain[none])
    assert not torch.equal(adapted[~none], plain[~none])
    assert history[-1][0] < history[0][0]
    assert all(np.isfinite(h).all() for h in history)


@pytest.mark.parametrize("capacity", [0, 3, 9])
def test_router_grad_with_a_capacity_balances_what_was_chosen(cuda_lib, capacity):
    """An expert's capacity turns rows away from the products; the balance loss
    still counts every choice of the router.  Against the objective in 64 bits
    with counts taken from the ids, and its differences."""
    T, E, k, H = 40, 16, 4, 256
    cfg, layer_np, layer, lora, x_bits, ids = make(cuda_lib, T, E, k, H, 128, 3, 8,
                                                   cuda_lib.PATH_AUTO, capacity=capacity)
    x = cuda_lib.bf16_from_bits(x_bits, dev())
    layer(x, adapter_ids=torch.tensor(ids, device=dev()))
    g = np.random.default_rng(5)
    d_out = torch.tensor(g.normal(size=(T, H)), dtype=torch.float32, device=dev()).bfloat16()
    d_logits, losses = layer.router_grad(d_out, balance_coef=0.5, z_coef=0.01)
    b = layer.buffers(T)
    y, topk, inv = b["y"].double().cpu().numpy(), to_np(b["topk_ids"]), to_np(b["inv_pos"])
    counts = np.bincount(topk[topk >= 0], minlength=E).astype(np.float64)
    assert (counts > capacity).any() and (inv == -2).any()  # the capacity binds
    D, l0 = d_out.double().cpu().numpy(), b["logits"].double().cpu().numpy()
    proj = np.array([[D[t] @ y[inv[t * k + j]] if inv[t * k + j] >= 0 else 0.0
                      for j in range(k)] for t in range(T)])

    def objective(l):
        s = 1 / (1 + np.exp(-l))
        w = np.take_along_axis(s, topk, 1)
        w = 2.5 * w / w.sum(1, keepdims=True)
        q = s / s.sum(1, keepdims=True)
        m = l.max(1, keepdims=True)
        lse = (m + np.log(np.exp(l - m).sum(1, keepdims=True)))[:, 0]
        return ((w * proj).sum(), 0.5 * E / (k * T) * (counts * q.mean(0)).sum(),
                0.01 * (lse ** 2).mean())

    assert np.allclose(to_np(losses), objective(l0)[1:], rtol=1e-5)
    num = np.zeros_like(l0)
    for t in range(T):
        for e in range(E):
            hi, lo = l0.copy(), l0.copy()
            hi[t, e] += 1e-5
            lo[t, e] -= 1e-5
            num[t, e] = (sum(objective(hi)) - sum(objective(lo))) / 2e-5
    # fp32 sums over H = 256 in d_w, then the gradient's own 1e-5
    assert rel_l2(to_np(d_logits), num) <= 2e-5


def test_adapters_of_a_served_layer_may_change(cuda_lib):
    """Another set of adapters (more of them, a rank whose rows are grouped, a
    pair that was missing) at a batch size already served: the same bits as a
    layer made with them."""
    T, E, k = 100, 8, 2
    moe = cuda_lib

    def layer_with(n, rank):
        return make(moe, T, E, k, 256, 128, n, rank, moe.PATH_AUTO)

    _, _, layer, small, x_bits, _ = layer_with(2, 8)
    large_layer = layer_with(3, 64)[2]
    large = large_layer.adapters
    assert moe.moe_lora_workspace_size(T, k, E, 3, 64) > moe.moe_lora_workspace_size(T, k, E, 2, 8)
    x = moe.bf16_from_bits(x_bits, dev())
    ids = torch.arange(-1, T - 1, device=dev(), dtype=torch.int32) % 3
    layer.adapters = moe.ExpertAdapters(down_a=small.down_a, down_b=small.down_b,
                                        scales=small.scales)
    layer(x, adapter_ids=ids % 2)
    layer.adapters = small
    layer(x, adapter_ids=ids % 2)
    layer.adapters = large
    assert torch.equal(layer(x, adapter_ids=ids), large_layer(x, adapter_ids=ids))
    layer.adapters = small                      # and back
    want = layer_with(2, 8)[2]
    assert torch.equal(layer(x, adapter_ids=ids % 2), want(x, adapter_ids=ids % 2))


def test_scoring_may_be_given_to_a_served_layer(cuda_lib):
    _, layer_np, want, _, x_bits, _ = make(cuda_lib, 100, 8, 2, 256, 128, 2, 8,
                                           cuda_lib.PATH_AUTO)
    x = cuda_lib.bf16_from_bits(x_bits, dev())
    plain = cuda_lib.MoELayer.from_workload(layer_np, dev())
    plain(x)
    with pytest.raises(ValueError):
        plain.router_grad(x)
    plain.scoring = want.scoring
    with pytest.raises(ValueError):
        plain.router_grad(x)                    # the last forward had no scores
    assert torch.equal(plain(x), want(x))
    plain.router_grad(x)


def test_host_buffers_with_adapters(cuda_lib):
    """forward_host with each token's adapter: the bits of forward; wrong ids
    are refused."""
    T = 37
    _, _, layer, _, x_bits, ids = make(cuda_lib, T, 16, 4, 512, 192, 5, 16, cuda_lib.PATH_AUTO)
    x_host = cuda_lib.bf16_from_bits(x_bits, pin=True)
    ids_host = torch.tensor(ids).pin_memory()
    out = torch.empty((T, 512), dtype=torch.bfloat16).pin_memory()
    plain = torch.empty_like(out).pin_memory()
    layer.forward_host(x_host, out, adapter_ids=ids_host)
    layer.forward_host(x_host, plain)
    torch.cuda.synchronize()
    x = x_host.to(dev())
    assert torch.equal(out, layer(x, adapter_ids=ids_host.to(dev())).cpu())
    assert torch.equal(plain, layer(x).cpu()) and not torch.equal(out, plain)
    for bad in (ids_host.long(), ids_host[:5]):
        with pytest.raises(ValueError):
            layer.forward_host(x_host, out, adapter_ids=bad)
