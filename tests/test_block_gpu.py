"""The layer as a block: shared expert, norms, the gradients of what learns, and
the optimizer on them, against 64-bit evaluations of the same formulas over the
routed rows that the layer's own kernels left.

Tolerances count bf16 roundings of 2^-8 each (the largest; 2-norms see less): the
shared expert's h and the two outputs for the layer (3), the norms' input and
output for the block (5), the gradients' held tensors besides (8).
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import workloads
from _parity import dev

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U8 = 2.0 ** -8


def m():
    import sparse_moe_expert_gb300 as moe
    return moe


def rand(shape, seed, scale=1.0, dtype=torch.bfloat16, centre=0.0):
    g = torch.Generator().manual_seed(seed)
    return (centre + torch.randn(shape, generator=g) * scale).to(dtype).to(dev())


def make(T=48, H=256, I=128, E=16, k=4, shared=192, scoring=True, out_norm=True, **kw):
    moe = m()
    cfg = workloads.CONFIGS["tiny"].scaled(H=H, I=I, E=E, k=k, T=T)
    layer_np = workloads.make_layer(cfg)
    if scoring:
        kw["scoring"] = moe.ScoredRouting(score=moe.SCORE_SIGMOID, n_groups=4, topk_groups=2, scale=2.0)
    layer = moe.MoELayer.from_workload(
        layer_np, dev(), shared=moe.SharedExpert(rand((2 * shared, H), 1, H ** -0.5),
                                                 rand((H, shared), 2, shared ** -0.5)),
        norm=moe.Norm(rand((H,), 3, 0.2, torch.float32, 1.0)),
        out_norm=moe.Norm(rand((H,), 4, 0.2, torch.float32, 1.0), rand((H,), 5, 0.1, torch.float32),
                          kind=moe.NORM_LAYER) if out_norm else None, **kw)
    return layer, rand((T, H), 6)


def close(got, want, tol, what=""):
    got, want = got.double(), want.double()
    assert got.shape == want.shape, what
    err = float((got - want).norm() / want.norm())
    assert err <= tol, (what, err)


def shared64(layer, x):
    g, u = (x.double() @ layer.shared.gate_up.double().t()).chunk(2, dim=1)
    return (torch.nn.functional.silu(g) * u) @ layer.shared.down.double().t()


def norm64(s, n):
    moe = m()
    mu = 0.0 if n.kind == moe.NORM_RMS else s.mean(1, keepdim=True)
    d = s - mu
    y = d / torch.sqrt((d * d).mean(1, keepdim=True) + n.eps)
    y = y * n.weight.double()
    return y if n.bias is None else y + n.bias.double()


@pytest.mark.parametrize("T", [0, 1, 7, 48, 700])
@pytest.mark.parametrize("kw", [{}, dict(scoring=False), dict(capacity=3)])
def test_shared_expert_is_added(T, kw):
    layer, _ = make(T=max(T, 1), **kw)
    x = rand((T, 256), 7)
    with_shared = layer(x).clone()
    keep, layer.shared = layer.shared, None
    alone = layer(x).clone()
    layer.shared = keep
    assert with_shared.shape == (T, 256)
    if T:
        close(with_shared, alone.double() + shared64(layer, x), 3 * U8)
        out = torch.empty_like(with_shared)
        assert layer(x, out=out) is out and torch.equal(out, with_shared)
        events = {}
        layer(x, events=events)
        assert "shared" in events


def test_adaptive_k_and_host_buffers_take_the_shared_expert():
    moe = m()
    cfg = workloads.CONFIGS["entropy"].scaled(H=256, I=128, E=8, T=100)
    layer_np = workloads.make_layer(cfg)
    sh = moe.SharedExpert(rand((128, 256), 1, 1 / 16), rand((256, 64), 2, 1 / 8))
    a = moe.MoELayer.from_workload(layer_np, dev(), shared=sh)
    b = moe.MoELayer.from_workload(layer_np, dev())
    x = rand((100, 256), 3)
    assert a.k_split(100)
    close(a(x), b(x).double() + shared64(a, x), 3 * U8)
    host, back = x.cpu().pin_memory(), torch.empty(100, 256, dtype=torch.bfloat16).pin_memory()
    a.forward_host(host, back)
    torch.cuda.synchronize()
    assert torch.equal(back.to(dev()), a(x))


def test_blocks_in_a_row():
    layers = [make()[0], make(out_norm=False)[0]]
    x = rand((48, 256), 9)
    y, s = layers[0].block(x)
    assert s is x
    first = layers[0].out_norm
    want = norm64(layers[0].buffers(48)["out"].double(), first)
    close(y, want, 2 * U8)
    y2, s2 = layers[1].block(y, residual=s)
    want_s = (y.float() + x.float()).to(torch.bfloat16)
    assert torch.equal(s2, want_s)
    h = layers[1].buffers(48)["normed"]
    close(h, norm64(want_s.double(), layers[1].norm), 2 * U8)
    assert torch.equal(y2, layers[1](h.clone()))
    with pytest.raises(ValueError):
        layers[1].norm = None
        layers[1].block(y, residual=s)


def routed64(layer, x, router_w):
    """The routed sum over the rows that the kernels left, as a function of the
    router: float64, differentiable."""
    b = layer.buffers(x.shape[0])
    l = (x.double() @ router_w.t()) * layer.inv_temperature
    if layer.logit_bias is not None:
        l = l + layer.logit_bias.double() * layer.inv_temperature
    s = torch.sigmoid(l)
    ids = b["topk_ids"].long()
    there = (ids >= 0) & (b["inv_pos"].view(ids.shape) >= 0)
    w = torch.gather(s, 1, ids.clamp_min(0)) * (ids >= 0)
    w = w / w.sum(1, keepdim=True) * layer.scoring.scale
    y = b["y"].double()[b["inv_pos"].clamp_min(0).long()].view(*ids.shape, -1)
    return ((w * there).unsqueeze(2) * y).sum(1), l, s


@pytest.mark.parametrize("T,capacity", [(48, None), (300, None), (48, 5)])
def test_gradients(T, capacity):
    layer, _ = make(T=T, capacity=capacity)
    x, d = rand((T, 256), 8), rand((T, 256), 9, 1.0 / T)
    layer.keep_for_grad = True
    layer.block(x)
    g, losses = layer.grads(d, balance_coef=0.01, z_coef=0.001)
    assert set(g) == set(layer.trainable())
    h = layer.buffers(T)["normed"]
    leaves = {n: t.detach().double().requires_grad_() for n, t in layer.trainable().items()}
    routed, l, s = routed64(layer, h, leaves["router_w"])
    gate, up = (h.double() @ leaves["shared.gate_up"].t()).chunk(2, dim=1)
    y = routed + (torch.nn.functional.silu(gate) * up) @ leaves["shared.down"].t()
    dev_ = y - y.mean(1, keepdim=True)
    out = dev_ / torch.sqrt((dev_ * dev_).mean(1, keepdim=True) + layer.out_norm.eps)
    out = out * leaves["out_norm.weight"] + leaves["out_norm.bias"]
    n = layer.chosen_counts().double()
    q = s / s.sum(1, keepdim=True)
    balance = 0.01 * layer.E / (layer.kmax * T) * (n * q.mean(0)).sum()
    z = 0.001 * torch.logsumexp(l, 1).square().mean()
    ((out * d.double()).sum() + balance + z).backward()
    for name, t in leaves.items():
        close(g[name], t.grad, 8 * U8, name)
    close(losses, torch.stack([balance, z]).detach(), 1e-4, "losses")
    # the same gradients again: nothing was used up
    again, _ = layer.grads(d, balance_coef=0.01, z_coef=0.001)
    assert all(torch.equal(a, again[k]) for k, a in g.items())


def test_gradients_without_norms_or_scoring_and_refusals():
    layer, x = make(scoring=False, out_norm=False)
    d = rand(x.shape, 3, 0.1)
    with pytest.raises(ValueError):
        layer.grads(d)
    layer.keep_for_grad = True
    layer(x)
    g, losses = layer.grads(d)
    assert losses is None and sorted(g) == ["shared.down", "shared.gate_up"]
    w1, w2 = (t.double().requires_grad_() for t in (layer.shared.gate_up, layer.shared.down))
    gate, up = (x.double() @ w1.t()).chunk(2, dim=1)
    (((torch.nn.functional.silu(gate) * up) @ w2.t()) * d.double()).sum().backward()
    close(g["shared.gate_up"], w1.grad, 4 * U8)
    close(g["shared.down"], w2.grad, 4 * U8)
    with pytest.raises(ValueError):
        layer.grads(d[:3])
    with pytest.raises(ValueError):
        layer.grads(d.float())
    layer(x[:0])
    g, _ = layer.grads(d[:0])
    assert not g["shared.down"].any() and g["shared.down"].shape == layer.shared.down.shape
    moe = m()
    with pytest.raises(ValueError):
        make(shared=12)
    with pytest.raises(ValueError):
        moe.MoELayer.from_workload(
            workloads.make_layer(workloads.CONFIGS["tiny"]), dev(),
            shared=moe.SharedExpert(rand((64, 256), 1), rand((256, 64), 2)))


@pytest.mark.parametrize("bits", [32, 8])
def test_a_training_step_together_eager_and_captured(bits):
    moe = m()

    def setup():
        layer, x = make(T=96)
        layer.keep_for_grad = True
        decay = {n: 0.1 for n in layer.trainable() if n.startswith("shared")}
        opt = moe.AdamW(layer.trainable(), lr=torch.tensor([1e-3], device=dev()), weight_decay=decay,
                        state_bits=bits)
        return layer, x, opt
    target = rand((96, 256), 20)

    def step(layer, x, opt):
        out, _ = layer.block(x)
        diff = out.float() - target.float()
        d = (diff * (2.0 / diff.numel())).to(torch.bfloat16)
        g, _ = layer.grads(d, balance_coef=1e-3, z_coef=1e-5)
        opt.step(g)
        return out
    a, xa, oa = setup()
    start = {n: t.clone() for n, t in a.trainable().items()}
    for _ in range(5):
        last = step(a, xa, oa).clone()
    b, xb, ob = setup()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # warm what is made once, on another layer
        w, xw, ow = setup()
        step(w, xw, ow)
    torch.cuda.synchronize()
    b.buffers(96)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(b, xb, ob)
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    for (n, p), (_, q) in zip(a.trainable().items(), b.trainable().items()):
        assert torch.equal(p, q), n
        assert not torch.equal(p, start[n]), n
    assert torch.equal(out, last)
    steps = {int(s["step"][0]) for s in ob.state_dict().values()}
    assert steps == {5} and moe.moe_get_device_error() == 0


def test_optimizer_states_travel():
    moe = m()
    for bits in (32, 8):
        p = {"a": rand((33, 7), 1, dtype=torch.float32), "b": rand((300,), 2), "c": rand((5,), 3)}
        g = {n: rand(t.shape, 4, dtype=torch.float32) for n, t in p.items()}
        one = moe.AdamW(p, lr=1e-2, state_bits=bits, weight_decay=0.01)
        one.step(g)
        saved = {n: {k: t.cpu() for k, t in s.items()} for n, s in one.state_dict().items()}
        at = {n: t.clone() for n, t in p.items()}
        one.step(g)
        q = {n: t.clone() for n, t in at.items()}
        two = moe.AdamW(q, lr=1e-2, state_bits=bits, weight_decay=0.01)
        two.load_state_dict(saved)
        two.step(g)
        assert all(torch.equal(p[n], q[n]) for n in p)
        with pytest.raises(ValueError):
            two.step({"a": g["a"]})
        with pytest.raises(ValueError):
            two.load_state_dict({"a": saved["a"]})
        with pytest.raises(ValueError):
            moe.AdamW(p, state_bits=32 if bits == 8 else 8).load_state_dict(saved)
    with pytest.raises(ValueError):
        moe.AdamW({"a": torch.zeros(3, dtype=torch.float16, device=dev())})
    with pytest.raises(ValueError):
        moe.AdamW({}, lr=1.0)
    with pytest.raises(ValueError):
        moe.AdamW({"a": torch.zeros(3, device=dev())}, state_bits=4)


def test_example_runs_and_its_gradients_are_the_formula():
    spec = importlib.util.spec_from_file_location(
        "block_finetuning", os.path.join(ROOT, "examples", "block_finetuning.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    history, layer, x, target = example.main(steps=3)
    assert len(history) == 3 and np.isfinite(history).all()
    # the output norm's weight: the sum over tokens of d_out times the normed rows
    d, g = example.gradients(layer, x, target)
    close(g["out_norm.weight"], (d.double() * ((layer.buffers(x.shape[0])["block_out"].double()
                                                / layer.out_norm.weight.double()))).sum(0), 4 * U8)
