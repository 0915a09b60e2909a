"""Norms, dense product and AdamW where they are large, late or side by side:
tensors of more than 2^31 elements, steps with and without launch overlap, host
threads and streams at once."""
import threading

import pytest
import torch

from _parity import dev

pytestmark = pytest.mark.gpu

B16, F32 = torch.bfloat16, torch.float32


def m():
    import sparse_moe_expert_gb300 as moe
    return moe


def rand(shape, seed, scale=1.0, dtype=B16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def same(got, want):
    assert torch.equal(got, want), float((got.double() - want.double()).abs().max())


def test_norm_past_2_31_elements():
    moe = m()
    T, H = 270_000, 8192
    x = torch.zeros(T, H, dtype=B16, device=dev())
    x[-64:] = rand((64, H), 1)
    w = rand((H,), 2, dtype=F32)
    out, _, mean, rstd = moe.moe_layer_norm(x, w, need_stats=True)
    ref = moe.moe_layer_norm(torch.cat([x[:1200], x[-64:]]), w, need_stats=True)
    same(out[-64:], ref[0][-64:])
    same(rstd[-64:], ref[3][-64:])
    assert not out[:1000].any()
    dx, dw, _ = moe.moe_layer_norm_backward(x, x, rstd, mean, w)
    part = moe.moe_layer_norm_backward(x[-64:].contiguous(), x[-64:].contiguous(), rstd[-64:].contiguous(),
                                       mean[-64:].contiguous(), w)
    same(dx[-64:], part[0])
    # all other rows are zero: the same 64 terms in another order
    assert float((dw - part[1]).norm()) <= 1e-5 * float(part[1].norm())


def test_linear_past_2_31_elements():
    moe = m()
    T, K, N = 1_060_000, 64, 2056  # 2.18e9 outputs
    x = torch.zeros(T, K, dtype=B16, device=dev())
    x[-40:] = rand((40, K), 1)
    w, b = rand((N, K), 2, 0.1), rand((N,), 3, dtype=F32)
    out = moe.moe_linear(x, w, b)[0]
    ref = x[-40:].double() @ w.double().t() + b.double()
    assert float((out[-40:].double() - ref).norm()) <= 2.0 ** -8 * float(ref.norm())
    same(out[1000], b.to(B16))
    dx, dw, db, _ = moe.moe_linear_backward(out, x, w, d_w_dtype=F32)
    want = out[-40:].double() @ w.double()
    assert float((dx[-40:].double() - want).norm()) <= 2.0 ** -8 * float(want.norm()) * 1.01
    want = out[-40:].double().t() @ x[-40:].double()
    assert float((dw.double() - want).norm()) <= 1e-5 * float(want.norm())


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_past_2_31_elements(bits):
    moe = m()
    n = 2 ** 31 + 1000
    p = torch.zeros(n, dtype=B16, device=dev())
    g = torch.zeros(n, dtype=B16, device=dev())
    g[-1000:] = 1.0
    if bits == 32:
        states = [torch.zeros(n, device=dev())], [torch.zeros(n, device=dev())]
        kw = {}
    else:
        states = [torch.zeros(n, dtype=torch.int8, device=dev())], [torch.zeros(n, dtype=torch.uint8, device=dev())]
        blocks = -(-n // moe.ADAMW_BLOCK)
        kw = dict(exp_avg_scales=[torch.zeros(blocks, device=dev())],
                  exp_avg_sq_scales=[torch.zeros(blocks, device=dev())])
    step = torch.zeros(2, dtype=torch.int32, device=dev())
    moe.moe_adamw_step([p], [g], *states, step, lr=0.5, **kw)
    same(p[-1000:], torch.full((1000,), -0.5, dtype=B16, device=dev()))
    assert not p[-5000:-1000].any() and not p[:5000].any() and step.tolist() == [1, 0]
    assert bool((states[0][0][-1000:] != 0).all()) and not states[0][0][-3000:-1000].any()


def block_step(overlap, steps=12):
    """Steps in which every kernel follows the one that writes what it reads."""
    moe = m()
    import workloads
    old = moe.moe_set_launch_overlap(overlap)
    try:
        cfg = workloads.CONFIGS["tiny"].scaled(H=512, I=128, E=16, k=4, T=6)
        layer = moe.MoELayer.from_workload(
            workloads.make_layer(cfg), dev(), scoring=moe.ScoredRouting(),
            shared=moe.SharedExpert(rand((256, 512), 1, 0.05), rand((512, 128), 2, 0.1)),
            norm=moe.Norm(torch.ones(512, device=dev())), out_norm=moe.Norm(torch.ones(512, device=dev())))
        layer.keep_for_grad = True
        # a large fp32 tensor last, so that the router's follows late in the step
        params = dict(layer.trainable(), ballast=torch.zeros(1 << 20, device=dev()))
        opt = moe.AdamW(params, lr=0.05)
        x, ballast = rand((6, 512), 3), torch.ones(1 << 20, device=dev())
        for _ in range(steps):
            out, _ = layer.block(x)
            g, _ = layer.grads(out)
            opt.step(dict(g, ballast=ballast))
            logits = moe.moe_router_logits(x, layer.router_w)
            plain = moe.moe_router_topk(x, layer.router_w, None, 1.0, 4, 4)
        return [logits, plain[0], plain[1], out.clone(), *params.values()]
    finally:
        moe.moe_set_launch_overlap(old)


def test_steps_do_not_depend_on_launch_overlap():
    with_overlap = block_step(1)
    without = block_step(0)
    for a, b in zip(with_overlap, without):
        same(a, b)


def test_host_threads_on_streams_of_their_own():
    moe = m()
    shapes = [(3, 512, 256), (100, 512, 300), (700, 512, 512)]
    data = [(rand((T, K), 1), rand((N, K), 2, 0.05), rand((T, N), 3)) for T, K, N in shapes]

    def work(stream=None):
        out = []
        for x, w, d in data:
            n, _, mean, rstd = moe.moe_layer_norm(x, need_stats=True, stream=stream)
            out += [n, *moe.moe_layer_norm_backward(n, x, rstd, mean, stream=stream)]
            y, pre = moe.moe_linear(n, w, activation=moe.ACT_SILU, need_preact=True, stream=stream)
            out += [y, pre, *moe.moe_linear_backward(d, n, w, pre, activation=moe.ACT_SILU, stream=stream)]
            p = [x.float(), w.float()]
            s = [torch.zeros_like(t) for t in p], [torch.zeros_like(t) for t in p]
            step = torch.zeros(2, dtype=torch.int32, device=dev())
            if stream is not None:
                stream.wait_stream(torch.cuda.current_stream())
            moe.moe_adamw_step(p, [x, w], *s, step, stream=stream)
            out += p + s[0] + s[1] + [step]
        return out
    want = [t.clone() for t in work()]
    torch.cuda.synchronize()
    got, errors = {}, []

    def run(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                got[i] = [work() for _ in range(4)]
        except Exception as e:  # shown by the main thread
            errors.append(e)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for outs in got.values():
        for o in outs:
            for a, b in zip(o, want):
                same(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for a, b in zip(work(side), want):
        side.synchronize()
        same(a, b)
    assert moe.moe_get_device_error() == 0
