"""A block of routed and shared experts between two norms: serving it, and
fine-tuning what is not quantized.

Two blocks run in a row, the second adding the first's output to the residual
stream inside its norm's kernel.  Then the first block's router, shared expert and
output norm learn a target for a few steps of AdamW with 8-bit states, the whole
step captured in one CUDA graph.

    python examples/block_finetuning.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_moe_expert_gb300 as moe  # noqa: E402
import workloads  # noqa: E402


def build(device, T=96, shared=768, seed=0):
    cfg = workloads.CONFIGS["batched"].scaled(H=1024, I=576, E=64, k=4, T=T)
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def normal(*shape, scale):
        return (torch.randn(shape, generator=g, device=device) * scale).to(torch.bfloat16)

    H = cfg.H
    layer = moe.MoELayer.from_workload(
        workloads.make_layer(cfg), device,
        scoring=moe.ScoredRouting(score=moe.SCORE_SIGMOID, n_groups=8, topk_groups=4, scale=2.5),
        shared=moe.SharedExpert(normal(2 * shared, H, scale=H ** -0.5),
                                normal(H, shared, scale=shared ** -0.5)),
        norm=moe.Norm(torch.ones(H, device=device)),
        out_norm=moe.Norm(torch.ones(H, device=device)))
    x = moe.bf16_from_bits(workloads.make_tokens(cfg), device)
    return layer, x


def gradients(layer, x, target):
    """-> (gradient of the mean squared distance to ``target``, the gradients of
    the layer's trainable tensors)."""
    out, _ = layer.block(x)
    diff = out.float() - target.float()
    d_out = (diff * (2.0 / diff.numel())).to(torch.bfloat16)
    return d_out, layer.grads(d_out, balance_coef=1e-3, z_coef=1e-5)[0]


def main(steps=8):
    device = torch.device("cuda:0")
    layer, x = build(device)
    other, _ = build(device, seed=1)
    y, s = layer.block(x)
    y2, s2 = other.block(y, residual=s)
    print("two blocks:", tuple((y2 + s2).shape))

    target = (y.float() + 0.2 * torch.randn_like(y.float())).to(torch.bfloat16)
    layer.keep_for_grad = True
    lr = torch.full((1,), 1e-3, device=device)
    opt = moe.AdamW(layer.trainable(), lr=lr, state_bits=8,
                    weight_decay={"shared.gate_up": 0.01, "shared.down": 0.01})
    gradients(layer, x, target)  # buffers and what is made once
    graph = torch.cuda.CUDAGraph()
    loss = torch.zeros((), device=device)
    with torch.cuda.graph(graph):
        _, g = gradients(layer, x, target)
        loss.copy_((layer.buffers(x.shape[0])["block_out"].float() - target.float()).square().mean())
        opt.step(g)
    history = []
    for i in range(steps):
        graph.replay()
        history.append(float(loss))
        print(f"step {i}: distance {history[-1]:.6f}")
        lr.mul_(0.95)
    return history, layer, x, target


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 8)
