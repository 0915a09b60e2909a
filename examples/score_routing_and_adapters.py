"""Score routing, per-request adapters and router fine-tuning on one layer.

A layer of 64 experts with sigmoid scores, a balance bias and group-limited
selection serves a batch in which every request names its own adapter (or
none); then its router is fine-tuned for a few steps towards a target output,
with the balance and z losses, while the quantized experts stay fixed.

    python examples/score_routing_and_adapters.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_moe_expert_gb300 as moe  # noqa: E402
import workloads  # noqa: E402


def build(device, T=96, adapters=6, rank=16, seed=0):
    cfg = workloads.CONFIGS["batched"].scaled(H=1024, I=576, E=64, k=4, T=T)
    layer_np = workloads.make_layer(cfg)
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def normal(*shape, scale):
        return (torch.randn(shape, generator=g, device=device) * scale).to(torch.bfloat16)

    E, H, I, n = cfg.E, cfg.H, cfg.I, adapters
    gu_a, gu_b = moe.ExpertAdapters.join_gate_up(
        normal(n, E, rank, H, scale=H ** -0.5), normal(n, E, I, rank, scale=0.05),
        normal(n, E, rank, H, scale=H ** -0.5), normal(n, E, I, rank, scale=0.05))
    lora = moe.ExpertAdapters(gu_a, gu_b, normal(n, E, rank, I, scale=I ** -0.5),
                              normal(n, E, H, rank, scale=0.05),
                              torch.full((n,), 2.0, device=device))
    scoring = moe.ScoredRouting(score=moe.SCORE_SIGMOID,
                                select_bias=torch.zeros(E, device=device), n_groups=8,
                                topk_groups=4, scale=2.5)
    layer = moe.MoELayer.from_workload(layer_np, device, scoring=scoring, adapters=lora)
    x = moe.bf16_from_bits(workloads.make_tokens(cfg), device)
    ids = torch.randint(-1, n, (T,), generator=g, device=device, dtype=torch.int32)
    return layer, x, ids


def finetune_router(layer, x, adapter_ids, target, steps, lr=0.3):
    """Gradient descent on the router weight: mean squared distance to
    ``target`` plus the balance and z losses.  -> the losses per step."""
    history = []
    for _ in range(steps):
        out = layer(x, adapter_ids=adapter_ids)
        diff = out.float() - target.float()
        d_out = (diff * (2.0 / diff.numel())).to(torch.bfloat16)
        d_logits, aux = layer.router_grad(d_out, balance_coef=1e-3, z_coef=1e-5)
        history.append((float(diff.square().mean()), float(aux[0]), float(aux[1])))
        layer.router_w -= lr * layer.inv_temperature * (d_logits.t() @ x.float())
        # the balance bias moves against the load, one step per batch
        load = layer.chosen_counts().float()
        layer.scoring.select_bias += 0.001 * torch.sign(load.mean() - load)
    return history


def main(steps=8):
    device = torch.device("cuda:0")
    layer, x, adapter_ids = build(device)
    plain = layer(x).clone()
    adapted = layer(x, adapter_ids=adapter_ids).clone()
    none = adapter_ids < 0
    print("rows with an adapter differ by", float((adapted - plain)[~none].float().norm()
                                                   / plain[~none].float().norm()))
    print("rows without one are unchanged:", torch.equal(adapted[none], plain[none]))
    # another routing's output as the target
    keep = layer.router_w.clone()
    layer.router_w += 0.02 * torch.randn_like(layer.router_w)
    target = layer(x, adapter_ids=adapter_ids).clone()
    layer.router_w.copy_(keep)
    history = finetune_router(layer, x, adapter_ids, target, steps)
    for i, (mse, balance, z) in enumerate(history):
        print(f"step {i}: distance {mse:.6f}, balance {balance:.6f}, z {z:.6f}")
    return history, plain, adapted, none


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 8)
