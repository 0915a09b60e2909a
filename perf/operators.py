"""Operators measured beside the layer: routing by scores, its gradient with the
balance and z losses, the combine's gradient, and low-rank adapters of many
requests on shared or per-expert projections.

``own`` false runs each operator in elementary torch operations in 32 bits;
``own`` true makes the package's calls.  Cases are plain dicts; ``prepare``
makes the inputs a serving or training program has in hand.
"""
import math

import torch

own = False

SIGMOID, SOFTMAX = "sigmoid", "softmax"
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one token of a decode loop: 256 experts in 8 groups, balance bias
        dict(name="route_decode", op="route", T=1, E=256, k=8, score=SIGMOID, dtype="fp32",
             groups=8, topk_groups=4, group_top=2, bias=True, renorm=True, scale=2.5, masked=0.0),
        # a decode batch over 64 experts, some of them offline for every token
        dict(name="route_batch", op="route", T=64, E=64, k=4, score=SOFTMAX, dtype="bf16",
             groups=1, topk_groups=1, group_top=1, bias=False, renorm=True, scale=1.0,
             masked=0.1),
        # a prefill chunk over 128 experts, softmax scores with a balance bias
        dict(name="route_prefill", op="route", T=4096, E=128, k=8, score=SOFTMAX, dtype="fp32",
             groups=1, topk_groups=1, group_top=1, bias=True, renorm=True, scale=1.0, masked=0.0),
        # a long packed batch: group-limited sigmoid routing of 64k tokens
        dict(name="route_long", op="route", T=65536, E=256, k=8, score=SIGMOID, dtype="bf16",
             groups=8, topk_groups=4, group_top=2, bias=True, renorm=True, scale=2.5, masked=0.0),
        # router fine-tuning on one prefill-sized batch
        dict(name="route_grad_prefill", op="route_grad", T=4096, E=128, k=8, score=SOFTMAX,
             dtype="fp32", renorm=True, scale=1.0, balance=0.01, z=0.001),
        # the same on a long packed batch with sigmoid scores and bf16 logits
        dict(name="route_grad_long", op="route_grad", T=32768, E=256, k=8, score=SIGMOID,
             dtype="bf16", renorm=True, scale=2.5, balance=0.01, z=0.0001),
        # gradient of the weighted sum, a small batch with fp32 expert rows
        dict(name="combine_grad_batch", op="combine_grad", T=64, k=4, H=4096, dtype="fp32",
             dropped=0.0),
        # the same for a prefill batch whose expert rows are bf16, some dropped by capacity
        dict(name="combine_grad_prefill", op="combine_grad", T=4096, k=8, H=2048, dtype="bf16",
             dropped=0.05),
        # one request decoding with its adapter on a square projection
        dict(name="lora_decode_one", op="lora", T=1, k=1, E=1, adapters=8, K=4096, N=4096, R=16,
             dtype="bf16", epilogue="raw", without=0.0, skew=0.0),
        # 64 requests decoding, each with its own adapter on every expert's gate and up
        dict(name="lora_decode_experts", op="lora", T=64, k=4, E=64, adapters=16, K=2048, N=1536,
             R=16, dtype="fp32", epilogue="swiglu", without=0.1, skew=0.5),
        # a mixed batch of decodes and short prompts of 40 adapters, fp32 rows
        dict(name="lora_mixed", op="lora", T=777, k=1, E=1, adapters=40, K=4096, N=4096, R=32,
             dtype="fp32", epilogue="raw", without=0.2, skew=1.5),
        # long prompts of eight adapters, wide rank and wide projection
        dict(name="lora_prefill", op="lora", T=8192, k=1, E=1, adapters=8, K=4096, N=11008, R=64,
             dtype="bf16", epilogue="raw", without=0.0, skew=0.7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A multiple of 64; past 1024 not of 1024 too."""
    n = _log(rng, lo // 64, hi // 64)
    return 64 * (n + 1 if n % 16 == 0 and n > 16 else n)


def draw(rng):
    op = rng.choice(["route", "route", "route_grad", "combine_grad", "lora", "lora"])
    if op in ("route", "route_grad"):
        groups = rng.choice([1, 1, 4, 8]) if op == "route" else 1
        E = groups * max(2, _log(rng, 8, 384) // groups)
        T = min(_log(rng, 1, 65536 if op == "route" else 32768),
                (65536 if op == "route" else 32768) * 256 // E)
        topk_groups = rng.randint(max(1, groups // 4), groups)
        k = rng.randint(1, min(8, topk_groups * (E // groups)))
        c = dict(op=op, T=T, E=E, k=k, score=rng.choice([SIGMOID, SOFTMAX]),
                 dtype=rng.choice(["fp32", "bf16"]), renorm=rng.random() < 0.75,
                 scale=rng.choice([1.0, 2.5]))
        if op == "route":
            return dict(c, groups=groups, topk_groups=topk_groups, group_top=rng.choice([1, 2]),
                        bias=rng.random() < 0.6, masked=rng.choice([0.0, 0.0, 0.2]))
        return dict(c, balance=rng.choice([0.0, 0.01, 0.1]), z=rng.choice([0.0, 0.001]))
    if op == "combine_grad":
        H = _width(rng, 128, 8064)
        k = rng.randint(1, 8)
        return dict(op=op, T=min(_log(rng, 1, 4096), 4096 * 8 * 2048 // (k * H)), k=k, H=H,
                    dtype=rng.choice(["fp32", "bf16"]), dropped=rng.choice([0.0, 0.1]))
    K, N, R = _width(rng, 256, 5440), _width(rng, 256, 5440), rng.choice([8, 16, 24, 32, 64])
    if rng.random() < 0.5:
        k = rng.randint(1, 4)
        return dict(op=op, T=_log(rng, 1, 256 // k), k=k, E=rng.choice([4, 24, 64]),
                    adapters=_log(rng, 1, 16), K=min(K, 2048), N=min(N, 1536), R=min(R, 32),
                    dtype=rng.choice(["fp32", "bf16"]) if rng.random() < 0.5 else "fp32",
                    epilogue="raw", without=rng.choice([0.0, 0.2]), skew=rng.uniform(0.0, 1.5))
    return dict(op=op, T=_log(rng, 1, 8192), k=1, E=1, adapters=_log(rng, 1, 16), K=K, N=N, R=R,
                dtype=rng.choice(["fp32", "bf16"]), epilogue=rng.choice(["raw", "raw", "swiglu"]),
                without=rng.choice([0.0, 0.2]), skew=rng.uniform(0.0, 1.5))


# ---- inputs ----------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _logits(g, case):
    """Router logits: a per-expert offset (some experts are popular) and noise."""
    T, E = case["T"], case["E"]
    l = _normal(g, T, E) * 1.2 + _normal(g, 1, E) * 0.5 - 0.5
    if case.get("masked", 0.0) > 0:  # experts that are offline for this batch
        l[:, torch.rand(E, generator=g, device="cuda") < case["masked"]] = -math.inf
        if T > 2:  # and a padding row that may use none
            l[T // 2] = -math.inf
    return l.to(DTYPES[case["dtype"]])


def _prepare_route(case, g):
    s = dict(logits=_logits(g, case))
    # a balance bias moves in steps of 0.001 while a model trains
    s["bias"] = torch.round(_normal(g, case["E"]) * 20) * 0.001 if case["bias"] else None
    return s


def _prepare_route_grad(case, g):
    T, E, k = case["T"], case["E"], case["k"]
    logits = _logits(g, case)
    # the ids the forward pass chose, with an empty slot now and then
    ids = torch.argsort(logits.float(), dim=1, descending=True, stable=True)[:, :k]
    ids = ids.to(torch.int32).contiguous()
    ids[T // 3, k - 1] = -1
    counts = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    flat = torch.where(ids < 0, E, ids).reshape(-1).long()
    counts.index_add_(0, flat, torch.ones_like(flat, dtype=torch.int32))
    return dict(logits=logits, ids=ids, counts=counts[:E].contiguous(),
                d_w=_normal(g, T, k) * (1.0 / T))


def _prepare_combine_grad(case, g):
    T, k, H = case["T"], case["k"], case["H"]
    A = T * k
    perm = torch.randperm(A, generator=g, device="cuda").to(torch.int32)
    drop = torch.rand(A, generator=g, device="cuda") < case["dropped"]
    w = torch.rand(T, k, generator=g, device="cuda")
    dt = DTYPES[case["dtype"]]
    return dict(d_out=_normal(g, T, H).to(torch.bfloat16), y=_normal(g, A, H).to(dt),
                inv_pos=torch.where(drop, -2, perm), w=w / w.sum(1, keepdim=True),
                k_dev=torch.full((1,), k, dtype=torch.int32, device="cuda"),
                d_y=torch.zeros(A, H, dtype=dt, device="cuda"))


def _prepare_lora(case, g):
    T, k, E, NA, K, N, R = (case[n] for n in ("T", "k", "E", "adapters", "K", "N", "R"))
    rows = T * k
    # requests of one adapter come in runs; popular adapters take more tokens
    pop = torch.arange(1, NA + 1, device="cuda", dtype=torch.float32) ** -case["skew"]
    adapter = torch.multinomial(pop, T, replacement=True, generator=g).to(torch.int32)
    adapter[torch.rand(T, generator=g, device="cuda") < case["without"]] = -1
    s = dict(adapter=adapter, scales=torch.rand(NA, generator=g, device="cuda") + 0.5)
    if E > 1:
        ids = torch.argsort(_normal(g, T, E), dim=1, descending=True)[:, :k]
        s["ids"] = ids.to(torch.int32).contiguous()
        flat = ids.reshape(-1)
        order = torch.argsort(flat, stable=True)
        s["sorted"] = order.to(torch.int32)
        s["offsets"] = torch.searchsorted(flat[order].contiguous(),
                                          torch.arange(E + 1, device="cuda")).to(torch.int32)
        s["k_dev"] = torch.full((1,), k, dtype=torch.int32, device="cuda")
        token, expert = order // k, flat[order]
    else:
        token = torch.arange(T, device="cuda")
        expert = torch.zeros_like(token)
    a = adapter.long()[token]
    s["slot"] = torch.where(a < 0, -1, a * E + expert)  # row -> adapter's weights, or -1
    s["token"] = token
    dt = DTYPES[case["dtype"]]
    s["x"] = _normal(g, T, K).to(torch.bfloat16)
    s["a"] = (_normal(g, NA * E, R, K) * K ** -0.5).to(torch.bfloat16).view(NA, E, R, K)
    s["b"] = (_normal(g, NA * E, N, R) * (0.3 * R ** -0.5)).to(torch.bfloat16).view(NA, E, N, R)
    s["base"] = _normal(g, rows, N).to(torch.float32 if case["epilogue"] == "swiglu" else dt)
    cols = N // 2 if case["epilogue"] == "swiglu" else N
    out_dt = torch.bfloat16 if case["epilogue"] == "swiglu" else dt
    s["out"] = torch.empty(rows, cols, dtype=out_dt, device="cuda")
    return s


def prepare(case, seed):
    make = dict(route=_prepare_route, route_grad=_prepare_route_grad,
                combine_grad=_prepare_combine_grad, lora=_prepare_lora)[case["op"]]
    return dict(make(case, _gen(seed)), case=case)


# ---- the plain forms -------------------------------------------------------


def _scores(l, score):
    """Scores in [0, 1]; an expert whose logit is not finite has none (0)."""
    on = torch.isfinite(l)
    if score == SIGMOID:
        return torch.where(on, 1.0 / (1.0 + torch.exp(-l)), 0.0), on
    l = torch.where(on, l, -math.inf)
    m = l.amax(dim=1, keepdim=True)
    e = torch.where(on, torch.exp(l - m), 0.0)
    # the sum over experts, neighbours first: the operator's summation order
    n = 1 << max(0, (l.shape[1] - 1).bit_length())
    t = torch.nn.functional.pad(e, (0, n - l.shape[1]))
    while t.shape[1] > 1:
        t = t[:, 0::2] + t[:, 1::2]
    return torch.where(on, e / t, 0.0), on


def _plain_route(s):
    c = s["case"]
    T, E, G = c["T"], c["E"], c["groups"]
    score, on = _scores(s["logits"].float(), c["score"])
    choice = score if s["bias"] is None else score + s["bias"]
    choice = torch.where(on, choice, -math.inf)
    if G > 1:
        grouped = choice.view(T, G, E // G)
        top = torch.sort(grouped, dim=2, descending=True).values[:, :, :c["group_top"]]
        value = torch.where(top == -math.inf, 0.0, top)
        value = value[:, :, 0] if c["group_top"] == 1 else value[:, :, 0] + value[:, :, 1]
        value = torch.where(top[:, :, 0] == -math.inf, -math.inf, value)
        best = torch.sort(value, dim=1, descending=True, stable=True).indices
        keep = torch.zeros(T, G, dtype=torch.bool, device=choice.device)
        keep.scatter_(1, best[:, :c["topk_groups"]], True)
        choice = torch.where(keep.unsqueeze(2), grouped, -math.inf).view(T, E)
    got, ids = torch.sort(choice, dim=1, descending=True, stable=True)
    got, ids = got[:, :c["k"]], ids[:, :c["k"]]
    w = torch.where(got == -math.inf, 0.0, torch.gather(score, 1, ids))
    if c["renorm"]:
        total = w.sum(dim=1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return [torch.where(got == -math.inf, -1, ids).to(torch.int32), w * c["scale"]]


def _plain_route_grad(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    l = s["logits"].float()
    score, on = _scores(l, c["score"])
    there = s["ids"] >= 0
    at = torch.where(there, s["ids"], 0).long()
    picked = torch.where(there, torch.gather(score, 1, at), 0.0)
    d_w = torch.where(there, s["d_w"], 0.0) * c["scale"]
    if c["renorm"]:
        total = picked.sum(dim=1, keepdim=True)
        dot = (d_w * picked).sum(dim=1, keepdim=True)
        d_p = torch.where(total > 0, (d_w - dot / total) / total, 0.0)
        d_p = torch.where(there, d_p, 0.0)
    else:
        d_p = d_w
    d_score = torch.zeros_like(score).scatter_add_(1, at, d_p)
    # balance loss: E / (k T) sum_e counts_e * mean_t q_te
    total = score.sum(dim=1, keepdim=True)
    q = torch.where(total > 0, score / total, 0.0)
    load = s["counts"].float() * (E / (k * T))
    balance = c["balance"] * (load * q.mean(dim=0)).sum()
    d_q = load * (c["balance"] / T)
    d_score = d_score + torch.where(
        total > 0, (d_q - (d_q * q).sum(dim=1, keepdim=True)) / total, 0.0)
    if c["score"] == SIGMOID:
        d_l = d_score * score * (1.0 - score)
    else:
        d_l = score * (d_score - (d_score * score).sum(dim=1, keepdim=True))
    # z loss: mean over tokens of the squared log-sum-exp of the logits
    some = on.any(dim=1, keepdim=True)
    m = torch.where(on, l, -math.inf).amax(dim=1, keepdim=True)
    e = torch.where(on, torch.exp(l - m), 0.0)
    lse = torch.where(some, m + torch.log(e.sum(dim=1, keepdim=True)), 0.0)
    z = c["z"] * (lse * lse).mean()
    p = torch.where(some, e / e.sum(dim=1, keepdim=True), 0.0)
    d_l = torch.where(on, d_l + (2.0 * c["z"] / T) * lse * p, 0.0)
    return [d_l.to(s["logits"].dtype), torch.stack([balance, z])]


def _plain_combine_grad(s):
    c = s["case"]
    T, k, H = c["T"], c["k"], c["H"]
    at = s["inv_pos"].long()
    kept = at >= 0
    d = s["d_out"].float().unsqueeze(1)
    y = s["y"].float()[torch.where(kept, at, 0)].view(T, k, H)
    d_w = torch.where(kept.view(T, k), (d * y).sum(dim=2), 0.0)
    rows = (s["w"].unsqueeze(2) * d).view(T * k, H)
    s["d_y"][at[kept]] = rows[kept].to(s["d_y"].dtype)
    return [d_w, s["d_y"]]


def _plain_lora(s):
    c = s["case"]
    rows, R, K, N = c["T"] * c["k"], c["R"], c["K"], c["N"]
    x, slot = s["x"].float()[s["token"]], s["slot"]
    there = slot >= 0
    at = torch.where(there, slot, 0)
    scale = torch.where(there, s["scales"][at // c["E"]], 0.0).unsqueeze(1)
    a, b = s["a"].float().view(-1, R, K), s["b"].float().view(-1, N, R)
    if rows <= 256:  # every row with its own adapter's matrices
        v = torch.bmm(a[at], x.unsqueeze(2)).squeeze(2) * scale
        delta = torch.bmm(b[at], v.unsqueeze(2)).squeeze(2)
    else:  # every row with all adapters, the others' products set to zero
        slots = a.shape[0]
        mine = (torch.arange(slots, device=slot.device) == slot.unsqueeze(1)).float() * scale
        v = (x @ a.view(slots * R, K).t()).view(rows, slots, R) * mine.unsqueeze(2)
        delta = v.view(rows, slots * R) @ b.permute(0, 2, 1).reshape(slots * R, N)
    y = s["base"].float() + delta
    if c["epilogue"] == "swiglu":
        gate, up = y[:, :N // 2], y[:, N // 2:]
        y = gate / (1.0 + torch.exp(-gate)) * up
    return y.to(s["out"].dtype)


# ---- the package's calls ---------------------------------------------------


def _own_route(s):
    import sparse_moe_expert_gb300 as moe
    c = s["case"]
    ids, w, _ = moe.moe_route_scored(
        s["logits"], c["k"], score=moe.SCORE_SIGMOID if c["score"] == SIGMOID else moe.SCORE_SOFTMAX,
        select_bias=s["bias"], n_groups=c["groups"], topk_groups=c["topk_groups"],
        group_top=c["group_top"], renormalize=c["renorm"], scale=c["scale"])
    return [ids, w]


def _own_route_grad(s):
    import sparse_moe_expert_gb300 as moe
    c = s["case"]
    d_logits, losses = moe.moe_route_scored_backward(
        s["logits"], s["ids"], s["d_w"], expert_counts=s["counts"],
        score=moe.SCORE_SIGMOID if c["score"] == SIGMOID else moe.SCORE_SOFTMAX,
        renormalize=c["renorm"], scale=c["scale"], balance_coef=c["balance"], z_coef=c["z"])
    return [d_logits, losses]


def _own_combine_grad(s):
    import sparse_moe_expert_gb300 as moe
    d_w, d_y = moe.moe_combine_backward(s["d_out"], s["y"], s["inv_pos"], s["w"], s["k_dev"],
                                        d_y=s["d_y"])
    return [d_w, d_y]


def _own_lora(s):
    import sparse_moe_expert_gb300 as moe
    c = s["case"]
    route = {}
    if c["E"] > 1:
        route = dict(topk_ids=s["ids"], sorted_assign=s["sorted"], expert_offsets=s["offsets"],
                     k_dev=s["k_dev"])
    return moe.moe_lora_apply(
        s["x"], s["adapter"], s["a"], s["b"], s["scales"], s["base"], out=s["out"],
        epilogue=moe.EPILOGUE_SWIGLU if c["epilogue"] == "swiglu" else moe.EPILOGUE_RAW, **route)


def run(state):
    op = state["case"]["op"]
    if own:
        return dict(route=_own_route, route_grad=_own_route_grad,
                    combine_grad=_own_combine_grad, lora=_own_lora)[op](state)
    return dict(route=_plain_route, route_grad=_plain_route_grad,
                combine_grad=_plain_combine_grad, lora=_plain_lora)[op](state)


# ---- bytes and operations --------------------------------------------------


def work(case):
    """Inputs read once and outputs written once.  For adapters: the expected
    number of different (adapter, expert) matrices that the rows need."""
    c, size = case, {"fp32": 4, "bf16": 2}[case["dtype"]]
    if c["op"] == "route":
        n = c["T"] * c["E"]
        return {"bytes": n * size + c["T"] * c["k"] * 8 + (4 * c["E"] if c["bias"] else 0) + 4,
                "flops": n * (8 + c["k"])}
    if c["op"] == "route_grad":
        n = c["T"] * c["E"]
        return {"bytes": 2 * n * size + c["T"] * c["k"] * 8 + 4 * c["E"] + 8, "flops": n * 24}
    if c["op"] == "combine_grad":
        A, kept = c["T"] * c["k"], 1.0 - c["dropped"]
        return {"bytes": int(2 * A * kept * c["H"] * size + c["T"] * c["H"] * 2 + A * 12),
                "flops": 3 * A * c["H"]}
    T, k, E, NA, K, N, R = (c[n] for n in ("T", "k", "E", "adapters", "K", "N", "R"))
    rows, served = T * k, T * k * (1.0 - c["without"])
    pop = [(a + 1) ** -c["skew"] for a in range(NA)]
    per = [served * p / sum(pop) / E for p in pop]  # mean rows of one (adapter, expert)
    slots = sum(E * (1.0 - math.exp(-m)) for m in per) if rows > 1 else 1
    base = 4 if c["epilogue"] == "swiglu" else size
    out = (N // 2) * 2 if c["epilogue"] == "swiglu" else N * size
    return {"bytes": int(T * K * 2 + slots * (K + N) * R * 2 + rows * (N * base + out) + T * 4),
            "flops": 2 * served * R * (K + N)}


# ---- 64 bits ---------------------------------------------------------------


def _exact_scores(l, score):
    on = torch.isfinite(l)
    if score == SIGMOID:
        return torch.where(on, torch.sigmoid(l), 0.0), on
    return torch.nan_to_num(torch.softmax(torch.where(on, l, -math.inf), dim=1), nan=0.0), on


def _exact_route(s):
    c = s["case"]
    T, E, G = c["T"], c["E"], c["groups"]
    score, on = _exact_scores(s["logits"].double(), c["score"])
    choice = score + (0.0 if s["bias"] is None else s["bias"].double())
    choice = choice.masked_fill(~on, -math.inf)
    if G > 1:
        left = choice.view(T, G, E // G).clone()
        value = left.amax(dim=2)
        if c["group_top"] == 2:
            left.scatter_(2, left.argmax(dim=2, keepdim=True), -math.inf)
            second = left.amax(dim=2)
            value = torch.where(torch.isinf(second), value, value + second)
        for _ in range(G - c["topk_groups"]):  # strike the weakest group, the last of equals
            worst = G - 1 - value.flip(1).argmin(dim=1)
            value[torch.arange(T, device=value.device), worst] = math.inf
        choice = choice.view(T, G, E // G).masked_fill((value == math.inf).unsqueeze(2),
                                                       -math.inf).view(T, E)
    w = torch.zeros(T, c["k"], dtype=torch.float64, device=choice.device)
    for j in range(c["k"]):
        top = choice.amax(dim=1, keepdim=True)
        at = (choice == top).to(torch.uint8).argmax(dim=1, keepdim=True)
        w[:, j:j + 1] = torch.where(torch.isinf(top), 0.0, torch.gather(score, 1, at))
        choice.scatter_(1, at, -math.inf)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True).clamp_min(1e-300)
    return [None, w * c["scale"]]


def _exact_route_grad(s):
    """Automatic differentiation of the losses and of sum(d_w * w)."""
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    l = s["logits"].double().requires_grad_()
    score, _ = _exact_scores(l, c["score"])
    there = s["ids"] >= 0
    w = torch.gather(score, 1, s["ids"].clamp_min(0).long()) * there
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True).clamp_min(1e-300)
    gate = (w * c["scale"] * s["d_w"].double()).sum()
    q = score / score.sum(dim=1, keepdim=True)
    balance = c["balance"] * E / (k * T) * (s["counts"].double() * q.mean(dim=0)).sum()
    z = c["z"] * torch.logsumexp(l, dim=1).square().mean()
    (gate + balance + z).backward()
    return [l.grad, torch.stack([balance, z]).detach()]


def _exact_combine_grad(s):
    c = s["case"]
    T, k, H = c["T"], c["k"], c["H"]
    d = s["d_out"].double()
    d_w = torch.zeros(T, k, dtype=torch.float64, device=d.device)
    d_y = torch.zeros(T * k, H, dtype=torch.float64, device=d.device)
    at = s["inv_pos"].view(T, k)
    for j in range(k):
        t = torch.nonzero(at[:, j] >= 0).squeeze(1)
        r = at[t, j].long()
        d_w[t, j] = torch.einsum("th,th->t", d[t], s["y"][r].double())
        d_y[r] = s["w"][t, j].double().unsqueeze(1) * d[t]
    return [d_w, d_y]


def _exact_lora(s):
    c = s["case"]
    R, K, N = c["R"], c["K"], c["N"]
    y = s["base"].double()
    a, b = s["a"].view(-1, R, K), s["b"].view(-1, N, R)
    for slot in torch.unique(s["slot"]).tolist():
        if slot < 0:
            continue
        r = torch.nonzero(s["slot"] == slot).squeeze(1)
        v = s["x"][s["token"][r]].double() @ a[slot].double().t()
        y[r] += s["scales"][slot // c["E"]].double() * (v @ b[slot].double().t())
    if c["epilogue"] == "swiglu":
        y = torch.nn.functional.silu(y[:, :N // 2]) * y[:, N // 2:]
    return y


def exact(case, seed):
    s = prepare(case, seed)
    return dict(route=_exact_route, route_grad=_exact_route_grad,
                combine_grad=_exact_combine_grad, lora=_exact_lora)[case["op"]](s)
