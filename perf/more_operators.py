"""Operators measured beside the layer: normalisation with its gradient, a dense
product with bias, activation and residual with its gradient, and the AdamW
step over many tensors.

``own`` false runs each operator in elementary torch operations in 32 bits;
``own`` true makes the package's calls.  Cases are plain dicts; ``prepare``
makes the inputs a serving or training program has in hand.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
NONE, SILU, GELU, SWIGLU = "none", "silu", "gelu", "swiglu"
BLOCK = 256  # consecutive elements of a tensor that share a scale of the 8-bit states


def listed():
    return [
        # one token of a decode loop: the layer's input plus the residual stream, RMS norm
        dict(name="norm_decode", op="norm", T=1, H=4096, kind="rms", dtype="bf16", residual=True,
             bias=False),
        # a long prompt: layer norm with weight and bias
        dict(name="norm_prefill", op="norm", T=8192, H=4096, kind="layer", dtype="bf16",
             residual=False, bias=True),
        # gradient of a small fine-tuning batch, fp32 activations
        dict(name="norm_grad_batch", op="norm_grad", T=64, H=2048, kind="layer", dtype="fp32",
             d_sum=False),
        # gradient of a packed batch; the sum of input and residual has a gradient of its own too
        dict(name="norm_grad_long", op="norm_grad", T=16384, H=4096, kind="rms", dtype="bf16",
             d_sum=True),
        # one token through a shared expert's gate and up, as wide as the decode workload's experts
        dict(name="linear_decode", op="linear", T=1, K=4096, N=22016, act=SWIGLU, bias=False,
             residual=False, save=False),
        # 64 tokens through a shared expert's down product, added to the routed experts' sum
        dict(name="linear_batch", op="linear", T=64, K=1536, N=4096, act=NONE, bias=False,
             residual=True, save=False),
        # a prompt through gate and up of a small shared expert, pre-activations kept for training
        dict(name="linear_prefill", op="linear", T=4096, K=2048, N=1536, act=SWIGLU, bias=False,
             residual=False, save=True),
        # a ragged prompt through a wide projection with bias, activation and residual
        dict(name="linear_ragged", op="linear", T=3001, K=11008, N=4096, act=GELU, bias=True,
             residual=True, save=False),
        # gradient of a small batch through a projection with bias and activation
        dict(name="linear_grad_batch", op="linear_grad", T=777, K=4096, N=1536, act=SILU, bias=True),
        # gradient of a prompt-sized batch through a wide shared expert's gate and up
        dict(name="linear_grad_prefill", op="linear_grad", T=4096, K=4096, N=11008, act=SWIGLU,
             bias=False),
        # router, its balance of norms and a few vectors, fp32 states: a small step
        dict(name="adamw_router", op="adamw", count=12, least=64, most=262144, bits=32,
             param="fp32", grad="fp32", scaled=False),
        # adapters of many projections, bf16 weights with fp32 masters, states in 8 bits
        dict(name="adamw_adapters", op="adamw", count=400, least=1024, most=1048576, bits=8,
             param="bf16", grad="bf16", scaled=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "linear", "linear", "linear_grad", "linear_grad", "adamw"])
    if op in ("norm", "norm_grad"):
        H = _log(rng, 48, 8192)
        c = dict(op=op, T=min(_log(rng, 1, 16384), 16384 * 4096 // H), H=H,
                 kind=rng.choice(["rms", "layer"]), dtype=rng.choice(["bf16", "bf16", "fp32"]))
        if op == "norm":
            return dict(c, residual=rng.random() < 0.5, bias=rng.random() < 0.5)
        return dict(c, T=min(c["T"], 8192) if c["dtype"] == "fp32" else c["T"],
                    d_sum=rng.random() < 0.5)
    if op in ("linear", "linear_grad"):
        K, act = 8 * _log(rng, 8, 1376), rng.choice([NONE, SILU, GELU, SWIGLU])
        N = _log(rng, 40, 11008)
        if act == SWIGLU:
            N += N % 2
        T = min(_log(rng, 1, 4096), 3001 * 11008 * 4096 // (K * N))
        c = dict(op=op, T=T, K=K, N=N, act=act, bias=rng.random() < 0.5)
        if op == "linear_grad":
            return c
        return dict(c, residual=rng.random() < 0.5, save=act != NONE and rng.random() < 0.3)
    most = _log(rng, 64, 1048576)
    count = min(_log(rng, 1, 400), max(1, 100_000_000 // most))
    return dict(op=op, count=count, least=rng.choice([1, 17, 64]), most=most,
                bits=rng.choice([32, 8]), param=rng.choice(["fp32", "bf16"]),
                grad=rng.choice(["fp32", "bf16"]), scaled=rng.random() < 0.5)


# ---- inputs ----------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, T, H):
    """Rows of a residual stream: each token has a size and an offset of its
    own, and a few channels are much larger than the others."""
    size = torch.exp(0.5 * _normal(g, T, 1))
    channel = torch.where(torch.rand(1, H, generator=g, device="cuda") < 0.005, 12.0, 1.0)
    return _normal(g, T, H) * size * channel + 0.1 * _normal(g, T, 1)


def _prepare_norm(case, g):
    T, H, dt = case["T"], case["H"], DTYPES[case["dtype"]]
    return dict(x=_activations(g, T, H).to(dt), weight=1.0 + 0.2 * _normal(g, H),
                bias=0.1 * _normal(g, H) if case["bias"] else None,
                residual=_activations(g, T, H).to(dt) if case["residual"] else None)


def _prepare_norm_grad(case, g):
    T, H, dt = case["T"], case["H"], DTYPES[case["dtype"]]
    x = _activations(g, T, H).to(dt)
    f = x.float()
    # the statistics as the forward pass left them
    mean = f.mean(dim=1) if case["kind"] == "layer" else None
    d = f if mean is None else f - mean.unsqueeze(1)
    rstd = torch.rsqrt((d * d).mean(dim=1) + 1e-6)
    return dict(x=x, mean=mean, rstd=rstd, weight=1.0 + 0.2 * _normal(g, H),
                d_out=(_normal(g, T, H) / T).to(dt),
                d_sum=(_normal(g, T, H) / T).to(dt) if case["d_sum"] else None)


def _prepare_linear(case, g):
    T, K, N = case["T"], case["K"], case["N"]
    cols = N // 2 if case["act"] == SWIGLU else N
    return dict(x=_normal(g, T, K).to(torch.bfloat16),
                w=(_normal(g, N, K) * K ** -0.5).to(torch.bfloat16),
                bias=0.2 * _normal(g, N) if case["bias"] else None,
                residual=_normal(g, T, cols).to(torch.bfloat16) if case["residual"] else None)


def _prepare_linear_grad(case, g):
    T, N = case["T"], case["N"]
    cols = N // 2 if case["act"] == SWIGLU else N
    s = _prepare_linear(dict(case, residual=False), g)
    # pre-activations as the forward pass kept them
    s["preact"] = None if case["act"] == NONE else _normal(g, T, N).to(torch.bfloat16)
    s["d_out"] = (_normal(g, T, cols) / T).to(torch.bfloat16)
    return s


def _sizes(case):
    """Sizes of a model's tensors: from vectors to matrices, odd ones among them."""
    n, lo, hi = case["count"], case["least"], case["most"]
    if n == 1:
        return [hi]
    out = [int(round(lo * (hi / lo) ** (i / (n - 1)))) for i in range(n)]
    return [out[(i * 7) % n] if n % 7 else out[i] for i in range(n)]  # not in order of size


def _views(flat, sizes):
    """The tensors of one flat buffer, each on a 64-byte boundary or better."""
    out, at = [], 0
    for n in sizes:
        out.append(flat[at:at + n])
        at += -(-n // 64) * 64
    return out


def _prepare_adamw(case, g):
    sizes = _sizes(case)
    total = sum(-(-n // 64) * 64 for n in sizes)
    master = 0.02 * _normal(g, total)
    # gradients of popular and of rare rows differ by orders of magnitude
    scale = 1e-3 * torch.exp(2.0 * _normal(g, total // 64)).repeat_interleave(64)
    grad = _normal(g, total) * scale
    m, v = 0.3 * scale * _normal(g, total), (scale * (0.5 + torch.rand(
        total, generator=g, device="cuda"))) ** 2
    s = dict(sizes=sizes, flat_master=master, flat_grad=grad.to(DTYPES[case["grad"]]))
    s["flat_param"] = master if case["param"] == "fp32" else master.to(torch.bfloat16)
    s["params"], s["grads"] = _views(s["flat_param"], sizes), _views(s["flat_grad"], sizes)
    s["masters"] = None if case["param"] == "fp32" else _views(master, sizes)
    s["scale"] = torch.full((1,), 0.37, device="cuda") if case["scaled"] else None
    s["decay"] = [0.0 if n < 4096 else 0.1 for n in sizes]
    s["step"] = torch.tensor([100, 0], dtype=torch.int32, device="cuda")
    if case["bits"] == 32:
        s["flat_m"], s["flat_v"] = m, v
        s["m"], s["v"] = _views(m, sizes), _views(v, sizes)
        return s
    s["m"], s["v"], s["m_scale"], s["v_scale"] = [], [], [], []
    for a, b in zip(_views(m, sizes), _views(v, sizes)):
        code, sc = _encode_m(a)
        s["m"].append(code)
        s["m_scale"].append(sc)
        code, sc = _encode_v(torch.sqrt(b), b)
        s["v"].append(code)
        s["v_scale"].append(sc)
    return s


def prepare(case, seed):
    make = dict(norm=_prepare_norm, norm_grad=_prepare_norm_grad, linear=_prepare_linear,
                linear_grad=_prepare_linear_grad, adamw=_prepare_adamw)[case["op"]]
    return dict(make(case, _gen(seed)), case=case)


# ---- the plain forms -------------------------------------------------------


def _plain_norm(s):
    c = s["case"]
    x = s["x"]
    if s["residual"] is not None:  # the sum that the next layer adds to is stored, and normed
        x = (x.float() + s["residual"].float()).to(x.dtype)
    f = x.float()
    mean = f.mean(dim=1) if c["kind"] == "layer" else None
    d = f if mean is None else f - mean.unsqueeze(1)
    rstd = 1.0 / torch.sqrt((d * d).mean(dim=1) + 1e-6)
    y = d * rstd.unsqueeze(1) * s["weight"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return [y.to(x.dtype), x if s["residual"] is not None else None, mean, rstd]


def _plain_norm_grad(s):
    d, f = s["d_out"].float(), s["x"].float()
    xh = f if s["mean"] is None else f - s["mean"].unsqueeze(1)
    xh = xh * s["rstd"].unsqueeze(1)
    c = d * s["weight"]
    d_x = c - xh * (c * xh).mean(dim=1, keepdim=True)
    if s["mean"] is not None:
        d_x = d_x - c.mean(dim=1, keepdim=True)
    d_x = d_x * s["rstd"].unsqueeze(1)
    if s["d_sum"] is not None:
        d_x = d_x + s["d_sum"].float()
    return [d_x.to(s["x"].dtype), (d * xh).sum(dim=0), d.sum(dim=0)]


def _activation(z, act):
    if act == SILU:
        return z / (1.0 + torch.exp(-z))
    if act == GELU:
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == SWIGLU:
        n = z.shape[1] // 2
        return z[:, :n] / (1.0 + torch.exp(-z[:, :n])) * z[:, n:]
    return z


def _slope(z, act):
    """Derivative of SiLU or GELU."""
    if act == GELU:
        return (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi)))
    s = 1.0 / (1.0 + torch.exp(-z))
    return s * (1.0 + z * (1.0 - s))


def _plain_linear(s):
    c = s["case"]
    z = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _activation(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return [y.to(torch.bfloat16), z.to(torch.bfloat16) if c["save"] else None]


def _plain_linear_grad(s):
    c = s["case"]
    d, n = s["d_out"].float(), c["N"] // 2
    if c["act"] != NONE:
        z = s["preact"].float()
        if c["act"] == SWIGLU:
            g, u = z[:, :n], z[:, n:]
            d = torch.cat([d * u * _slope(g, SILU), d * (g / (1.0 + torch.exp(-g)))], dim=1)
        else:
            d = d * _slope(z, c["act"])
    d_bias = d.sum(dim=0) if c["bias"] else None
    # the gradient of the pre-activations is kept in their type, and multiplied from there
    d_pre = d.to(torch.bfloat16)
    f = d_pre.float()
    return [(f @ s["w"].float()).to(torch.bfloat16), (f.t() @ s["x"].float()).to(torch.bfloat16),
            d_bias, d_pre]


def _blocks(t, fill=0.0):
    n = t.numel()
    return torch.nn.functional.pad(t, (0, -n % BLOCK), value=fill).view(-1, BLOCK)


def _encode_m(m):
    """Sign and 127 sqrt(|m| / largest |m| of the block)."""
    b = _blocks(m)
    s = b.abs().amax(dim=1, keepdim=True)
    inv = torch.where(s > 0, 1.0 / s, 0.0)
    code = torch.round(torch.sqrt(b.abs() * inv) * 127.0) * torch.sign(b)
    return code.to(torch.int8).view(-1)[:m.numel()], s.view(-1)


def _encode_v(r, v):
    """255 sqrt(r / largest r of the block) of r = sqrt(v); 1 at least where v > 0."""
    b = _blocks(r)
    s = b.amax(dim=1, keepdim=True)
    inv = torch.where(s > 0, 1.0 / s, 0.0)
    code = torch.round(torch.sqrt(b * inv) * 255.0)
    code = torch.where(_blocks(v) > 0, code.clamp_min(1.0), 0.0)
    return code.to(torch.uint8).view(-1)[:r.numel()], s.view(-1)


def _decode_m(code, scale):
    a = _blocks(code.float()) * (1.0 / 127.0)
    return (a * a.abs() * scale.view(-1, 1)).view(-1)[:code.numel()]


def _decode_r(code, scale):
    a = _blocks(code.float()) * (1.0 / 255.0)
    return (a * a * scale.view(-1, 1)).view(-1)[:code.numel()]


LR, B1, B2, EPS = 1e-3, 0.9, 0.999, 1e-8


def _plain_adamw(s):
    c = s["case"]
    masters = s["params"] if s["masters"] is None else s["masters"]
    s["step"][:1] += 1
    t = s["step"][:1].double()
    inv_bc1 = (1.0 / (1.0 - B1 ** t)).float()
    inv_r2 = (1.0 / torch.sqrt(1.0 - B2 ** t)).float()
    values = [[], []]
    for i, p in enumerate(masters):
        g = s["grads"][i].float()
        if s["scale"] is not None:
            g = g * s["scale"]
        if c["bits"] == 32:
            m, v = s["m"][i], s["v"][i]
        else:
            m = _decode_m(s["m"][i], s["m_scale"][i])
            v = _decode_r(s["v"][i], s["v_scale"][i])
            v = v * v
        m = m * B1 + g * (1.0 - B1)
        v = v * B2 + g * g * (1.0 - B2)
        r = torch.sqrt(v)
        step = m * inv_bc1 / (r * inv_r2 + EPS)
        p.copy_(p * (1.0 - LR * s["decay"][i]) - step * LR)
        if s["masters"] is not None:
            s["params"][i].copy_(p)
        if c["bits"] == 32:
            s["m"][i].copy_(m)
            s["v"][i].copy_(v)
            continue
        code, scale = _encode_m(m)
        s["m"][i].copy_(code)
        s["m_scale"][i].copy_(scale)
        values[0].append(_decode_m(code, scale))
        code, scale = _encode_v(r, v)
        s["v"][i].copy_(code)
        s["v_scale"][i].copy_(scale)
        r = _decode_r(code, scale)
        values[1].append(r * r)
    if c["bits"] == 32:
        return [s["flat_param"], s["flat_master"], s["flat_m"], s["flat_v"]]
    return [s["flat_param"], s["flat_master"], torch.cat(values[0]), torch.cat(values[1])]


# ---- the package's calls ---------------------------------------------------


def _act(moe, name):
    return {NONE: moe.ACT_NONE, SILU: moe.ACT_SILU, GELU: moe.ACT_GELU,
            SWIGLU: moe.ACT_SWIGLU}[name]


def _own_norm(s):
    import sparse_moe_expert_gb300 as moe
    kind = moe.NORM_RMS if s["case"]["kind"] == "rms" else moe.NORM_LAYER
    return list(moe.moe_layer_norm(s["x"], s["weight"], s["bias"], residual=s["residual"],
                                   eps=1e-6, kind=kind, need_stats=True))


def _own_norm_grad(s):
    import sparse_moe_expert_gb300 as moe
    kind = moe.NORM_RMS if s["case"]["kind"] == "rms" else moe.NORM_LAYER
    return list(moe.moe_layer_norm_backward(s["d_out"], s["x"], s["rstd"], s["mean"], s["weight"],
                                            d_sum=s["d_sum"], kind=kind))


def _own_linear(s):
    import sparse_moe_expert_gb300 as moe
    c = s["case"]
    out, preact = moe.moe_linear(s["x"], s["w"], s["bias"], residual=s["residual"],
                                 activation=_act(moe, c["act"]), need_preact=c["save"])
    return [out, preact]


def _own_linear_grad(s):
    import sparse_moe_expert_gb300 as moe
    c = s["case"]
    return list(moe.moe_linear_backward(s["d_out"], s["x"], s["w"], s["preact"],
                                        activation=_act(moe, c["act"]), need_d_bias=c["bias"],
                                        d_w_dtype=torch.bfloat16))


def _own_adamw(s):
    import sparse_moe_expert_gb300 as moe
    eight = s["case"]["bits"] == 8
    scales = dict(exp_avg_scales=s["m_scale"], exp_avg_sq_scales=s["v_scale"]) if eight else {}
    moe.moe_adamw_step(s["params"], s["grads"], s["m"], s["v"], s["step"], lr=LR, beta1=B1,
                       beta2=B2, eps=EPS, weight_decay=s["decay"], masters=s["masters"],
                       grad_scale=s["scale"], **scales)
    if not eight:
        return [s["flat_param"], s["flat_master"], s["flat_m"], s["flat_v"]]
    m, v = moe.moe_adamw_values(s["m"], s["v"], **scales)
    return [s["flat_param"], s["flat_master"], m, v]


def run(state):
    op = state["case"]["op"]
    if own:
        return dict(norm=_own_norm, norm_grad=_own_norm_grad, linear=_own_linear,
                    linear_grad=_own_linear_grad, adamw=_own_adamw)[op](state)
    return dict(norm=_plain_norm, norm_grad=_plain_norm_grad, linear=_plain_linear,
                linear_grad=_plain_linear_grad, adamw=_plain_adamw)[op](state)


# ---- bytes and operations --------------------------------------------------


def work(case):
    """Inputs read once and outputs written once."""
    c = case
    if c["op"] == "norm":
        n, size = c["T"] * c["H"], DTYPES[c["dtype"]].itemsize
        stats = 4 * c["T"] * (2 if c["kind"] == "layer" else 1)
        return {"bytes": n * size * (4 if c["residual"] else 2) + stats
                + 4 * c["H"] * (2 if c["bias"] else 1), "flops": 8 * n}
    if c["op"] == "norm_grad":
        n, size = c["T"] * c["H"], DTYPES[c["dtype"]].itemsize
        stats = 4 * c["T"] * (2 if c["kind"] == "layer" else 1)
        return {"bytes": n * size * (4 if c["d_sum"] else 3) + stats + 12 * c["H"], "flops": 12 * n}
    if c["op"] == "linear":
        T, K, N = c["T"], c["K"], c["N"]
        cols = N // 2 if c["act"] == SWIGLU else N
        return {"bytes": 2 * (T * K + N * K + T * cols * (2 if c["residual"] else 1)
                              + (T * N if c["save"] else 0)) + (4 * N if c["bias"] else 0),
                "flops": 2 * T * K * N}
    if c["op"] == "linear_grad":
        T, K, N = c["T"], c["K"], c["N"]
        cols = N // 2 if c["act"] == SWIGLU else N
        pre = 0 if c["act"] == NONE else T * N
        return {"bytes": 2 * (2 * T * K + 2 * N * K + T * cols + 2 * pre)
                + (4 * N if c["bias"] else 0), "flops": 4 * T * K * N}
    n = sum(_sizes(c))
    param = 8 if c["param"] == "fp32" else 8 + 2
    state = 16 if c["bits"] == 32 else 4 + 16 / BLOCK + 8  # and the values handed out
    return {"bytes": int(n * (param + DTYPES[c["grad"]].itemsize + state)), "flops": 16 * n}


# ---- 64 bits ---------------------------------------------------------------


def _exact_norm(s):
    c = s["case"]
    x = s["x"].double()
    total = None
    if s["residual"] is not None:
        total = (x + s["residual"].double()).to(s["x"].dtype)  # held in the input's type
        x = total.double()
    if c["kind"] == "layer":
        var, mean = torch.var_mean(x, dim=1, unbiased=False)
    else:
        var, mean = x.square().sum(dim=1) / c["H"], None
    rstd = (var + 1e-6).pow(-0.5)
    y = torch.einsum("th,t,h->th", x if mean is None else x - mean[:, None], rstd,
                     s["weight"].double())
    if s["bias"] is not None:
        y += s["bias"].double()
    return [y, total, mean, rstd]


def _exact_norm_grad(s):
    """With the statistics as given: the gradient's projections in 64 bits."""
    H = s["case"]["H"]
    d, r = s["d_out"].double(), s["rstd"].double()[:, None]
    centre = 0.0 if s["mean"] is None else s["mean"].double()[:, None]
    xh = (s["x"].double() - centre) * r
    c = d * s["weight"].double()
    along = torch.einsum("th,th->t", c, xh)[:, None] / H
    d_x = r * (c - xh * along)
    if s["mean"] is not None:
        d_x -= r * (c.sum(dim=1, keepdim=True) / H)
    if s["d_sum"] is not None:
        d_x += s["d_sum"].double()
    return [d_x, torch.einsum("th,th->h", d, xh), torch.einsum("th->h", d)]


def _exact_linear(s):
    c = s["case"]
    z = torch.nn.functional.linear(s["x"].double(), s["w"].double(),
                                   None if s["bias"] is None else s["bias"].double())
    if c["act"] == SWIGLU:
        gate, up = z.chunk(2, dim=1)
        y = torch.nn.functional.silu(gate) * up
    else:
        y = {NONE: lambda t: t, SILU: torch.nn.functional.silu,
             GELU: torch.nn.functional.gelu}[c["act"]](z)
    if s["residual"] is not None:
        y = y + s["residual"].double()
    return [y, z if c["save"] else None]


def _exact_linear_grad(s):
    """Automatic differentiation of the activation; then the products."""
    c = s["case"]
    d_pre = s["d_out"].double()
    if c["act"] != NONE:
        z = s["preact"].double().requires_grad_()
        if c["act"] == SWIGLU:
            y = torch.nn.functional.silu(z[:, :c["N"] // 2]) * z[:, c["N"] // 2:]
        else:
            y = (torch.nn.functional.gelu if c["act"] == GELU else torch.nn.functional.silu)(z)
        d_pre, = torch.autograd.grad(y, z, d_pre)
    held = d_pre.to(torch.bfloat16).double()  # held in the pre-activations' type
    return [torch.mm(held, s["w"].double()), torch.mm(held.t(), s["x"].double()),
            torch.einsum("tn->n", d_pre) if c["bias"] else None, held.to(torch.float32)
            if c["act"] == NONE else d_pre]


def _exact_adamw(s):
    c = s["case"]
    t = int(s["step"][0]) + 1
    flat = [s["flat_param"].double(), s["flat_master"].double()]
    states = [[], []]
    if c["bits"] == 32:
        flat += [s["flat_m"].double(), s["flat_v"].double()]
    places = [_views(f, s["sizes"]) for f in flat]
    for i, n in enumerate(s["sizes"]):
        g = s["grads"][i].double()
        if s["scale"] is not None:
            g = g * float(s["scale"])
        if c["bits"] == 32:
            m, v = s["m"][i].double(), s["v"][i].double()
        else:
            at = torch.arange(n, device=g.device) // BLOCK
            q, r = s["m"][i].double() / 127, s["v"][i].double() / 255
            m = q.sign() * q.square() * s["m_scale"][i].double()[at]
            v = (r.square() * s["v_scale"][i].double()[at]).square()
        m, v = torch.lerp(g, m, B1), torch.lerp(g.square(), v, B2)
        p = places[1][i]
        new = p - LR * s["decay"][i] * p - LR * (m / (1 - B1 ** t)) / (
            (v / (1 - B2 ** t)).sqrt() + EPS)
        places[0][i].copy_(new)
        places[1][i].copy_(new)
        if c["bits"] == 32:
            places[2][i].copy_(m)
            places[3][i].copy_(v)
            continue
        top_m, top_r = torch.zeros_like(s["m_scale"][i]).double(), torch.zeros_like(
            s["v_scale"][i]).double()
        top_m.scatter_reduce_(0, at, m.abs(), "amax")
        top_r.scatter_reduce_(0, at, v.sqrt(), "amax")
        q = (m.abs() / top_m[at].clamp_min(1e-300)).sqrt().mul(127).round()
        r = (v.sqrt() / top_r[at].clamp_min(1e-300)).sqrt().mul(255).round()
        r = torch.where(v > 0, r.clamp_min(1), 0)
        states[0].append(m.sign() * (q / 127).square() * top_m[at])
        states[1].append(((r / 255).square() * top_r[at]).square())
    if c["bits"] == 32:
        return flat
    return flat + [torch.cat(states[0]), torch.cat(states[1])]


def exact(case, seed):
    s = prepare(case, seed)
    return dict(norm=_exact_norm, norm_grad=_exact_norm_grad, linear=_exact_linear,
                linear_grad=_exact_linear_grad, adamw=_exact_adamw)[case["op"]](s)
