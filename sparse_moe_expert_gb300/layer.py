"""MoELayer: the six C-ABI calls composed into one quantized SwitchGLU MoE layer.

Pages: "Qwen3.5 Block在llama.cpp中的映射与优化原理" section 4 (router, then
only the chosen experts' FFN, then the weighted sum); "oMLX MoE gate/up 融合
优化：qwen35_moe_gate_up 实现剖析" (gate and up fused once at load, one
gate_up product per layer; the environment switch turns fusion off).
"""
from __future__ import annotations

import dataclasses
import os
from typing import Optional

import numpy as np
import torch

from . import binding as B
from ._lib import (ACT_SWIGLU, EPILOGUE_RAW, EPILOGUE_SWIGLU, NORM_LAYER, NORM_MAX_WIDTH, NORM_RMS,
                   PATH_AUTO, PATH_FLAG_WEIGHTS_EARLY, PATH_GEMV, PATH_TC, SCORE_SIGMOID,
                   SCORE_SOFTMAX, MoEError, path_k_range)

FUSE_ENV = "MOE_GB300_FUSE_GATE_UP"
TC_MIN_TOKENS_PER_EXPERT = 24  # mirrors the library's automatic path choice
TC_BUILT = True                # the tensor-core grouped GEMM (tcgen05) is available


@dataclasses.dataclass
class QTensor:
    """Affine-quantized weights of E experts on the device."""
    q: torch.Tensor  # uint32 [E, rows, cols*bits/32]
    s: torch.Tensor  # float16 [E, rows, cols/64]
    b: torch.Tensor  # float16 [E, rows, cols/64]
    bits: int

    @property
    def rows(self) -> int:
        return self.q.shape[1]

    @property
    def cols(self) -> int:
        return self.q.shape[2] * 32 // self.bits


def qtensor_from_numpy(m, device) -> QTensor:
    """Upload a workloads.QuantMatrix (numpy) to the device."""
    q = torch.from_numpy(np.ascontiguousarray(m.q)).to(device)
    s = torch.from_numpy(np.ascontiguousarray(m.s)).to(device)
    b = torch.from_numpy(np.ascontiguousarray(m.b)).to(device)
    return QTensor(q, s, b, m.bits)


def bf16_from_bits(x_bits: np.ndarray, device=None, pin: bool = False) -> torch.Tensor:
    t = torch.from_numpy(np.ascontiguousarray(x_bits, dtype=np.uint16)).view(torch.bfloat16)
    if pin:
        t = t.pin_memory()
    return t.to(device) if device is not None else t


@dataclasses.dataclass
class ScoredRouting:
    """How a layer turns router logits into experts (moe_route_scored).

    ``select_bias`` (fp32 [E], on the device) steers the selection and does
    not weigh; with ``n_groups`` > 1 the experts of the ``topk_groups`` best
    groups compete, a group ranking by the sum of its ``group_top`` best."""
    score: int = SCORE_SOFTMAX
    select_bias: Optional[torch.Tensor] = None
    n_groups: int = 1
    topk_groups: int = 1
    group_top: int = 2
    scale: float = 1.0


@dataclasses.dataclass
class ExpertAdapters:
    """Low-rank adapters of many requests on every expert (moe_lora_apply).

    gate_up_a bf16 [n, E, R, H], gate_up_b bf16 [n, E, 2*I, R] and down_a bf16
    [n, E, R', I], down_b bf16 [n, E, H, R'] (either pair may be None); scales
    fp32 [n] or None."""
    gate_up_a: Optional[torch.Tensor] = None
    gate_up_b: Optional[torch.Tensor] = None
    down_a: Optional[torch.Tensor] = None
    down_b: Optional[torch.Tensor] = None
    scales: Optional[torch.Tensor] = None

    @staticmethod
    def join_gate_up(gate_a, gate_b, up_a, up_b):
        """(gate_up_a, gate_up_b) of separate gate and up adapters: the two
        ranks side by side, each half of B reading its own (rank doubled)."""
        a = torch.cat([gate_a, up_a], dim=-2).contiguous()
        r, r2 = gate_b.shape[-1], up_b.shape[-1]
        top = torch.nn.functional.pad(gate_b, (0, r2))
        low = torch.nn.functional.pad(up_b, (r, 0))
        return a, torch.cat([top, low], dim=-2).contiguous()


@dataclasses.dataclass
class Norm:
    """A norm of the block around the layer (moe_layer_norm): weight and bias
    [H], fp32 or bf16, either may be None; kind NORM_RMS or NORM_LAYER.  H is at
    most NORM_MAX_WIDTH."""
    weight: Optional[torch.Tensor] = None
    bias: Optional[torch.Tensor] = None
    kind: int = NORM_RMS
    eps: float = 1e-6


@dataclasses.dataclass
class SharedExpert:
    """A dense SwiGLU expert that every token passes beside the routed ones
    (moe_linear): gate_up bf16 [2*I', H] (gate rows first), down bf16 [H, I']."""
    gate_up: torch.Tensor
    down: torch.Tensor


class MoELayer:
    """Forward of one quantized sparse-MoE SwitchGLU layer on one GPU.

    k_fixed > 0 routes every token to k experts; k_fixed = 0 applies the
    batch-entropy rule (k in {1, 2, 3}, kmax = 3).  ``fuse_gate_up`` (default:
    the environment variable MOE_GB300_FUSE_GATE_UP, on unless "0") packs
    gate and up once here; unfused layers run two RAW products plus the
    separate activation.  ``path`` forces a kernel family for the products.
    ``groups`` > 0 routes each token to the best expert of each of ``groups``
    groups of consecutive expert ids (k_fixed must equal it).  ``capacity``
    limits the assignments each expert takes per call (the lowest token
    slots stay; the others are dropped).  ``y_dtype`` is the storage type of
    the down product's rows between the down and combine kernels: None
    stores bf16 when a call's products run on the tensor cores (large
    batches, where y is hundreds of MB written and read again) and fp32
    otherwise.  ``scoring`` routes by scores (ScoredRouting) instead of the
    plain softmax top-k; it needs a fixed k and takes the place of ``groups``.
    ``adapters`` (ExpertAdapters) serve calls that name each token's adapter;
    they need the fused gate_up matrix.  ``shared`` (SharedExpert) is added to
    the routed experts' sum.  ``norm`` and ``out_norm`` (Norm) stand in front of
    and behind the layer in block().  With ``keep_for_grad`` a forward keeps what
    grads() needs (the input, which must not change until then and may not be the
    memory of the result, and the shared expert's pre-activations).
    """
    scoring: Optional[ScoredRouting] = None
    adapters: Optional[ExpertAdapters] = None
    shared: Optional[SharedExpert] = None
    norm: Optional[Norm] = None
    out_norm: Optional[Norm] = None
    keep_for_grad = False

    def __init__(self, router_w: torch.Tensor, logit_bias: Optional[torch.Tensor], gate: QTensor,
                 up: QTensor, down: QTensor, k_fixed: int, kmax: Optional[int] = None,
                 inv_temperature: float = 1.0, renormalize: bool = True,
                 thresholds=(1.2, 2.5), fuse_gate_up: Optional[bool] = None,
                 path: int = PATH_AUTO, free_sources: bool = False, groups: int = 0,
                 capacity: Optional[int] = None, y_dtype: Optional[torch.dtype] = None,
                 scoring: Optional[ScoredRouting] = None,
                 adapters: Optional[ExpertAdapters] = None,
                 shared: Optional[SharedExpert] = None, norm: Optional[Norm] = None,
                 out_norm: Optional[Norm] = None):
        self.device = router_w.device
        self.router_w = router_w.contiguous()
        self.logit_bias = None if logit_bias is None else logit_bias.contiguous()
        self.E, self.H = router_w.shape
        self.I = gate.rows
        self.bits = gate.bits
        self.k_fixed = k_fixed
        self.kmax = kmax if kmax is not None else (k_fixed if k_fixed > 0 else 3)
        self.inv_temperature = float(inv_temperature)
        self.renormalize = renormalize
        self.thr = tuple(float(t) for t in thresholds)
        self.path = path
        self.groups = int(groups)
        self.capacity = None if capacity is None else int(capacity)
        if y_dtype not in (None, torch.float32, torch.bfloat16):
            raise ValueError("y_dtype must be None, torch.float32 or torch.bfloat16")
        self.y_dtype = y_dtype
        if self.groups > 0 and (self.E % self.groups or k_fixed != self.groups):
            raise ValueError("group-limited routing needs k_fixed == groups dividing E")
        self.scoring = scoring
        if scoring is not None and (k_fixed < 1 or self.groups > 0):
            raise ValueError("scoring needs a fixed k and takes the place of groups")
        self.down = down
        if fuse_gate_up is None:
            fuse_gate_up = os.environ.get(FUSE_ENV, "1") != "0"
        self.fused = False
        self.gate, self.up, self.gate_up = gate, up, None
        if fuse_gate_up:
            gd = B.qdesc(gate.rows, gate.cols, gate.bits)
            ud = B.qdesc(up.rows, up.cols, up.bits)
            try:
                q, s, b = B.moe_pack_gate_up(gd, ud, gate.q, gate.s, gate.b, up.q, up.s, up.b)
                self.gate_up = QTensor(q, s, b, gate.bits)
                self.fused = True
                if free_sources:
                    self.gate = self.up = None
            except MoEError as err:
                if err.status != 3:  # MOE_ERR_INCOMPATIBLE keeps the unfused path
                    raise
        self.adapters = adapters
        if adapters is not None and not self.fused:
            raise ValueError("adapters need the fused gate_up matrix")
        if shared is not None:
            two_i, h = shared.gate_up.shape
            if h != self.H or two_i % 16 or tuple(shared.down.shape) != (self.H, two_i // 2):
                raise ValueError("shared needs gate_up [2*I', H] and down [H, I'] with I' a multiple of 8")
            if any(t.dtype != torch.bfloat16 or not t.is_contiguous() for t in (shared.gate_up, shared.down)):
                raise ValueError("shared needs contiguous bfloat16 matrices")
        for name, n in (("norm", norm), ("out_norm", out_norm)):
            if n is None:
                continue
            if self.H > NORM_MAX_WIDTH:
                raise ValueError(f"{name}: rows of {self.H} are wider than {NORM_MAX_WIDTH}")
            ts = [t for t in (n.weight, n.bias) if t is not None]
            if any(tuple(t.shape) != (self.H,) or t.dtype not in (torch.float32, torch.bfloat16)
                   or t.dtype != ts[0].dtype for t in ts):
                raise ValueError(f"{name} needs weight and bias {(self.H,)}, both float32 or both bfloat16")
        self.shared, self.norm, self.out_norm = shared, norm, out_norm
        self._kept = None
        self._bufs = {}
        # tokens of the last forward and whether it routed by scores, for router_grad
        self._last, self._scored = None, False

    @classmethod
    def from_workload(cls, layer_inputs, device, batch: int = 0, **kw) -> "MoELayer":
        cfg = layer_inputs.cfg
        rw = torch.from_numpy(layer_inputs.router_w).to(device)
        lb = None if layer_inputs.logit_bias is None else torch.from_numpy(layer_inputs.logit_bias).to(device)
        kw.setdefault("inv_temperature", cfg.inv_temperature(batch))
        return cls(rw, lb, qtensor_from_numpy(layer_inputs.gate, device),
                   qtensor_from_numpy(layer_inputs.up, device),
                   qtensor_from_numpy(layer_inputs.down, device), k_fixed=cfg.k,
                   kmax=cfg.slots, **kw)

    def resolved_path(self, T: int) -> int:
        """The kernel family of the products (with an adaptive k, the one for
        k = kmax; k_split says when smaller k take the other family)."""
        if self.path != PATH_AUTO:
            return self.path
        return self._family(T, self.kmax)

    def _family(self, T: int, k: int) -> int:
        if self.bits not in (4, 8):  # 5- and 6-bit codes: the GEMV family only
            return PATH_GEMV
        if (TC_BUILT and (T * k) // self.E >= TC_MIN_TOKENS_PER_EXPERT
                and min(self.H, self.I) * self.bits // 8 >= 128):
            return PATH_TC
        return PATH_GEMV

    def k_split(self, T: int) -> int:
        """With an adaptive k and the automatic path, the k (if any) from
        which the products take the tensor cores while smaller k take the
        streamed GEMV.  k is known only on the device, so both families are
        queued, each gated on its k values; 0 when one family serves every k."""
        if self.path != PATH_AUTO or self.k_fixed != 0 or not self.fused or self.E > 1024:
            return 0
        if self._family(T, 1) == self._family(T, self.kmax):
            return 0
        step = 256 if self.bits == 4 else 128  # the streamed GEMV's row granularity
        if self.H % step or self.I % step:
            return 0
        return next(k for k in range(2, self.kmax + 1) if self._family(T, k) == PATH_TC)

    def y_storage(self, T: int) -> torch.dtype:
        """Storage type of y for calls of T tokens."""
        if self.y_dtype is not None:
            return self.y_dtype
        tc = self.k_split(T) or self.resolved_path(T) == PATH_TC
        return torch.bfloat16 if tc else torch.float32

    def launches_per_call(self, T: int) -> int:
        """Kernels one forward of T tokens launches: the router (plus its
        batch finalize when the tokens span more than one token group of 32,
        16 when E > 256), the grouping (inside those launches when E <= 256
        and T * kmax <= 512, else its own kernel), the row permute on the
        tensor-core path, the gate_up product (or two RAW products and the
        activation when unfused), down and combine.  With a capacity the
        capped grouping is a kernel of its own.  When k_split is set both
        kernel families of each product are launched (one of them returns at
        once).  With scoring the logits, the scores and the grouping are a
        kernel each.  Calls with adapters add theirs, a shared expert its two
        products, block() one for each norm."""
        return self._routed_launches(T) + (2 if self.shared is not None else 0)

    def _routed_launches(self, T: int) -> int:
        if self.scoring is not None:
            # logits, scores, grouping, [row permute], products, combine
            n = 3 + (1 if self.resolved_path(T) == PATH_TC else 0)
            return n + (1 if self.fused else 3) + 2
        group = 32 if self.E <= 256 else 16
        one_group = (T + group - 1) // group == 1
        n = 1 + (0 if one_group else 1)
        fused = self.E <= 256 and T * self.kmax <= 512
        if self.capacity is None:
            n += 0 if fused else 1
        else:
            # the capped grouping, after the group-limited route's own grouping
            n += 1 + ((0 if fused else 1) if self.groups > 0 else 0)
        if self.k_split(T):
            return n + 6  # row permute, two gated gate_up and two gated down launches, combine
        n += 1 if self.resolved_path(T) == PATH_TC else 0
        n += 1 if self.fused else 3
        return n + 2

    def buffers(self, T: int) -> dict:
        key = T
        if key not in self._bufs:
            dev, A = self.device, max(T * self.kmax, 1)
            # both kernel families consume h as bf16 (the GEMV's FMAs take bf16
            # operands, the tensor cores bf16 tiles)
            h_dtype = torch.bfloat16
            bufs = dict(
                topk_ids=torch.empty((T, self.kmax), dtype=torch.int32, device=dev),
                topk_w=torch.empty((T, self.kmax), dtype=torch.float32, device=dev),
                k_dev=torch.empty(1, dtype=torch.int32, device=dev),
                mean_entropy=torch.empty(1, dtype=torch.float32, device=dev),
                ws=torch.empty(B.moe_router_workspace_size(T), dtype=torch.uint8, device=dev),
                counts=torch.empty(self.E, dtype=torch.int32, device=dev),
                offsets=torch.empty(self.E + 1, dtype=torch.int32, device=dev),
                sorted=torch.empty(A, dtype=torch.int32, device=dev),
                inv_pos=torch.empty(A, dtype=torch.int32, device=dev),
                h=torch.empty((A, self.I), dtype=h_dtype, device=dev),
                x_sorted=torch.empty((A, self.H), dtype=torch.bfloat16, device=dev),
                y=torch.empty((A, self.H), dtype=self.y_storage(T), device=dev),
                out=torch.empty((T, self.H), dtype=torch.bfloat16, device=dev),
            )
            if not self.fused:
                bufs["g_raw"] = torch.empty((A, self.I), dtype=torch.float32, device=dev)
                bufs["u_raw"] = torch.empty((A, self.I), dtype=torch.float32, device=dev)
            self._bufs[key] = bufs
        bufs = self._bufs[key]
        if self.scoring is not None and "logits" not in bufs:
            bufs["logits"] = torch.empty((T, self.E), dtype=torch.float32, device=self.device)

        def rows(name, width):
            if name not in bufs or bufs[name].shape[1] != width:
                if name in bufs:  # a captured graph may go on using the one outgrown
                    bufs.setdefault("outgrown", []).append(bufs[name])
                bufs[name] = torch.empty((T, width), dtype=torch.bfloat16, device=self.device)
        if self.shared is not None:
            rows("shared_h", self.shared.down.shape[1])
            if self.keep_for_grad:
                rows("shared_z", self.shared.gate_up.shape[0])
        if self.norm is not None:
            rows("normed", self.H)
            rows("summed", self.H)
        if self.out_norm is not None:
            rows("block_out", self.H)
        return bufs

    def _adapter_buffers(self, b: dict, T: int) -> None:
        ad, dev = self.adapters, self.device
        if ad.gate_up_a is not None and "gu_raw" not in b:
            b["gu_raw"] = torch.empty((max(T * self.kmax, 1), 2 * self.I), dtype=torch.float32,
                                      device=dev)
        # the adapters of a served layer may change, and the need with them
        sizes = tuple((a.shape[0], a.shape[2]) for a in (ad.gate_up_a, ad.down_a)
                      if a is not None)
        if b.get("lora_sizes") != sizes:
            need = max((B.moe_lora_workspace_size(T, self.kmax, self.E, n, r) for n, r in sizes),
                       default=1)
            if "lora_ws" not in b or b["lora_ws"].numel() < need:
                # a captured graph may go on using the one outgrown
                b.setdefault("lora_ws_outgrown", []).append(b.get("lora_ws"))
                b["lora_ws"] = torch.empty(need, dtype=torch.uint8, device=dev)
            b["lora_sizes"] = sizes

    def _route_scored(self, x, b, it):
        """Logits, scored selection and the grouping (empty slots allowed)."""
        s = self.scoring
        B.moe_router_logits(x, self.router_w, self.logit_bias, it, b["logits"])
        B.moe_route_scored(b["logits"], self.k_fixed, s.score, s.select_bias, s.n_groups,
                           s.topk_groups, s.group_top, self.renormalize, s.scale, self.kmax,
                           b["topk_ids"], b["topk_w"], b["k_dev"])
        B.moe_permute_masked(b["topk_ids"], b["k_dev"], self.E, self.capacity, b["counts"],
                             b["offsets"], b["sorted"], b["inv_pos"])

    def forward(self, x: torch.Tensor, out: Optional[torch.Tensor] = None,
                inv_temperature: Optional[float] = None, events: Optional[dict] = None,
                adapter_ids: Optional[torch.Tensor] = None) -> torch.Tensor:
        """x: bf16 [T, H] on the device.  Returns bf16 [T, H] (a reused buffer
        unless ``out`` is given); x may be the result's memory.  ``events``, if
        given, receives per kernel ("router", "permute", "permute_rows", "gate_up",
        "down", "combine") a list of (start, end) CUDA events around its launches
        ("shared" with a shared expert, once for each product).  ``adapter_ids``
        (int32 [T], negative: none) names each token's adapter."""
        self._kept = None
        if self.shared is None and not self.keep_for_grad:
            return self._routed(x, out, inv_temperature, events, adapter_ids)
        T = x.shape[0]
        shared, b = self.shared if T > 0 else None, self.buffers(T)
        res = out if out is not None else b["out"]
        if self.keep_for_grad and (shared is not None or self.scoring is not None) and _overlap(x, res):
            raise ValueError("keep_for_grad needs an input apart from the result: grads() reads it again")
        if shared is not None:  # x may be the result's memory, which the routed experts write
            ev = _Timer(events, "shared")
            B.moe_linear(x, shared.gate_up, activation=ACT_SWIGLU, out=b["shared_h"],
                         preact=b["shared_z"] if self.keep_for_grad else None)
            ev.stop()
        self._routed(x, res, inv_temperature, events, adapter_ids)
        if self.keep_for_grad:
            self._kept = dict(x=x, shared=_fields(self.shared), scoring=self._scores(), inv_temperature=(
                self.inv_temperature if inv_temperature is None else float(inv_temperature)))
        if shared is not None:
            ev = _Timer(events, "shared")
            # the routed sum comes as the layer's result, in bf16: half a bf16 step of it
            # more than one rounding of the whole
            B.moe_linear(b["shared_h"], shared.down, residual=res, out=res)
            ev.stop()
        return res

    def block(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
              out: Optional[torch.Tensor] = None, **forward_args):
        """The layer with its norms, as a block of a model: with s = x + residual
        (x without one), out_norm(layer(norm(s))) -> (out, s), both bf16 [T, H] and
        buffers that the next call of T tokens writes again unless ``out`` is
        given (s is x itself without a residual, or a copy where x is memory that the
        block writes).  The next block takes them as x and residual, so the sum is part of
        its norm's kernel; out + s ends the last."""
        if residual is not None and self.norm is None:
            raise ValueError("a residual needs a layer with a norm, whose kernel adds it")
        b = self.buffers(x.shape[0])
        res = out if out is not None else b["out" if self.out_norm is None else "block_out"]
        if residual is not None and _overlap(b["summed"], res):
            raise ValueError("out is the memory of the sum that is returned beside it")
        if self.keep_for_grad and self.out_norm is not None:
            kept = [b["out"]]
            if self.shared is not None or self.scoring is not None:
                kept.append(x if self.norm is None else b["normed"])
            if _overlap(res, *kept):
                raise ValueError("out is the memory of what grads() reads again")
        # what is written on the way to the result, and the result
        written = (res, b["out"]) if self.norm is None else (res, b["out"], b["normed"])
        s, h = x.clone() if residual is None and _overlap(x, *written) else x, x
        if self.norm is not None:
            n = self.norm
            h, summed, _, _ = B.moe_layer_norm(
                x, n.weight, n.bias, residual=residual, eps=n.eps, kind=n.kind, out=b["normed"],
                summed=None if residual is None else b["summed"])
            s = s if residual is None else summed
        y = self.forward(h, out=out if self.out_norm is None else None, **forward_args)
        if self.out_norm is None:
            return y, s
        n = self.out_norm
        _, _, mean, rstd = B.moe_layer_norm(y, n.weight, n.bias, eps=n.eps, kind=n.kind,
                                            need_stats=self.keep_for_grad, out=res)
        if self._kept is not None:
            self._kept.update(y=y, mean=mean, rstd=rstd, out_norm=_fields(n))
        return res, s

    def _routed(self, x, out, inv_temperature, events, adapter_ids):
        T = x.shape[0]
        b = self.buffers(T)
        path = self.resolved_path(T)
        if adapter_ids is not None:
            if self.adapters is None:
                raise ValueError("adapter_ids given to a layer without adapters")
            self._adapter_buffers(b, T)
        self._last, self._scored = T, self.scoring is not None
        it = self.inv_temperature if inv_temperature is None else float(inv_temperature)
        # router, top-k and the expert grouping (one launch for small batches)
        ev = _Timer(events, "route")
        if self.scoring is not None:
            self._route_scored(x, b, it)
        elif self.capacity is not None:
            # router (group-limited or top-k), then the grouping with each
            # expert's capacity (it replaces the uncapped grouping that the
            # group-limited route also writes)
            if self.groups > 0:
                B.moe_route_grouped(x, self.router_w, self.logit_bias, it, self.groups,
                                    self.kmax, self.renormalize, b["topk_ids"], b["topk_w"],
                                    b["k_dev"], b["mean_entropy"], b["ws"], b["counts"],
                                    b["offsets"], b["sorted"], b["inv_pos"])
            else:
                B.moe_router_topk(x, self.router_w, self.logit_bias, it, self.k_fixed, self.kmax,
                                  self.thr[0], self.thr[1], self.renormalize, b["topk_ids"],
                                  b["topk_w"], b["k_dev"], b["mean_entropy"], b["ws"])
            B.moe_permute_capped(b["topk_ids"], b["k_dev"], self.E, self.capacity, b["counts"],
                                 b["offsets"], b["sorted"], b["inv_pos"])
        elif self.groups > 0:
            B.moe_route_grouped(x, self.router_w, self.logit_bias, it, self.groups, self.kmax,
                                self.renormalize, b["topk_ids"], b["topk_w"], b["k_dev"],
                                b["mean_entropy"], b["ws"], b["counts"], b["offsets"],
                                b["sorted"], b["inv_pos"])
        else:
            B.moe_route(x, self.router_w, self.logit_bias, it, self.k_fixed, self.kmax,
                        self.thr[0], self.thr[1], self.renormalize, b["topk_ids"], b["topk_w"],
                        b["k_dev"], b["mean_entropy"], b["ws"], b["counts"], b["offsets"],
                        b["sorted"], b["inv_pos"])
        ev.stop()
        ks = self.k_split(T) if adapter_ids is None else 0
        if ks:
            return self._forward_k_split(x, b, ks, T, out, events)
        # tensor cores: token rows copied once into expert order, so every
        # tile loads contiguous rows; the GEMV reads x through sorted_assign
        if path == PATH_TC:
            ev = _Timer(events, "permute_rows")
            xs = B.moe_permute_rows(x, b["sorted"], b["k_dev"], self.kmax, b["x_sorted"])
            ev.stop()
            srt = None
        else:
            xs, srt = x, b["sorted"]
        ev = _Timer(events, "gate_up")
        ad = self.adapters if adapter_ids is not None else None
        route = dict(topk_ids=b["topk_ids"], sorted_assign=b["sorted"],
                     expert_offsets=b["offsets"])
        if ad is not None and ad.gate_up_a is not None:
            # the raw halves, then adapters and activation in one kernel
            g = self.gate_up
            B.moe_gate_up_qmm(xs, srt, b["offsets"], b["k_dev"], self.kmax, g.q, g.s, g.b,
                              self.bits, EPILOGUE_RAW, torch.float32, b["gu_raw"], path, T=T)
            B.moe_lora_apply(x, adapter_ids, ad.gate_up_a, ad.gate_up_b, ad.scales, b["gu_raw"],
                             b["h"], EPILOGUE_SWIGLU, workspace=b["lora_ws"], **route)
        elif self.fused:
            g = self.gate_up
            B.moe_gate_up_qmm(xs, srt, b["offsets"], b["k_dev"], self.kmax, g.q, g.s, g.b,
                              self.bits, EPILOGUE_SWIGLU, b["h"].dtype, b["h"], path, T=T)
        else:
            for m, dst in ((self.gate, b["g_raw"]), (self.up, b["u_raw"])):
                B.moe_gate_up_qmm(xs, srt, b["offsets"], b["k_dev"], self.kmax, m.q, m.s,
                                  m.b, self.bits, EPILOGUE_RAW, torch.float32, dst, path, T=T)
            B.moe_swiglu(b["g_raw"], b["u_raw"], b["k_dev"], T, self.kmax, b["h"].dtype, b["h"])
        ev.stop()
        d = self.down
        ev = _Timer(events, "down")
        # the kernel just before this one (gate_up or the activation) writes
        # only h: the down weights may stream while it finishes
        B.moe_down_qmm(b["h"], b["offsets"], b["k_dev"], T, self.kmax, d.q, d.s, d.b, self.bits,
                       b["y"], path | PATH_FLAG_WEIGHTS_EARLY)
        if ad is not None and ad.down_a is not None:
            B.moe_lora_apply(b["h"], adapter_ids, ad.down_a, ad.down_b, ad.scales, b["y"], b["y"],
                             workspace=b["lora_ws"], x_by_token=False, **route)
        ev.stop()
        res = out if out is not None else b["out"]
        ev = _Timer(events, "combine")
        B.moe_combine(b["y"], b["inv_pos"], b["topk_w"], b["k_dev"], T, self.kmax, res)
        ev.stop()
        return res

    def chosen_counts(self) -> torch.Tensor:
        """int32 [E]: how often the last forward's routing chose each expert,
        the assignments that a capacity turned away included (the grouping's
        own counts hold the kept ones).  May be a buffer that the next forward
        writes again."""
        if self._last is None:
            raise ValueError("chosen_counts needs a forward first")
        b = self.buffers(self._last)
        if self.capacity is None:
            return b["counts"]
        return B.moe_permute_masked(b["topk_ids"], b["k_dev"], self.E)[0]

    def router_grad(self, d_out: torch.Tensor, balance_coef: float = 0.0, z_coef: float = 0.0):
        """Gradient of the last forward with respect to the router logits, the
        experts held fixed: -> (d_logits fp32 [T, E], losses fp32 [2]).

        d_out bf16 [T, H]: the gradient of the layer's output.  Adds the
        balance and z losses (their values are returned); the balance loss
        counts the router's choices, whatever a capacity kept.  Only for layers
        with ``scoring``; the router weight's gradient is
        inv_temperature * d_logits^T x."""
        if self.scoring is None or self._last is None:
            raise ValueError("router_grad needs a layer with scoring, after a forward")
        T = self._last
        b = self.buffers(T)
        if not self._scored:
            raise ValueError("router_grad needs a forward with the layer's scoring")
        if tuple(d_out.shape) != (T, self.H):
            raise ValueError(f"d_out must be {(T, self.H)}, got {tuple(d_out.shape)}")
        if T == 0:
            return (torch.zeros((0, self.E), device=self.device),
                    torch.zeros(2, device=self.device))
        d_w, _ = B.moe_combine_backward(d_out, b["y"], b["inv_pos"], b["topk_w"], b["k_dev"],
                                        need_d_y=False)
        s = self.scoring
        counts = self.chosen_counts() if balance_coef else None
        return B.moe_route_scored_backward(
            b["logits"], b["topk_ids"], d_w, counts, s.score, self.k_fixed, self.renormalize,
            s.scale, balance_coef, z_coef)

    def _scores(self) -> tuple:
        """What the weights of the chosen experts are made with."""
        return () if self.scoring is None else (self.scoring.score, self.scoring.scale, self.renormalize)

    def trainable(self) -> dict:
        """The tensors that grads() gives gradients of, by name: ``router_w`` (with
        scoring; ``logit_bias`` stays as it is), the shared expert's and out_norm's.
        The quantized experts stay as they are, and with them whatever reaches the
        loss through their input: ``norm`` is not among them."""
        t = {}
        if self.scoring is not None:
            t["router_w"] = self.router_w
        if self.shared is not None:
            t["shared.gate_up"], t["shared.down"] = self.shared.gate_up, self.shared.down
        if self.out_norm is not None:
            for name in ("weight", "bias"):
                if getattr(self.out_norm, name) is not None:
                    t["out_norm." + name] = getattr(self.out_norm, name)
        return t

    def grads(self, d_out: torch.Tensor, balance_coef: float = 0.0, z_coef: float = 0.0):
        """Gradients of the last block() or forward() with keep_for_grad, for the
        gradient ``d_out`` (bf16 [T, H]) of its output and the balance and z losses
        (see router_grad) -> (gradients by the names of trainable(), fp32, losses
        fp32 [2] or None without scoring)."""
        k = self._kept
        if k is None:
            raise ValueError("grads needs a forward with keep_for_grad")
        norm = self.out_norm if "rstd" in k else None
        if not (_same(_fields(self.shared), k["shared"]) and _same(_fields(norm), k.get("out_norm", ()))
                and _same(self._scores(), k["scoring"])):
            raise ValueError("grads needs a forward with the layer's shared expert, norm and scoring as they are")
        x, g, losses = k["x"], {}, None
        T = x.shape[0]
        if tuple(d_out.shape) != (T, self.H) or d_out.dtype != torch.bfloat16:
            raise ValueError(f"d_out must be bfloat16 {(T, self.H)}")
        if T == 0:
            zeros = {n: torch.zeros(t.shape, device=t.device) for n, t in self.trainable().items()}
            return zeros, None if self.scoring is None else torch.zeros(2, device=self.device)
        if "rstd" in k:
            n = self.out_norm
            d_out, d_w, d_b = B.moe_layer_norm_backward(
                d_out, k["y"], k["rstd"], k["mean"], n.weight, kind=n.kind,
                need_d_weight=n.weight is not None, need_d_bias=n.bias is not None)
            for name, t in (("weight", d_w), ("bias", d_b)):
                if t is not None:
                    g["out_norm." + name] = t
        if self.scoring is not None:
            d_logits, losses = self.router_grad(d_out, balance_coef, z_coef)
            # inv_temperature d_logits^T x with the gradient as two bf16 terms, 2^-17 of it
            d = d_logits * k["inv_temperature"]
            hi = d.to(torch.bfloat16)
            lo = (d - hi.float()).to(torch.bfloat16)
            only = dict(need_d_x=False, need_d_bias=False)
            w = B.moe_linear_backward(hi, x, None, **only)[1]
            B.moe_linear_backward(lo, x, None, d_w=w, accumulate=True, **only)
            g["router_w"] = w
        if self.shared is not None:
            b, s = self.buffers(T), self.shared
            d_h, g["shared.down"], _, _ = B.moe_linear_backward(d_out, b["shared_h"], s.down,
                                                                need_d_bias=False)
            g["shared.gate_up"] = B.moe_linear_backward(
                d_h, x, s.gate_up, b["shared_z"], activation=ACT_SWIGLU, need_d_x=False,
                need_d_bias=False)[1]
        return g, losses

    def _forward_k_split(self, x, b, ks, T, out, events):
        """The products after routing when k < ks takes the streamed GEMV and
        k >= ks the tensor cores: each product's two launches are gated on k,
        so exactly one of them computes."""
        lo_gate, hi_gate = path_k_range(1, ks - 1), path_k_range(ks, self.kmax)
        ev = _Timer(events, "permute_rows")
        xs = B.moe_permute_rows(x, b["sorted"], b["k_dev"], self.kmax, b["x_sorted"])
        ev.stop()
        g = self.gate_up
        ev = _Timer(events, "gate_up")
        B.moe_gate_up_qmm(x, b["sorted"], b["offsets"], b["k_dev"], self.kmax, g.q, g.s, g.b,
                          self.bits, EPILOGUE_SWIGLU, b["h"].dtype, b["h"], PATH_GEMV | lo_gate,
                          T=T)
        B.moe_gate_up_qmm(xs, None, b["offsets"], b["k_dev"], self.kmax, g.q, g.s, g.b,
                          self.bits, EPILOGUE_SWIGLU, b["h"].dtype, b["h"], PATH_TC | hi_gate, T=T)
        ev.stop()
        d = self.down
        ev = _Timer(events, "down")
        # the GEMV's weights may stream early: the kernel ahead of it (the
        # gated tensor-core gate_up) writes only h
        B.moe_down_qmm(b["h"], b["offsets"], b["k_dev"], T, self.kmax, d.q, d.s, d.b, self.bits,
                       b["y"], PATH_GEMV | PATH_FLAG_WEIGHTS_EARLY | lo_gate)
        B.moe_down_qmm(b["h"], b["offsets"], b["k_dev"], T, self.kmax, d.q, d.s, d.b, self.bits,
                       b["y"], PATH_TC | hi_gate)
        ev.stop()
        res = out if out is not None else b["out"]
        ev = _Timer(events, "combine")
        B.moe_combine(b["y"], b["inv_pos"], b["topk_w"], b["k_dev"], T, self.kmax, res)
        ev.stop()
        return res

    __call__ = forward

    def forward_host(self, x_host: torch.Tensor, out_host: torch.Tensor,
                     inv_temperature: Optional[float] = None,
                     adapter_ids: Optional[torch.Tensor] = None) -> torch.Tensor:
        """End-to-end call with host buffers: copies x (pinned host, bf16
        [T, H]) and, if given, adapter_ids (pinned host, int32 [T]) to the
        device, runs the layer and copies the result back into out_host, all
        enqueued on the current stream (no synchronization)."""
        T = x_host.shape[0]
        b = self.buffers(T)
        if "x_dev" not in b:
            b["x_dev"] = torch.empty((T, self.H), dtype=torch.bfloat16, device=self.device)
        b["x_dev"].copy_(x_host, non_blocking=True)
        if adapter_ids is not None:
            if adapter_ids.dtype != torch.int32 or tuple(adapter_ids.shape) != (T,):
                raise ValueError(f"adapter_ids must be int32 {(T,)}")
            if "adapters_dev" not in b:
                b["adapters_dev"] = torch.empty(T, dtype=torch.int32, device=self.device)
            b["adapters_dev"].copy_(adapter_ids, non_blocking=True)
            adapter_ids = b["adapters_dev"]
        res = self.forward(b["x_dev"], inv_temperature=inv_temperature, adapter_ids=adapter_ids)
        out_host.copy_(res, non_blocking=True)
        return out_host


def _fields(part) -> tuple:
    """The tensors and settings of a SharedExpert or a Norm; none of None."""
    return () if part is None else tuple(getattr(part, f.name) for f in dataclasses.fields(part))


def _same(a: tuple, b: tuple) -> bool:
    """The same tensors and equal settings."""
    return len(a) == len(b) and all(
        x is y or not (torch.is_tensor(x) or torch.is_tensor(y)) and x == y for x, y in zip(a, b))


def _overlap(t: torch.Tensor, *others: torch.Tensor) -> bool:
    """Whether the memory between t's first and last elements meets that of one of the others."""
    def span(t):
        p = t.data_ptr()
        if t.is_contiguous():
            return p, p + t.nbytes
        return p, p + (sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) * t.element_size()
    if t.numel() == 0:
        return False
    lo, hi = span(t)
    for o in others:
        p, q = span(o)
        if lo < q and p < hi:
            return True
    return False


class _Timer:
    def __init__(self, events: Optional[dict], name: str):
        self.events, self.name = events, name
        if events is not None:
            self.start = torch.cuda.Event(enable_timing=True)
            self.start.record()

    def stop(self):
        if self.events is not None:
            end = torch.cuda.Event(enable_timing=True)
            end.record()
            self.events.setdefault(self.name, []).append((self.start, end))
