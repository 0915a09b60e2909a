"""A layer refuses norms and shared experts that do not fit it when it is made, not at its
first block.
The layer is made of host tensors, without the fused matrix."""
import pytest
import torch

import sparse_moe_expert_gb300 as moe
from sparse_moe_expert_gb300.layer import MoELayer, Norm, QTensor, SharedExpert


def make(H, **kw):
    def q(rows, cols):
        z = torch.empty(2, rows, cols // 64, dtype=torch.float16)
        return QTensor(torch.empty(2, rows, cols // 8, dtype=torch.int32), z, z, 4)
    return MoELayer(torch.empty(2, H), None, q(64, H), q(64, H), q(H, 64), k_fixed=1, fuse_gate_up=False, **kw)


@pytest.mark.parametrize("name", ["norm", "out_norm"])
def test_norms_are_checked_when_the_layer_is_made(name):
    H = 128
    for good in (Norm(), Norm(torch.ones(H)), Norm(torch.ones(H, dtype=torch.bfloat16)),
                 Norm(None, torch.ones(H), kind=moe.NORM_LAYER)):
        assert getattr(make(H, **{name: good}), name) is good
    for bad in (Norm(torch.ones(H - 1)), Norm(torch.ones(1, H)), Norm(None, torch.ones(H + 64)),
                Norm(torch.ones(H, dtype=torch.float16)),
                Norm(torch.ones(H), torch.ones(H, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            make(H, **{name: bad})
    assert moe.NORM_MAX_WIDTH == 8192
    make(8192, **{name: Norm()})
    make(8256)
    with pytest.raises(ValueError):
        make(8256, **{name: Norm()})
    # the limit is the kernel's
    from sparse_moe_expert_gb300 import _build
    _build.build()
    assert moe.moe_layer_norm_workspace_size(4, moe.NORM_MAX_WIDTH) > 16
    assert moe.moe_layer_norm_workspace_size(4, moe.NORM_MAX_WIDTH + 1) == 16


def test_shared_experts_are_checked_when_the_layer_is_made():
    H, B16 = 128, torch.bfloat16
    gate_up, down = torch.zeros(128, H, dtype=B16), torch.zeros(H, 64, dtype=B16)
    assert make(H, shared=SharedExpert(gate_up, down)).shared.down is down
    for a, b in ((gate_up.float(), down), (gate_up, down.float()), (gate_up, down.half()),
                 (torch.zeros(H, 128, dtype=B16).t(), down), (gate_up, torch.zeros(64, H, dtype=B16).t()),
                 (gate_up[:96], down), (gate_up[:, :64], down), (torch.zeros(24, H, dtype=B16), down[:, :12])):
        with pytest.raises(ValueError):
            make(H, shared=SharedExpert(a, b))
