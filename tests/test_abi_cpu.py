"""Host-side checks of the C ABI that need no GPU: the library loads, exports
every function include/moe_gb300.h declares, and rejects bad arguments
before launching anything."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    from sparse_moe_expert_gb300 import _build
    _build.build()
    import sparse_moe_expert_gb300 as moe
    return moe.lib()


def declared_functions():
    names = set()
    for fn in os.listdir(os.path.join(ROOT, "include")):
        if fn.endswith(".h"):
            src = open(os.path.join(ROOT, "include", fn)).read()
            names |= set(re.findall(r"^\s*(?:const\s+)?[A-Za-z_][A-Za-z0-9_]*\**\s+\**\s*(moe_[a-z0-9_]+)\s*\(",
                                    src, re.M))
    return names


def test_exports_every_declared_function(L):
    names = declared_functions()
    assert len(names) >= 11, names
    import sparse_moe_expert_gb300 as moe
    assert names == set(moe.EXPORTS)
    for n in names:
        assert hasattr(L, n), n


def test_status_strings_and_version(L):
    import sparse_moe_expert_gb300 as moe
    assert moe.moe_abi_version() == 2
    assert moe.moe_status_string(0) == "ok"
    assert moe.moe_status_string(3) == "gate and up cannot be fused"
    assert moe.moe_status_string(99) == "unknown status"


def vp(v):
    return ctypes.c_void_p(v)


GOOD = 0x10000  # an aligned fake address; never dereferenced by a rejected call


def test_router_rejects_bad_shapes_before_launch(L):
    f = L.moe_router_topk
    args = dict(x=GOOD, w=GOOD, b=None, it=1.0, T=4, H=256, E=8, k=2, kmax=2, t1=1.2, t2=2.5, rn=1,
                ids=GOOD, tw=GOOD, kd=GOOD, me=GOOD, ws=GOOD, wsb=1 << 20)

    def call(**over):
        a = dict(args, **over)
        return f(vp(a["x"]), vp(a["w"]), a["b"], ctypes.c_float(a["it"]), a["T"], a["H"], a["E"],
                 a["k"], a["kmax"], ctypes.c_float(a["t1"]), ctypes.c_float(a["t2"]), a["rn"],
                 vp(a["ids"]), vp(a["tw"]), vp(a["kd"]), vp(a["me"]), vp(a["ws"]), a["wsb"], None)
    assert call(H=100) == 1          # H % 64
    assert call(E=0) == 1
    assert call(E=2000) == 1
    assert call(k=3) == 1            # k > kmax
    assert call(k=0, kmax=2) == 1    # adaptive needs kmax >= 3
    assert call(kmax=17) == 1
    assert call(x=GOOD + 4) == 1     # misaligned
    assert call(wsb=0) == 1          # workspace too small
    assert call(t1=3.0, t2=2.0) == 1
    assert call(kd=0) == 1


def test_qmm_and_pack_reject_before_launch(L):
    import sparse_moe_expert_gb300 as moe
    g = L.moe_gate_up_qmm
    base = [vp(GOOD), vp(GOOD), vp(GOOD), vp(GOOD), 4, 2, 8, 256, 512, vp(GOOD), vp(GOOD),
            vp(GOOD)]
    assert g(*base, 3, 1, 0, vp(GOOD), 0, None) == 2                    # bits 3 unsupported
    gated = moe.PATH_GEMV | moe.path_k_range(1, 2)
    for bits in (5, 6):           # the GEMV family only, and without a k gate
        assert g(*base, bits, 1, 0, vp(GOOD), moe.PATH_TC, None) == 2
        assert g(*base, bits, 1, 0, vp(GOOD), gated, None) == 2
    assert g(*base, 4, 0, 1, vp(GOOD), 0, None) == 2                    # RAW needs fp32 out
    assert g(*base, 4, 7, 0, vp(GOOD), 0, None) == 1                    # bad epilogue
    assert g(*base, 4, 1, 0, vp(GOOD), 9, None) == 1                    # bad path
    bad = list(base)
    bad[7] = 200                                                        # H % 64
    assert g(*bad, 4, 1, 0, vp(GOOD), 0, None) == 1
    d = L.moe_down_qmm
    assert d(vp(GOOD), 0, vp(GOOD), vp(GOOD), 4, 2, 8, 100, 256, vp(GOOD), vp(GOOD), vp(GOOD), 4,
             vp(GOOD), 0, 0, None) == 1                                 # I % 64
    assert d(vp(GOOD), 0, vp(GOOD), vp(GOOD), 4, 2, 8, 128, 256, vp(GOOD), vp(GOOD), vp(GOOD), 4,
             vp(GOOD), 5, 0, None) == 1                                 # bad y dtype
    a = moe.qdesc(512, 256, 4)
    for field, val in [("bits", 8), ("group_size", 32), ("has_bias", 1), ("rows", 256),
                       ("cols", 512), ("mode", 1), ("quantized", 0), ("scale_dtype", 1)]:
        b = moe.qdesc(512, 256, 4)
        setattr(b, field, val)
        st = L.moe_pack_gate_up(ctypes.byref(a), ctypes.byref(b), *[vp(GOOD)] * 6, 8,
                                *[vp(GOOD)] * 3, None)
        assert st == 3, field                                           # MOE_ERR_INCOMPATIBLE
    c = moe.qdesc(512, 256, 3)
    st = L.moe_pack_gate_up(ctypes.byref(c), ctypes.byref(c), *[vp(GOOD)] * 6, 8, *[vp(GOOD)] * 3,
                            None)
    assert st == 2                                                      # bits 3 unsupported
    assert L.moe_permute(vp(GOOD), vp(GOOD), 4, 2, 0, vp(GOOD), vp(GOOD), vp(GOOD), vp(GOOD),
                         None) == 1
    assert L.moe_combine(vp(GOOD), 0, vp(GOOD), vp(GOOD), vp(GOOD), 4, 2, 100, vp(GOOD),
                         None) == 1                                     # H % 64
    assert L.moe_combine(vp(GOOD), 7, vp(GOOD), vp(GOOD), vp(GOOD), 4, 2, 128, vp(GOOD),
                         None) == 1                                     # bad y dtype
    assert L.moe_swiglu(vp(GOOD), vp(GOOD), vp(GOOD), 4, 2, 256, 5, vp(GOOD), None) == 1


def test_workspace_size_grows_with_tokens(L):
    import sparse_moe_expert_gb300 as moe
    assert moe.moe_router_workspace_size(0) > 0
    assert moe.moe_router_workspace_size(4096) >= 2 * 4 * 4096


def test_header_constants_match_the_binding(tmp_path):
    """The header compiles as C, and its path flags, k-range macro, dropped
    marker and dtype codes agree with the Python binding's constants."""
    import shutil
    import subprocess
    import sparse_moe_expert_gb300 as moe
    from sparse_moe_expert_gb300 import _lib
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "consts.c"
    src.write_text(
        '#include <stdio.h>\n#include "moe_gb300.h"\n'
        "int main(void) {\n"
        '  printf("%d %d %d %d %d %d %d\\n", MOE_PATH_GEMV, MOE_PATH_TC, MOE_PATH_FLAG_WEIGHTS_EARLY,\n'
        "         MOE_PATH_FLAG_K_GATED, MOE_PATH_K_RANGE(2, 3), MOE_DROPPED, MOE_PATH_AUTO);\n"
        "  return 0;\n}\n")
    exe = tmp_path / "consts"
    subprocess.run([cc, "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    vals = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True,
                                           check=True).stdout.split()]
    assert vals == [moe.PATH_GEMV, moe.PATH_TC, moe.PATH_FLAG_WEIGHTS_EARLY,
                    moe.PATH_FLAG_K_GATED, moe.path_k_range(2, 3), moe.DROPPED,
                    moe.PATH_AUTO]


def test_native_entry_points_load_and_refuse_host_tensors(L):
    """The CPython entry points of the short calls load next to the library
    and refuse wrong arguments with ValueError before any C call."""
    import torch
    import sparse_moe_expert_gb300 as moe
    from sparse_moe_expert_gb300 import _lib
    assert _lib.native() is _lib.native()
    i32 = torch.int32
    with pytest.raises(ValueError, match="logits must be a CUDA tensor"):
        moe.moe_route_scored(torch.zeros(2, 8), 2)
    with pytest.raises(ValueError, match="must be a tensor"):
        moe.moe_route_scored([1.0], 2)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_route_scored_backward(torch.zeros(2, 8), torch.zeros((2, 2), dtype=i32))
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_combine_backward(torch.zeros((2, 64), dtype=torch.bfloat16), torch.zeros(4, 64),
                                 torch.zeros(4, dtype=i32), torch.zeros(2, 2),
                                 torch.zeros(1, dtype=i32))
    with pytest.raises(ValueError, match="CUDA"):
        b = torch.zeros((1, 64, 8), dtype=torch.bfloat16)
        moe.moe_lora_apply(torch.zeros((2, 64), dtype=torch.bfloat16), torch.zeros(2, dtype=i32),
                           b.view(1, 8, 64), b)
    with pytest.raises(TypeError):
        moe.moe_route_scored(torch.zeros(2, 8), "two")


def test_operator_calls_reject_bad_shapes_before_launch(L):
    f = L.moe_route_scored
    base = dict(l=GOOD, dt=0, ld=64, b=None, T=4, E=64, s=0, g=1, tg=1, gt=1, k=4, km=4, rn=1,
                sc=1.0, ids=GOOD, w=GOOD, kd=GOOD)

    def route(**over):
        a = dict(base, **over)
        return f(vp(a["l"]), a["dt"], a["ld"], a["b"], a["T"], a["E"], a["s"], a["g"], a["tg"],
                 a["gt"], a["k"], a["km"], a["rn"], ctypes.c_float(a["sc"]), vp(a["ids"]),
                 vp(a["w"]), vp(a["kd"]), None)
    for bad in (dict(E=0), dict(E=1025), dict(ld=63), dict(k=5), dict(km=17), dict(g=3),
                dict(g=4, tg=5), dict(gt=0), dict(s=2), dict(dt=2), dict(sc=0.0), dict(kd=0),
                dict(ids=0), dict(w=GOOD + 2), dict(l=GOOD + 2), dict(T=-1), dict(b=vp(GOOD + 1))):
        assert route(**bad) == 1, bad
    b = L.moe_route_scored_backward

    def back(T=4, E=64, ws=GOOD, wsb=1 << 30, d=GOOD * 2, bal=0.0, counts=None, losses=GOOD):
        return b(vp(GOOD), 0, 64, vp(GOOD), vp(GOOD), counts, T, E, 0, 2, 2, 1, ctypes.c_float(1),
                 ctypes.c_float(bal), ctypes.c_float(0), vp(d), 64, vp(losses), vp(ws), wsb, None)
    assert back(wsb=16) == 1 and back(d=GOOD) == 1 and back(bal=0.1) == 1
    assert back(E=2000) == 1 and back(losses=0) == 1 and back(ws=0) == 1 and back(T=-1) == 1
    c = L.moe_combine_backward
    args = [vp(GOOD), vp(GOOD), 0, vp(GOOD), vp(GOOD), vp(GOOD), 4, 2, 128, vp(GOOD), None, None]
    for i, v in ((2, 5), (7, 0), (7, 17), (8, 100), (0, vp(GOOD + 4)), (5, None), (10, vp(GOOD))):
        bad = list(args)
        bad[i] = v
        assert c(*bad) == 1, i
    a = L.moe_lora_apply
    good = [vp(GOOD), 1, vp(GOOD), None, None, None, 4, 1, 1, 3, 128, 128, 16, vp(GOOD), vp(GOOD),
            None, vp(GOOD), 0, 0, 0, vp(GOOD), vp(GOOD), 1 << 30, None]
    for i, v, st in ((6, -1, 1), (7, 2, 1), (8, 4, 1), (9, 0, 1), (10, 96, 1), (11, 100, 1),
                     (12, 12, 1), (12, 136, 1), (13, None, 1), (16, vp(GOOD + 8), 1), (17, 1, 2),
                     (18, 2, 1), (19, 7, 1), (20, None, 1), (22, 8, 1), (3, vp(GOOD), 1)):
        bad = list(good)
        bad[i] = v
        assert a(*bad) == st, i
    assert L.moe_permute_masked(vp(GOOD), vp(GOOD), 4, 2, 8, -2, vp(GOOD), vp(GOOD), vp(GOOD),
                                vp(GOOD), None) == 1
    assert L.moe_router_logits(vp(GOOD), vp(GOOD), None, ctypes.c_float(0), 4, 256, 8, vp(GOOD),
                               None) == 1
    assert L.moe_router_logits(vp(GOOD), vp(GOOD), None, ctypes.c_float(1), 4, 100, 8, vp(GOOD),
                               None) == 1


def test_the_c_library_is_built_without_torch(monkeypatch, tmp_path):
    """Users of the C ABI need no torch: libmoe_gb300.so is linked before the
    CPython entry points are asked for, whose failure is still raised."""
    import sys
    from sparse_moe_expert_gb300 import _build
    src = tmp_path / "csrc"
    src.mkdir()
    (src / "one.cu").write_text('extern "C" int moe_one(void) { return 1; }\n')
    monkeypatch.setattr(_build, "CSRC", str(src))
    monkeypatch.setattr(_build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(_build, "NATIVE", str(tmp_path / "_native.so"))
    monkeypatch.setitem(sys.modules, "torch", None)
    with pytest.raises(ImportError):
        _build.build()
    assert ctypes.CDLL(str(tmp_path / "lib.so")).moe_one() == 1


def test_misaligned_integers_and_scales_are_refused(L):
    """Arrays of 4-byte entries off their boundary, which the kernels could
    only fault on."""
    a = L.moe_lora_apply
    good = [vp(GOOD), 1, vp(GOOD), vp(GOOD), vp(GOOD), vp(GOOD), 4, 2, 8, 3, 128, 128, 16,
            vp(GOOD), vp(GOOD), vp(GOOD), vp(GOOD), 0, 0, 0, vp(GOOD), vp(GOOD), 1 << 30, None]
    for i in (2, 3, 4, 5, 15):
        for off in (1, 2, 3):
            bad = list(good)
            bad[i] = vp(GOOD + off)
            assert a(*bad) == 1, i
    c = L.moe_combine_backward
    args = [vp(GOOD), vp(GOOD), 0, vp(GOOD), vp(GOOD), vp(GOOD + 2), 4, 2, 128, vp(GOOD), None,
            None]
    assert c(*args) == 1
    m = L.moe_permute_masked
    good = [vp(GOOD), vp(GOOD), 4, 2, 8, -1, vp(GOOD), vp(GOOD), vp(GOOD), vp(GOOD), None]
    for i in (0, 1, 6, 7, 8, 9):
        bad = list(good)
        bad[i] = vp(GOOD + 2)
        assert m(*bad) == 1, i
