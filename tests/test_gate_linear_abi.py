"""CPU checks of moe_gate, moe_dispatch and moe_linear: their refusals and workspace sizes, which are decided
on the host before any CUDA call."""
import ctypes

import pytest

from quantized_grouped_gemm_gb300 import _lib, build as build_mod

INV, UNS, WS = _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_WORKSPACE
GATE = dict(T=4, E=256, k=8, logits_type=_lib.MOE_F32, score=_lib.MOE_SCORE_SOFTMAX, groups=1, group_topk=1,
            group_score=_lib.MOE_GROUP_TOP2, renormalise=1, scale=1.0, logits_stride=0)
LINEAR = dict(T=4, N=64, K=64, type=_lib.MOE_BF16, out_type=_lib.MOE_BF16, activation=_lib.MOE_ACT_NONE, x_stride=0,
              w_stride=0, residual_stride=0, y_stride=0)


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return _lib.load()


def gate(lib, logits=None, idx=None, w=None, bias=None, **kw):
    c = _lib.moe_gate_config(**{**GATE, **kw})
    return lib.moe_gate(ctypes.byref(c), logits, bias, idx, w, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(T=-1), INV), (dict(E=0), INV), (dict(k=0), INV), (dict(E=4, k=5), INV), (dict(logits_stride=255), INV),
    (dict(logits_stride=-1), INV), (dict(logits_type=3), INV), (dict(logits_type=-1), INV), (dict(score=2), INV),
    (dict(group_score=2), INV), (dict(renormalise=2), INV), (dict(scale=float("nan")), INV),
    (dict(scale=float("inf")), INV), (dict(groups=-1), INV), (dict(groups=3), INV),                 # 256 % 3
    (dict(groups=8, group_topk=0), INV), (dict(groups=8, group_topk=9), INV),
    (dict(E=32, groups=8, group_topk=1), INV),                                                      # 8 of 4 experts
    (dict(E=8, groups=8, group_topk=8, k=4), INV),                                                  # top 2 of one expert
    (dict(E=1025), UNS), (dict(k=33), UNS), (dict(T=(1 << 20) + 1), UNS), (dict(groups=64, group_topk=64), UNS),
])
def test_gate_refusals(lib, kw, rc):
    assert gate(lib, **kw) == rc


def test_gate_pointers(lib):
    assert gate(lib) == INV
    assert gate(lib, T=0) == _lib.MOE_OK
    assert lib.moe_gate(None, None, None, None, None, None) == INV
    # misaligned pointers are refused before anything is launched
    assert gate(lib, logits=2, idx=16, w=16) == INV
    assert gate(lib, logits=1, idx=16, w=16, logits_type=_lib.MOE_BF16) == INV
    assert gate(lib, logits=16, idx=18, w=16) == INV
    assert gate(lib, logits=16, idx=16, w=16, bias=2) == INV


def linear(lib, x=None, w=None, bias=None, r=None, y=None, ws=None, bytes=1 << 30, **kw):
    c = _lib.moe_linear_config(**{**LINEAR, **kw})
    return lib.moe_linear(ctypes.byref(c), x, w, bias, r, y, ws, bytes, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(T=-1), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(type=_lib.MOE_F32, out_type=_lib.MOE_F32), INV),
    (dict(type=3), INV), (dict(out_type=_lib.MOE_F16), INV), (dict(out_type=-1), INV), (dict(activation=6), INV),
    (dict(activation=-1), INV), (dict(x_stride=63), INV), (dict(w_stride=63), INV), (dict(y_stride=63), INV),
    (dict(residual_stride=63), INV), (dict(x_stride=-64), INV), (dict(T=(1 << 20) + 1), UNS),
    (dict(N=(1 << 20) + 1), UNS), (dict(K=65537), UNS), (dict(x_stride=(1 << 36) + 8), UNS),
])
def test_linear_refusals(lib, kw, rc):
    assert linear(lib, **kw) == rc
    c = _lib.moe_linear_config(**{**LINEAR, **kw})
    assert lib.moe_linear_workspace_bytes(ctypes.byref(c)) == 0


def test_linear_pointers(lib):
    ok = dict(x=256, w=256, y=256, ws=256)
    assert linear(lib) == INV
    assert linear(lib, T=0) == _lib.MOE_OK
    assert lib.moe_linear(None, None, None, None, None, None, None, 0, None) == INV
    assert lib.moe_linear_workspace_bytes(None) == 0
    for name, bad in (("x", 8), ("w", 8), ("y", 8), ("ws", 128), ("x", None), ("w", None), ("y", None), ("ws", None)):
        assert linear(lib, **{**ok, name: bad}) == INV, name
    assert linear(lib, **ok, bias=2) == INV
    assert linear(lib, **ok, r=8) == INV
    assert linear(lib, **ok, bytes=255) == WS


def test_dispatch_refusals(lib):
    s = _lib.moe_shape(16, 512, 256, 8, 128, 128, 64)
    rt = _lib.moe_routing()
    assert lib.moe_dispatch(ctypes.byref(s), None, ctypes.byref(rt), None, 0, None, None) == INV
    o = _lib.moe_options(32, 1, 0, 0, 1)   # host_routing
    assert lib.moe_dispatch(ctypes.byref(s), None, ctypes.byref(rt), None, 0, ctypes.byref(o), None) == UNS
    for bad, rc in (((16, 512, 128, 8, 128, 128, 64), UNS), ((-1, 512, 256, 8, 128, 128, 64), INV)):
        b = _lib.moe_shape(*bad)
        assert lib.moe_dispatch(ctypes.byref(b), None, ctypes.byref(rt), None, 0, None, None) == rc
    z = _lib.moe_shape(0, 512, 256, 8, 128, 128, 64)
    assert lib.moe_dispatch(ctypes.byref(z), None, None, None, 0, None, None) == _lib.MOE_OK
    full = _lib.moe_routing(*([256] * 8))
    assert lib.moe_dispatch(ctypes.byref(s), 256, ctypes.byref(full), 256, 1024, None, None) == WS


def test_linear_workspace_sizes(lib):
    """A status word; rows that start at no multiple of 16 bytes add an aligned copy of their operand."""
    def size(**kw):
        return lib.moe_linear_workspace_bytes(ctypes.byref(_lib.moe_linear_config(**{**LINEAR, **kw})))
    up = lambda v: (v + 255) // 256 * 256   # noqa: E731
    assert size() == size(T=0) == size(T=1 << 20, N=1 << 20, K=65536) == 256
    assert size(T=500, K=1001) == 256 + up(64 * 1008 * 2) + up(500 * 1008 * 2)
    assert size(T=500, K=1001, activation=_lib.MOE_ACT_SWIGLU) == 256 + up(128 * 1008 * 2) + up(500 * 1008 * 2)
    assert size(T=500, K=1000, x_stride=1003) == 256 + up(500 * 1000 * 2)
    assert size(T=500, K=1000, w_stride=1003) == 256 + up(64 * 1000 * 2)
    assert size(T=500, K=1001, x_stride=1008, w_stride=1008) == 256
    assert size(T=500, y_stride=67, residual_stride=65) == 256
