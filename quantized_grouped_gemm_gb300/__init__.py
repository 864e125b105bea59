"""GB300 (sm_103a) sparse-MoE expert path -- Python binding of ``include/moe.h``.

Argument marshalling only: every step of the path runs in the CUDA kernels of
``libmoe_gb300.so``.  PyTorch provides device memory and streams.  bf16 tensors may be passed
as ``torch.bfloat16`` or as 16-bit integer tensors holding the bit patterns.

Calls have the names of the C ABI: ``moe_route``, ``moe_grouped_ffn`` (= ``moe_ffn_gate_up``
then ``moe_ffn_down``), ``moe_combine``, ``moe_forward``, ``moe_pack_weights``,
``moe_read_status``; ``moe_gate`` and ``moe_dispatch`` (any gate in place of the router's own
choice) and ``moe_linear`` (the unquantised projections beside the experts).
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import _lib
from ._lib import (MOE_ERR_CUDA, MOE_ERR_DEVICE_STATUS, MOE_ERR_DEVICE_TIMEOUT, MOE_ERR_INVALID_ARG,
                   MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_OK, MOE_STATUS_BAD_EXPERT, MOE_STATUS_TIMEOUT)

__all__ = ["MoEError", "shape", "options", "Routing", "workspace", "moe_workspace_bytes", "moe_packed_bytes",
           "moe_pack_weights", "moe_route", "moe_grouped_ffn", "moe_ffn_gate_up", "moe_ffn_down", "moe_combine",
           "moe_forward", "moe_read_status", "moe_check_shape", "moe_launch_count", "moe_forward_decode_static",
           "gate_config", "moe_gate", "moe_dispatch", "linear_config", "linear_workspace",
           "moe_linear_workspace_bytes", "moe_linear", "lib"]


class MoEError(RuntimeError):
    def __init__(self, what: str, rc: int):
        super().__init__(f"{what}: {lib().moe_error_string(rc).decode()} ({rc})")
        self.rc = rc


def lib():
    return _lib.load()


def _check(rc: int, what: str) -> None:
    if rc != MOE_OK:
        raise MoEError(what, rc)


def shape(T: int, d: int, E: int = 256, k: int = 8, I: int = 512, I_shared: Optional[int] = None,
          group: int = 64) -> _lib.moe_shape:
    return _lib.moe_shape(T, d, E, k, I, I if I_shared is None else I_shared, group)


DECODE_AUTO, DECODE_GEMV = 0, 1


def options(tile_rows: int = 32, decode_max_tokens: int = 1, decode_path: int = DECODE_AUTO,
            deterministic: int = 0, host_routing: int = 0, unfused_dequant: int = 0,
            gemm_rows: int = 0) -> _lib.moe_options:
    """decode_path: DECODE_AUTO (one fused launch per token when it fits) or DECODE_GEMV.
    deterministic: 1 = prefill sums each token's rows in a fixed order at every size.
    host_routing: 1 = ablation of GPU-resident routing: the scan and block map run on the
    host after a device-to-host copy of the counts (synchronises the stream; same results).
    unfused_dequant: 1 = ablation of on-chip dequantisation: each FFN call first writes the
    projection's weights as bf16 into the (larger) workspace, then streams them (same results).
    gemm_rows: 16, 32, 64 or 128 = largest token block of the grouped GEMMs (0: default 128)."""
    return _lib.moe_options(tile_rows, decode_max_tokens, decode_path, deterministic, host_routing, unfused_dequant,
                            gemm_rows)


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _s(stream: Optional[torch.cuda.Stream]):
    # the raw handle of the current stream: a Stream object costs about 3 us a call, as much as a launch, and
    # torch.cuda.current_device() another 0.2 (CUDA is initialised: the caller's tensors are on it)
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()) if stream is None else stream.cuda_stream


def _o(opts):
    return ctypes.byref(opts) if opts is not None else None


def moe_check_shape(shp) -> int:
    return lib().moe_check_shape(ctypes.byref(shp))


def moe_workspace_bytes(shp, opts=None) -> int:
    return int(lib().moe_workspace_bytes(ctypes.byref(shp), _o(opts)))


def moe_packed_bytes(shp, num_experts: int, intermediate: int) -> int:
    return int(lib().moe_packed_bytes(ctypes.byref(shp), num_experts, intermediate))


def moe_launch_count() -> int:
    return int(lib().moe_launch_count())


def workspace(shp, opts=None, device="cuda") -> torch.Tensor:
    """A zero-filled workspace (the library needs it zeroed once, before first use)."""
    n = moe_workspace_bytes(shp, opts)
    if n == 0:
        raise MoEError("moe_workspace_bytes", moe_check_shape(shp) or MOE_ERR_INVALID_ARG)
    return torch.zeros(n, dtype=torch.uint8, device=device)


class Routing:
    """Caller-owned device buffers of the routing results (see moe_routing in moe.h)."""

    def __init__(self, T: int, k: int = 8, E: int = 256, tile_rows: int = 32, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        self.topk_idx = torch.empty(max(T, 1), k, **i32)
        self.topk_w = torch.empty(max(T, 1), k, dtype=torch.float32, device=device)
        self.counts = torch.empty(E, **i32)
        self.offsets = torch.empty(E + 1, **i32)
        self.perm = torch.empty(max(k * T, 1), **i32)
        self.pos = torch.empty(max(T, 1), k, **i32)
        mt = int(lib().moe_max_tiles(T, k, E, tile_rows))
        self.tiles = torch.empty(mt, 3, **i32)
        self.num_tiles = torch.zeros(1, **i32)
        self._s = _lib.moe_routing(*(t.data_ptr() for t in (self.topk_idx, self.topk_w, self.counts, self.offsets,
                                                              self.perm, self.pos, self.tiles, self.num_tiles)))

    def ref(self):
        return ctypes.byref(self._s)


def _q4(m: Sequence[torch.Tensor]) -> _lib.moe_q4:
    codes, scales, biases = m
    return _lib.moe_q4(codes.data_ptr(), scales.data_ptr(), biases.data_ptr())


def moe_pack_weights(shp, gate, up, down, intermediate: int, out: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """Relayout one expert stack (each of gate/up/down = (codes, scales, biases) device tensors,
    expert outermost) into the packed 4-bit form; returns the packed uint8 tensor."""
    E = gate[0].shape[0]
    n = moe_packed_bytes(shp, E, intermediate)
    if n == 0:
        raise MoEError("moe_packed_bytes", MOE_ERR_UNSUPPORTED)
    if out is None:
        out = torch.empty(n, dtype=torch.uint8, device=gate[0].device)
    w = _lib.moe_expert_weights(_q4(gate), _q4(up), _q4(down), E)
    _check(lib().moe_pack_weights(ctypes.byref(shp), ctypes.byref(w), intermediate, _p(out), out.numel(),
                                  _s(stream)), "moe_pack_weights")
    return out


def moe_route(shp, x, w_router, logit_bias, routing: Routing, ws, opts=None, stream=None) -> None:
    _check(lib().moe_route(ctypes.byref(shp), _p(x), _p(w_router), _p(logit_bias), routing.ref(), _p(ws),
                           ws.numel(), _o(opts), _s(stream)), "moe_route")


def moe_router_logits(shp, x, w_router, logit_bias, out, stream=None) -> None:
    """Every exact router logit (fp32 [T][E] into out), as moe_route defines them."""
    _check(lib().moe_router_logits(ctypes.byref(shp), _p(x), _p(w_router), _p(logit_bias), _p(out), _s(stream)),
           "moe_router_logits")


def moe_ffn_gate_up(shp, x, routing: Routing, packed_routed, packed_shared, ws, opts=None, stream=None) -> None:
    _check(lib().moe_ffn_gate_up(ctypes.byref(shp), _p(x), routing.ref(), _p(packed_routed), _p(packed_shared),
                                 _p(ws), ws.numel(), _o(opts), _s(stream)), "moe_ffn_gate_up")


def moe_ffn_down(shp, routing: Routing, packed_routed, packed_shared, ws, opts=None, stream=None) -> None:
    _check(lib().moe_ffn_down(ctypes.byref(shp), routing.ref(), _p(packed_routed), _p(packed_shared), _p(ws),
                              ws.numel(), _o(opts), _s(stream)), "moe_ffn_down")


def moe_grouped_ffn(shp, x, routing: Routing, packed_routed, packed_shared, ws, opts=None, stream=None) -> None:
    _check(lib().moe_grouped_ffn(ctypes.byref(shp), _p(x), routing.ref(), _p(packed_routed), _p(packed_shared),
                                 _p(ws), ws.numel(), _o(opts), _s(stream)), "moe_grouped_ffn")


def moe_combine(shp, routing: Routing, ws, y, opts=None, stream=None) -> None:
    _check(lib().moe_combine(ctypes.byref(shp), routing.ref(), _p(ws), ws.numel(), _p(y), _o(opts), _s(stream)),
           "moe_combine")


def moe_forward(shp, x, w_router, logit_bias, packed_routed, packed_shared, routing: Routing, ws, y, opts=None,
                stream=None) -> None:
    _check(lib().moe_forward(ctypes.byref(shp), _p(x), _p(w_router), _p(logit_bias), _p(packed_routed),
                             _p(packed_shared), routing.ref(), _p(ws), ws.numel(), _p(y), _o(opts), _s(stream)),
           "moe_forward")


def moe_forward_decode_static(shp, x, w_router, logit_bias, packed_routed, packed_shared, routing: Routing, y,
                              stream=None) -> None:
    """One-token forward with no workspace: the scratch is a fixed device array inside the
    library (see moe_forward_decode_static in include/moe.h).  For callers that cannot
    allocate scratch memory; calls that overlap on the GPU race on the shared array."""
    _check(lib().moe_forward_decode_static(ctypes.byref(shp), _p(x), _p(w_router), _p(logit_bias),
                                           _p(packed_routed), _p(packed_shared), routing.ref(), _p(y), _s(stream)),
           "moe_forward_decode_static")


def moe_read_status(ws, stream=None):
    """Synchronise, read and clear the device status word: (return code, raw status bits)."""
    bits = ctypes.c_int(0)
    rc = lib().moe_read_status(_p(ws), _s(stream), ctypes.byref(bits))
    return rc, bits.value


_TYPES = {torch.float32: _lib.MOE_F32, torch.bfloat16: _lib.MOE_BF16, torch.float16: _lib.MOE_F16}
_SCORES = {"softmax": _lib.MOE_SCORE_SOFTMAX, "sigmoid": _lib.MOE_SCORE_SIGMOID}
_GROUP_SCORES = {"top2": _lib.MOE_GROUP_TOP2, "max": _lib.MOE_GROUP_MAX}
_ACTIVATIONS = {"none": _lib.MOE_ACT_NONE, "relu": _lib.MOE_ACT_RELU, "silu": _lib.MOE_ACT_SILU,
                "gelu": _lib.MOE_ACT_GELU, "gelu_tanh": _lib.MOE_ACT_GELU_TANH, "swiglu": _lib.MOE_ACT_SWIGLU}


def gate_config(T: int, E: int = 256, k: int = 8, score: str = "softmax", dtype: torch.dtype = torch.float32,
                groups: int = 1, group_topk: int = 1, group_score: str = "top2", renormalise: bool = True,
                scale: float = 1.0, logits_stride: int = 0) -> _lib.moe_gate_config:
    """The gate of moe_gate (see moe_gate_config in moe.h): score "softmax" or "sigmoid", group_score
    "top2" or "max", dtype that of the logits, logits_stride in elements (0: E)."""
    return _lib.moe_gate_config(T, E, k, _TYPES[dtype], _SCORES[score], groups, group_topk, _GROUP_SCORES[group_score],
                                int(renormalise), scale, logits_stride)


def moe_gate(cfg, logits, select_bias, topk_idx, topk_w, stream=None) -> None:
    """The k experts and weights of every token, into topk_idx (int32) and topk_w (fp32) [T, k]."""
    rc = lib().moe_gate(cfg, logits.data_ptr(), _p(select_bias), topk_idx.data_ptr(), topk_w.data_ptr(), _s(stream))
    if rc != MOE_OK:
        raise MoEError("moe_gate", rc)


def moe_dispatch(shp, x, routing: Routing, ws, opts=None, stream=None) -> None:
    """The routing metadata and gathered rows for the choice in routing.topk_idx / topk_w."""
    _check(lib().moe_dispatch(ctypes.byref(shp), _p(x), routing.ref(), _p(ws), ws.numel(), _o(opts), _s(stream)),
           "moe_dispatch")


def linear_config(T: int, N: int, K: int, dtype: torch.dtype = torch.bfloat16,
                  out_dtype: Optional[torch.dtype] = None, activation: str = "none", x_stride: int = 0,
                  w_stride: int = 0, residual_stride: int = 0, y_stride: int = 0) -> _lib.moe_linear_config:
    """The projection of moe_linear (see moe_linear_config in moe.h): dtype of x and w, out_dtype of y and
    residual (default: dtype), strides in elements (0: dense rows)."""
    return _lib.moe_linear_config(T, N, K, _TYPES[dtype], _TYPES[dtype if out_dtype is None else out_dtype],
                                  _ACTIVATIONS[activation], x_stride, w_stride, residual_stride, y_stride)


def moe_linear_workspace_bytes(cfg) -> int:
    return int(lib().moe_linear_workspace_bytes(ctypes.byref(cfg)))


def linear_workspace(cfg, device="cuda") -> torch.Tensor:
    """A workspace for moe_linear (its status word zeroed)."""
    n = moe_linear_workspace_bytes(cfg)
    if n == 0:
        raise MoEError("moe_linear_workspace_bytes", MOE_ERR_UNSUPPORTED)
    if n <= 4096:
        return torch.zeros(n, dtype=torch.uint8, device=device)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def moe_linear(cfg, x, w, bias, residual, y, ws, stream=None) -> None:
    """y = act(x w^T + bias) + residual; bias (fp32) and residual may be None, y may be residual."""
    rc = lib().moe_linear(cfg, x.data_ptr(), w.data_ptr(), _p(bias), _p(residual), y.data_ptr(), ws.data_ptr(),
                          ws.numel(), _s(stream))
    if rc != MOE_OK:
        raise MoEError("moe_linear", rc)
