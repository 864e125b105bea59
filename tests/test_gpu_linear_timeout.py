"""Bounded waits of moe_linear's tensor-core kernels that run out: the kernel records a timeout in the workspace's
status word and unwinds, in every CTA of its cluster, and the same process then gets right results.

The failure is made by a separate copy of the library built for this test only: its waits give up after 2e7 SM
cycles (about 10 ms), and the producer leaves out the second stage of the first tile, so that the issuer's wait on
it can never complete.  The product library is built without either change.
"""
import ctypes
import os

import pytest
import torch

import quantized_grouped_gemm_gb300 as moe
from quantized_grouped_gemm_gb300 import _lib, build as build_mod

pytestmark = pytest.mark.gpu

_DIR = os.path.join(os.path.dirname(build_mod.__file__), "_build", "linear_timeout_test")


@pytest.fixture(scope="module")
def faulty():
    path = os.path.join(_DIR, "libmoe_timeout.so")
    build_mod.build(out=path, build_dir=os.path.join(_DIR, "objs"),
                    defines=["MOE_WAIT_LIMIT_CYCLES=20000000ll", "MOE_TEST_DROP_LINEAR_BLOCK=1"])
    L = ctypes.CDLL(path)
    for name, (res, args) in _lib._SIG.items():
        fn = getattr(L, name)
        fn.restype, fn.argtypes = res, args
    return L


# CTA pairs; one CTA to a tile, many tiles; slices of K over a cluster
@pytest.mark.parametrize("T,N,K", [(4096, 2048, 2048), (24, 40000, 1024), (64, 512, 4096)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_timeout_is_reported_and_the_next_call_is_right(faulty, T, N, K, out):
    cfg = moe.linear_config(T, N, K, out_dtype=out)
    x = torch.randn(T, K, device="cuda").bfloat16()
    w = (torch.randn(N, K, device="cuda") * K ** -0.5).bfloat16()
    y = torch.empty(T, N, device="cuda", dtype=out)
    ws = moe.linear_workspace(cfg)
    st = torch.cuda.current_stream().cuda_stream
    rc = faulty.moe_linear(ctypes.byref(cfg), x.data_ptr(), w.data_ptr(), None, None, y.data_ptr(), ws.data_ptr(),
                           ws.numel(), st)
    assert rc == moe.MOE_OK                                   # the launch itself succeeds
    bits = ctypes.c_int(0)
    rc = faulty.moe_read_status(ws.data_ptr(), st, ctypes.byref(bits))
    assert rc == moe.MOE_ERR_DEVICE_TIMEOUT and bits.value & moe.MOE_STATUS_TIMEOUT, (rc, bits.value)
    moe.moe_linear(cfg, x, w, None, None, y, ws)              # the status word was cleared by reading it
    assert moe.moe_read_status(ws)[0] == moe.MOE_OK
    ref = x.double() @ w.double().t()
    assert ((y.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-4).all()
