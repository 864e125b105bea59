"""moe_linear on the GPU against the formula in 64 bits: types, activations, biases, residuals, odd sizes and
strides, every kernel's range of token counts."""
import math

import pytest
import torch

import quantized_grouped_gemm_gb300 as moe

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ROUND = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}   # half a unit of 24, 8 and 11 bits


def act64(name, z):
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def check(T, N, K, dt="bf16", out=None, act="none", bias=False, residual=False, xpad=0, wpad=0, rpad=0, ypad=0,
          in_place=False, seed=0, stream=None):
    out = out or dt
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * T + 11 * N + 13 * K)
    rows = 2 * N if act == "swiglu" else N
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    nan = float("nan")
    xb = torch.full((T, K + xpad), nan, device="cuda", dtype=DT[dt])      # what lies between the rows is never used
    wb = torch.full((rows, K + wpad), nan, device="cuda", dtype=DT[dt])
    xb[:, :K] = rand(T, K).to(DT[dt])
    wb[:, :K] = (rand(rows, K) * K ** -0.5).to(DT[dt])
    b = rand(rows) if bias else None
    r = None
    if residual:
        r = torch.full((T, N + rpad), nan, device="cuda", dtype=DT[out])
        r[:, :N] = rand(T, N).to(DT[out])
    yb = r if in_place else torch.full((T + 1, N + ypad), -7.0, device="cuda", dtype=DT[out])
    r0 = None if r is None else r[:, :N].double()
    cfg = moe.linear_config(T, N, K, dtype=DT[dt], out_dtype=DT[out], activation=act, x_stride=K + xpad,
                            w_stride=K + wpad, residual_stride=N + rpad, y_stride=N + (rpad if in_place else ypad))
    ws = moe.linear_workspace(cfg)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    moe.moe_linear(cfg, xb, wb, b, r, yb, ws, stream=stream)
    rc, bits = moe.moe_read_status(ws, stream)
    assert rc == moe.MOE_OK, bits
    torch.cuda.synchronize()
    y = yb[:T, :N].double()
    if not in_place:
        assert (yb[T:] == -7).all() and (yb[:, N:] == -7).all(), "written outside y"

    # z is a sum of K products whose partial sums are rounded (the tensor cores truncate) at most K/16 + 16
    # times to 24 bits, each time by at most 2^-23 of the sum of magnitudes
    x64, w64 = xb[:, :K].double(), wb[:, :K].double()
    z = x64 @ w64.t()
    ez = 2.0 ** -23 * (K / 16 + 16) * (x64.abs() @ w64.abs().t())
    if bias:
        z = z + b.double()
        ez = ez + 2.0 ** -23 * z.abs()
    if act == "swiglu":
        gz, uz = z[:, :N], z[:, N:]
        a = gz * torch.sigmoid(gz)
        v = a * uz
        ev = 1.1 * ez[:, :N] * uz.abs() + a.abs() * ez[:, N:] + 1.1 * ez[:, :N] * ez[:, N:]
    else:
        v = act64(act, z)
        ev = 1.13 * ez                                     # the activations' slopes are at most 1.13
    if act != "none" and act != "relu":
        ev = ev + 2.0 ** -18 * v.abs() + 2.0 ** -23        # the exponentials: a few 2^-23 and 2^-23 of their argument
    if residual:
        v = v + r0
    tol = ev + ROUND[out] * (v.abs() + ev) * 1.01 + 2.0 ** -23 * v.abs() + (2.0 ** -25 if out == "f16" else 0.0)
    err = (y - v).abs()
    assert torch.isfinite(y).all()
    worst = (err / tol).max().item() if tol.numel() else 0.0
    assert worst <= 1.0, f"{(err > tol).sum().item()} of {err.numel()} outside, worst {worst:.2f} x the bound"
    if out == "f32" and act == "none" and T * N > 256:
        assert ((y - v).norm() / v.norm()).item() <= 1e-6
    return yb


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"])
@pytest.mark.parametrize("T", [1, 5, 40, 300])
@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
def test_types_and_activations(act, T, dt, out):
    check(T, 272, 320, dt, out, act, bias=True, residual=True)


@pytest.mark.parametrize("T,N,K", [(1, 1, 1), (1, 16, 8), (3, 17, 33), (8, 15, 7), (9, 100, 129), (16, 33, 1000),
                                   (17, 300, 65), (32, 31, 4097), (33, 129, 64), (64, 64, 63), (65, 200, 127),
                                   (127, 255, 513), (128, 128, 128), (129, 130, 136), (257, 513, 250), (511, 96, 2048),
                                   (1000, 77, 72), (2049, 520, 264)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_sizes(T, N, K, dt):
    check(T, N, K, dt, bias=True)
    check(T, N, K, dt, act="swiglu", residual=True)


@pytest.mark.parametrize("T", [1, 12, 70, 400])
@pytest.mark.parametrize("xpad,wpad,rpad,ypad", [(8, 8, 8, 8), (1, 0, 0, 0), (0, 1, 0, 0), (0, 0, 1, 3), (3, 5, 7, 1),
                                                (64, 0, 2, 4)])
def test_strides(T, xpad, wpad, rpad, ypad):
    check(T, 200, 264, "bf16", bias=True, residual=True, xpad=xpad, wpad=wpad, rpad=rpad, ypad=ypad)
    check(T, 200, 264, "f16", "f32", residual=True, xpad=xpad, wpad=wpad, rpad=rpad, ypad=ypad)


@pytest.mark.parametrize("T", [1, 20, 130, 700, 3000])
@pytest.mark.parametrize("dt,out,rpad", [("bf16", "bf16", 0), ("f16", "f16", 5), ("bf16", "f32", 8)])
def test_residual_in_place(T, dt, out, rpad):
    check(T, 264, 512, dt, out, residual=True, in_place=True, rpad=rpad)


@pytest.mark.parametrize("T,N,K,out,act", [(1, 2048, 2048, "bf16", "none"), (8, 40000, 512, "f32", "none"),
                                           (128, 2048, 2048, "bf16", "silu"), (512, 2048, 1024, "bf16", "swiglu"),
                                           (2048, 256, 2048, "f32", "none"), (4096, 2048, 1024, "bf16", "none"),
                                           (4000, 4100, 520, "f32", "gelu"), (5000, 2056, 1000, "bf16", "swiglu"),
                                           (700, 1024, 7168, "f32", "none")])
def test_larger(T, N, K, out, act):
    check(T, N, K, "bf16", out, act, bias=True, residual=act == "none")


@pytest.mark.parametrize("K", [512, 4096, 8192, 16384, 65536])
@pytest.mark.parametrize("T,N,act", [(1, 64, "none"), (1, 2048, "none"), (1, 16, "swiglu"), (8, 256, "none"),
                                     (1, 256, "swiglu"), (16, 100, "swiglu"), (200, 300, "none"), (200, 300, "swiglu")])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_fp32_sums_of_long_rows(T, N, act, K, dt):
    """At most 512 products meet in the tensor cores' accumulator.  One product is 2^24 and the others 2^-5, which are
    lost, 16 at a time and truncated, where they are added to it there, but not where they are first added to each other:
    512 make 16, a multiple of the 2 that 2^24 counts in.  So at most 16 may be missing of the K / 32."""
    big = 2.0 ** 24
    rows = 2 * N if act == "swiglu" else N
    for at in (0, 127, 128, K // 2, K - 1):
        x = torch.ones(T, K, device="cuda", dtype=DT[dt])
        w = torch.full((rows, K), 2.0 ** -5, device="cuda", dtype=DT[dt])
        x[:, at] = 2.0 ** 12
        w[:, at] = 2.0 ** 12
        if act == "swiglu":                            # gates of 64, whose sigmoid is 1 in fp32
            w[:N] = 0.0
            w[:N, (at + 1) % K] = 64.0
        cfg = moe.linear_config(T, N, K, dtype=DT[dt], out_dtype=torch.float32, activation=act)
        y = torch.empty(T, N, device="cuda")
        moe.moe_linear(cfg, x, w, None, None, y, moe.linear_workspace(cfg))
        z = (y.double() if act == "none" else y.double() / 64.0) - big
        # the quotient of the sigmoid and two products: 2^-22 of 2^24
        slack = 0.0 if act == "none" else 4.0
        lost = (K - 1) / 32 - z
        assert lost.min().item() >= -slack - 2.0, (at, lost.min().item())   # (a multiple of 2: rounded by less than that)
        assert lost.max().item() <= 16.0 + slack, (at, lost.max().item())


@pytest.mark.parametrize("K", [8192, 8200, 16384, 40000, 65536])
@pytest.mark.parametrize("T,N", [(1, 64), (8, 1000), (24, 2000), (200, 300), (600, 1024)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_16_bit_outputs_of_long_rows(T, N, act, K, dt):
    """At most 8192 products meet in the tensor cores' accumulator.  As above, with one product of 2^10 and others of 2^-18,
    16 of which are half of what 2^10 counts in; the residual takes the 2^10 off again, so that what is left shows in 16
    bits.  8192 of the others make 2^-5, which is all that may be missing."""
    at = K // 3
    x = torch.full((T, K), 2.0 ** -9, device="cuda", dtype=DT[dt])
    w = torch.full((2 * N if act == "swiglu" else N, K), 2.0 ** -9, device="cuda", dtype=DT[dt])
    x[:, at], w[:, at] = 32.0, 32.0
    unit = 1.0
    if act == "swiglu":                                # gates of 32, whose sigmoid is 1 in fp32
        unit = 32.0
        w[:N] = 0.0
        w[:N, at + 1] = 2.0 ** 14
    r = torch.full((T, N), -unit * 2.0 ** 10, device="cuda", dtype=DT[dt])
    y = torch.empty(T, N, device="cuda", dtype=DT[dt])
    cfg = moe.linear_config(T, N, K, dtype=DT[dt], activation=act)
    ws = moe.linear_workspace(cfg)
    moe.moe_linear(cfg, x, w, None, r, y, ws)
    assert moe.moe_read_status(ws)[0] == moe.MOE_OK
    small = (K - 1) * 2.0 ** -18
    lost = small - y.double() / unit
    # the sum counts in 2^-13, once rounded and once truncated; the gate's quotient and products: 2^-22 of 2^10; y's rounding
    slack = 2.0 ** -12 + (2.0 ** -12 if act == "swiglu" else 0.0) + ROUND[dt] * small
    assert lost.min().item() >= -slack and lost.max().item() <= 2.0 ** -5 + slack, (lost.min().item(), lost.max().item())


@pytest.mark.parametrize("T,N,K", [(1 << 20, 24, 64), ((1 << 20) - 1, 264, 40), (1, 1 << 20, 72), (17, (1 << 20) - 3, 64),
                                   (300, 1 << 20, 64), (2, 24, 65536), (70, 40, 65535), (300, 264, 65536)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_largest_sizes(T, N, K, out):
    """The ends of the accepted ranges: tokens, features, columns."""
    check(T, N, K, "bf16", out, bias=True, residual=T * N < 1 << 27)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,N,out", [(1 << 20, 16, "bf16"), ((1 << 20) - 5, 136, "f32")])
def test_outputs_past_32_bits(T, N, out):
    """Row offsets of y and of the residual above 2^31 elements."""
    check(T, N, 64, "bf16", out, residual=True, rpad=2300 - N, ypad=2304 - N)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("T", [3, 40, 600])
def test_activations_far_from_zero(T, act, dt, out):
    """Large arguments, given by the bias: 0 (or next to it) on the negative side, the argument itself on the other."""
    z = torch.tensor([0.0, 8.0, 12.0, 12.99, 13.01, 13.1, 13.3, 14.0, 16.0, 19.9, 20.1, 30.0, 86.0, 100.0, 500.0, 6e4, 1e10, 1e20,
                      1e36, 3e38], device="cuda")
    z = torch.cat([z, -z])
    N = z.numel()
    cfg = moe.linear_config(T, N, 64, dtype=DT[dt], out_dtype=DT[out], activation=act)
    x = torch.zeros(T, 64, device="cuda", dtype=DT[dt])
    w = torch.zeros(N, 64, device="cuda", dtype=DT[dt])
    y = torch.empty(T, N, device="cuda", dtype=DT[out])
    moe.moe_linear(cfg, x, w, z, None, y, moe.linear_workspace(cfg))
    z = z.double()
    # forms that keep their digits in the tail (1 + tanh and torch's ndtr, which is 1 + erf, are 0 there)
    v = {"silu": z * torch.sigmoid(z), "gelu": 0.5 * z * torch.special.erfc(-z * math.sqrt(0.5)),
         "gelu_tanh": z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))}[act]
    assert not torch.isnan(y).any() and torch.equal(y, y[:1].expand(T, N))
    y = y[0].double()
    fits = v.abs() < torch.finfo(DT[out]).max
    assert torch.equal(y[~fits], v[~fits].sign() * (float("inf") if out == "f16" else torch.finfo(DT[out]).max))
    # a value's relative error: 2^-24 of the exponential's argument, up to 85 (gelu's square is rounded: 5e-6), for 16-bit
    # outputs again of its product with log2 e (7e-6), 4e-7 of the fit; beside it half the least number of fp16 and 90 times
    # (z) 2^-126, below which an exponential is 0
    rel = 2.0 ** -15 if out != "f32" else 2.0 ** -17
    tol = rel * v.abs() + ROUND[out] * v.abs() * 1.01 + 90 * 2.0 ** -126 + (2.0 ** -24 if out == "f16" else 0.0)
    assert ((y - v).abs() <= tol)[fits].all(), ((y - v).abs() / tol)[fits].max().item()


@pytest.mark.parametrize("T", [4, 50, 600])
def test_a_bad_row_stays_a_row(T):
    """NaN and infinity in one token's row, and in one weight row, reach that row and column only."""
    N, K = 320, 256
    x = torch.randn(T, K, device="cuda").bfloat16()
    w = torch.randn(N, K, device="cuda").bfloat16()
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    w[300, 9] = float("nan")
    cfg = moe.linear_config(T, N, K)
    y = torch.empty(T, N, device="cuda", dtype=torch.bfloat16)
    moe.moe_linear(cfg, x, w, None, None, y, moe.linear_workspace(cfg))
    assert torch.isnan(y[1]).all() and torch.isnan(y[:, 300]).all()
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[1:3] = False
    cols = torch.ones(N, dtype=torch.bool, device="cuda")
    cols[300] = False
    assert torch.isfinite(y[keep][:, cols]).all()
    assert not torch.isfinite(y[2][cols]).any()


@pytest.mark.parametrize("T,N,K", [(1, 2048, 2048), (24, 2048, 2048), (200, 1024, 4096), (3000, 1000, 777)])
def test_same_bits_every_time(T, N, K):
    x = torch.randn(T, K, device="cuda").bfloat16()
    w = torch.randn(N, K, device="cuda").bfloat16()
    cfg = moe.linear_config(T, N, K, out_dtype=torch.float32)
    ws = moe.linear_workspace(cfg)
    ys = [torch.empty(T, N, device="cuda") for _ in range(4)]
    for y in ys:
        moe.moe_linear(cfg, x, w, None, None, y, ws)
    assert all(torch.equal(ys[0], y) for y in ys[1:])


def test_zero_tokens_and_other_stream():
    check(0, 64, 64)
    for T in (3, 90, 900):
        check(T, 640, 512, stream=torch.cuda.Stream())


def test_in_a_cuda_graph():
    """Captured once and replayed on new inputs: no call-time state is kept."""
    for T in (2, 64, 1024):
        cfg = moe.linear_config(T, 512, 512)
        x = torch.randn(T, 512, device="cuda").bfloat16()
        w = torch.randn(512, 512, device="cuda").bfloat16()
        y = torch.empty(T, 512, device="cuda", dtype=torch.bfloat16)
        ws = moe.linear_workspace(cfg)
        moe.moe_linear(cfg, x, w, None, None, y, ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.moe_linear(cfg, x, w, None, None, y, ws)
        x.copy_(torch.randn(T, 512, device="cuda"))
        g.replay()
        ref = x.double() @ w.double().t()
        err = (y.double() - ref).abs()
        assert (err <= 2.0 ** -8 * ref.abs() + 1e-2).all()


def test_rows_past_32_bits():
    """Row offsets above 2^31 elements: the last rows of a buffer with a wide stride."""
    T, N, K, stride = 2100, 64, 64, 1 << 20
    buf = torch.empty(T * stride, dtype=torch.bfloat16, device="cuda")
    x = buf.view(T, stride)
    x[:, :K] = torch.randn(T, K, device="cuda").bfloat16()
    w = torch.randn(N, K, device="cuda").bfloat16()
    for t in (4, T):                       # few tokens (the last ones) and all
        cfg = moe.linear_config(t, N, K, x_stride=stride)
        y = torch.empty(t, N, device="cuda", dtype=torch.bfloat16)
        moe.moe_linear(cfg, x[T - t:], w, None, None, y, moe.linear_workspace(cfg))
        ref = x[T - t:, :K].double() @ w.double().t()
        assert ((y.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-2).all()


def test_refusal_raises():
    cfg = moe.linear_config(4, 64, 64)
    t = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(moe.MoEError):
        moe.moe_linear(cfg, t, t, None, None, t, torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(moe.MoEError):
        moe.linear_workspace(moe.linear_config(4, 64, 0))
