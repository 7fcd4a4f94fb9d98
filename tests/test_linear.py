"""moe_linear: refusals on the host, and the GPU kernels against the formula in 64 bits."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

from routed_grouped_gemm_softmax_b200 import api, build


def lin(M=4, N=16, K=32, act=0, out=0, ldx=None, ldw=None, ldr=None, ldo=None):
    return api.Linear(M, N, K, act, out, K if ldx is None else ldx, K if ldw is None else ldw,
                      N if ldr is None else ldr, N if ldo is None else ldo)


def test_host_refusals():
    build.build()
    L = api.lib()
    buf = ctypes.create_string_buffer(8192)
    p = (ctypes.addressof(buf) + 255) // 256 * 256
    assert L.moe_linear_workspace_size() == 256

    def call(d, x=p, w=p, w_up=None, bias=None, bias_up=None, res=None, out=p, ws=p, n=256):
        return L.moe_linear(None if d is None else ctypes.byref(d), x, w, w_up, bias, bias_up, res, out, ws, n, None)

    assert call(None) == 1
    for d in (lin(M=-1), lin(N=0), lin(K=0), lin(act=5), lin(act=-1), lin(out=2), lin(ldx=31), lin(ldx=36), lin(ldw=24),
              lin(ldw=36), lin(ldo=15), lin(K=30)):
        assert call(d) == 1
    assert call(lin(ldr=15), res=p) == 1
    assert call(lin(), x=p + 8) == 1 and call(lin(), w=p + 8) == 1 and call(lin(), w_up=p + 8) == 1
    assert call(lin(), bias=p + 2) == 1 and call(lin(), out=p + 1) == 1 and call(lin(out=1), out=p + 2) == 1
    assert call(lin(), w_up=p, bias_up=p + 2) == 1 and call(lin(), res=p + 1) == 1
    assert call(lin(), bias_up=p) == 1                       # without w_up
    assert call(lin(), x=None) == 1 and call(lin(), w=None) == 1 and call(lin(), out=None) == 1
    assert call(lin(), ws=None) == 3 and call(lin(), ws=p + 16) == 3 and call(lin(), n=255) == 3
    assert call(lin(ldx=1 << 38)) == 2
    assert call(lin(M=(1 << 31) - 1, N=(1 << 31) - 1)) == 2
    assert call(lin(M=0), None, None, None, None, None, None, None, None, 0) == 0


def test_sizes_that_no_longer_round_up_in_32_bits_are_refused():
    build.build()
    L = api.lib()
    buf = ctypes.create_string_buffer(8192)
    p = (ctypes.addressof(buf) + 255) // 256 * 256
    most = 2 ** 31 - 256
    for over in (most + 1, 2 ** 31 - 1):
        for d in (lin(M=over, N=8, K=8), lin(M=1, N=over, K=8), lin(M=1, N=1, K=over, ldx=8, ldw=8)):
            # without a workspace: what is let through comes to that check and no further
            assert L.moe_linear(ctypes.byref(d), p, p, None, None, None, None, p, None, 0, None) == 2
    for d in (lin(M=most, N=8, K=8), lin(M=1, N=most, K=8), lin(M=1, N=1, K=most, ldx=8, ldw=8)):
        assert L.moe_linear(ctypes.byref(d), p, p, None, None, None, None, p, None, 0, None) == 3


def test_python_refusals_need_no_gpu():
    with pytest.raises(ValueError):
        api.moe_linear(torch.zeros(4, 8).bfloat16(), torch.zeros(4, 8).bfloat16())
    with pytest.raises(ValueError):
        api.moe_linear(torch.zeros(8).bfloat16(), torch.zeros(4, 8).bfloat16())


def test_the_fit_of_gelu_s_tail():
    # the constants as the source has them, in fp32, against exp(z^2) erfc(z) in 64 bits
    with open(os.path.join(build.CSRC, "linear.cuh")) as f:
        src = f.read()
    src = src[src.index("float lin_gelu(float v)"):]
    src = src[:src.index("}\n")]
    f32 = lambda m: float(np.float32(m))
    a = f32(re.search(r"fmaf\(([0-9.]+)f, fabsf\(v\)", src).group(1))
    coefs = [f32(c) for c in re.findall(r"float p = ([-+.e0-9]+)f;", src) + re.findall(r"fmaf\(p, x, ([-+.e0-9]+)f\)", src)]
    assert len(coefs) == 11
    t = torch.linspace(1e-9, 1.0, 200001, dtype=torch.float64)
    z = (1.0 / t - 1.0) / a * math.sqrt(0.5)
    p = torch.zeros_like(t)
    for c in coefs:
        p = p * (2.0 * t - 1.0) + c
    assert float((p * t / torch.special.erfcx(z) - 1.0).abs().max()) < 4.5e-8


# ------------------------------------------------------------------ the formula in 64 bits

def act64(v, act):
    if act == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if act == "gelu":
        return 0.5 * v * torch.special.erfc(-v * math.sqrt(0.5))
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    return v


# |d act / dv| is at most this (gelu's slope peaks at 1.13, silu's at 1.10)
SLOPE = 1.13


def check(x, w, bias=None, act="none", residual=None, w_up=None, bias_up=None, out_dtype=torch.bfloat16, **kw):
    r64 = None if residual is None else residual.double()
    out = api.moe_linear(x, w, bias, act, residual, w_up, bias_up, out_dtype=out_dtype, **kw)
    torch.cuda.synchronize()
    c = lambda t: None if t is None else t.double()
    X, W, U = c(x), c(w), c(w_up)
    K = X.shape[1]
    v, mag = X @ W.T, X.abs() @ W.abs().T
    # fp32 sums: every product is exact, a sum of K terms in any order is off by at most K steps of
    # 2^-23 (a tensor core may truncate) of the sum of magnitudes; the bias adds one rounding
    err = K * 2.0 ** -23 * mag
    if bias is not None:
        v = v + c(bias)
        err = err + 2.0 ** -24 * v.abs() + 2.0 ** -24 * err
    y = act64(v, act)
    # the activation's own evaluation: a few units in the last place of the result and of its argument,
    # and gelu_tanh's argument u carries 4 roundings of up to |2u| into the exponent
    u = 2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3).abs().clamp(max=200.0)
    rel = {"none": 0.0, "relu": 0.0}.get(act, (12.0 + (6.0 * u if act == "gelu_tanh" else 4.0 * v.abs().clamp(max=200.0) ** 2
                                                       if act == "gelu" else 2.0 * v.abs().clamp(max=200.0))) * 2.0 ** -24)
    err = SLOPE * err + rel * y.abs() + 2.0 ** -126
    if w_up is not None:
        z, zmag = X @ U.T, X.abs() @ U.abs().T
        zerr = K * 2.0 ** -23 * zmag
        if bias_up is not None:
            z = z + c(bias_up)
            zerr = zerr + 2.0 ** -24 * z.abs()
        err = err * z.abs() + zerr * y.abs() + err * zerr + 2.0 ** -24 * (y * z).abs()
        y = y * z
    if r64 is not None:
        y = y + r64
        err = err + 2.0 ** -24 * y.abs()
    half = torch.finfo(out_dtype).eps / 2  # the one rounding of the result
    tol = err * (1 + half) + half * y.abs()
    d = (out.double() - y).abs()
    bad = ~(d <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, worst {float((d / tol).max()):.2f}, first {bad.nonzero()[0].tolist()}"
    assert out.dtype == out_dtype
    return out


def mat(rows, cols, seed, pad=0, dtype=torch.bfloat16, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(rows, cols + pad, generator=g, device="cuda") * std).to(dtype)[:, :cols]


def operands(M, N, K, pad=0):
    ld = (-K) % 8 + pad  # rows a multiple of 8 apart
    return mat(M, K, 1, ld), mat(N, K, 2, ld, std=K ** -0.5), mat(N, K, 3, ld, std=K ** -0.5)


SHAPES = [(1, 8, 8), (1, 2048, 2048), (1, 1, 1), (2, 130, 64), (7, 257, 1000), (16, 128, 128), (17, 300, 72), (32, 2048, 512),
          (33, 64, 136), (64, 129, 4096), (65, 127, 200), (100, 1, 640), (128, 256, 256), (129, 513, 1416), (255, 384, 90),
          (512, 96, 2048), (1000, 1023, 328), (1024, 1024, 1024), (2049, 520, 264),
          (2100, 2400, 136), (2305, 2071, 64), (4999, 1031, 520), (300, 9500, 700), (9300, 511, 90)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_products(M, N, K):
    x, w, u = operands(M, N, K)
    b, bu = mat(1, N, 4, dtype=torch.float32)[0], mat(1, N, 5, dtype=torch.float32)[0]
    check(x, w)
    check(x, w, out_dtype=torch.float32)
    check(x, w, b, "silu", mat(M, N, 6), u, bu)
    check(x, w, b, "gelu", mat(M, N, 6, 3, torch.float32), out_dtype=torch.float32)
    check(x, w, None, "none", None, u, None, torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("act", list(api.ACTS))
@pytest.mark.parametrize("M,N", [(3, 256), (40, 256), (300, 256), (1100, 256), (5000, 1024)])
def test_activations_over_their_range(act, M, N):
    x, w, u = operands(M, N, 64, 8)
    b = torch.linspace(-12.0, 12.0, N, device="cuda")
    for out_dtype in (torch.bfloat16, torch.float32):
        check(x, w, b, act, out_dtype=out_dtype)
        check(x, w, b * 20, act, w_up=u, out_dtype=out_dtype)  # far past where exp leaves fp32


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 100, 64), (16, 1000, 200), (50, 255, 130), (300, 333, 512), (1500, 1030, 136), (2500, 2050, 72)])
def test_strides_in_place_and_rows_behind(M, N, K):
    x, w, u = operands(M, N, K, 16)
    for dtype in (torch.bfloat16, torch.float32):
        for pad in (0, 1, 4, 8):
            big = mat(M + 2, N, 7, pad, dtype).clone()
            keep = big.clone()
            r = mat(M, N, 8, 3, dtype)
            out = big.as_strided((M, N), (N + pad, 1)) if pad == 0 else torch.empty(M + 2, N + pad, dtype=dtype, device="cuda")
            if pad:
                out.fill_(7.0)
                check(x, w, None, "relu", r, out_dtype=dtype, out=out[:M, :N])
                assert bool((out[M:] == 7.0).all()) and bool((out[:, N:] == 7.0).all())
            else:
                check(x, w, None, "relu", r, out_dtype=dtype, out=out)
                assert torch.equal(big.view(-1)[M * N:], keep.view(-1)[M * N:])
        res = mat(M, N, 9, 5, dtype).clone()
        check(x, w, None, "silu", res, u, out_dtype=dtype, out=res)     # onto the residual


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(257, 4104, 200), (1500, 1000, 136), (2600, 2056, 72), (3001, 520, 1100), (129, 2048, 2048)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_and_columns_behind_aligned_outputs(M, N, K, dtype):
    # rows of out 16-byte aligned, M and N not multiples of any tile: nothing behind either is written
    x, w, u = operands(M, N, K)
    b = mat(1, N, 4, dtype=torch.float32)[0]
    for pad in (0, 8, 24):
        for gate, act in ((None, "gelu"), (u, "silu")):
            out = torch.full((M + 3, N + pad), 7.0, dtype=dtype, device="cuda")
            check(x, w, b, act, mat(M, N, 8, 16, dtype), gate, out_dtype=dtype, out=out[:M, :N])
            assert bool((out[M:] == 7.0).all()) and bool((out[:, N:] == 7.0).all())
            check(x, w, None, act, None, gate, out_dtype=dtype, out=out[:M, :N])
            assert bool((out[M:] == 7.0).all()) and bool((out[:, N:] == 7.0).all())
            res = mat(M, N, 9, pad, dtype).clone()
            check(x, w, b, act, res, gate, out_dtype=dtype, out=res)     # onto the residual
    # one of the two not aligned
    out = torch.empty(M, N + 8, dtype=dtype, device="cuda")
    check(x, w, b, "relu", mat(M, N, 8, 3, dtype), out_dtype=dtype, out=out[:, :N])
    check(x, w, b, "relu", mat(M, N, 8, 8, dtype), out_dtype=dtype, out=out[:, 1:N + 1])


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,ld", [(36000, 64, 60000), (36000, 70, 60001), (64, 96, 35000000)])
def test_offsets_past_32_bits(M, N, ld):
    # rows of out and residual more than 2^31 elements from the first
    assert (M - 1) * ld > 2 ** 31
    K = 72
    x, w, _ = operands(M, N, K)
    big = torch.empty(M * ld, dtype=torch.bfloat16, device="cuda")
    out = big.as_strided((M, N), (ld, 1))
    out.copy_(mat(M, N, 8))
    check(x, w, None, "silu", out, out=out)  # onto the residual
    ldx = ld // 8 * 8
    far = big.as_strided((M, K), (ldx, 1))
    far.copy_(x)
    assert torch.equal(api.moe_linear(far, w), api.moe_linear(x.contiguous(), w))


@pytest.mark.gpu
@pytest.mark.parametrize("act", list(api.ACTS))
@pytest.mark.parametrize("M", [5, 200, 2000])
def test_activations_of_extreme_values(act, M):
    # as the formula in 64 bits has them, NaN where that is NaN
    v = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e-42, 3e4, -3e4, 1e20, -1e20, 3e38, -3e38, math.inf, -math.inf, math.nan, 88.0, -88.0,
                      -103.0, 13.0, -13.0], device="cuda")
    N = 512
    b = v.repeat(N // v.numel() + 1)[:N].contiguous()
    x, w = torch.zeros(M, 64, device="cuda").bfloat16(), torch.zeros(N, 64, device="cuda").bfloat16()
    got = api.moe_linear(x, w, b, act, out_dtype=torch.float32)
    want = act64(b.double(), act)
    if act == "gelu_tanh":  # 1 + tanh loses all it has left of 64 bits below -5; the same formula by exp keeps it
        z = 2.0 * math.sqrt(2.0 / math.pi) * (b.double() + 0.044715 * b.double() ** 3)
        want = torch.where(b < 0, b.double() * torch.exp(z) / (1.0 + torch.exp(z)), want)
    # a relative error that grows with the exponent (up to 6 roundings of an argument of up to 104), and
    # what fp32 cannot hold
    tol = (12.0 + 6.0 * 104.0) * 2.0 ** -24 * want.abs() + 2.0 ** -125
    same = (got.double() == want) | (torch.isnan(want) & torch.isnan(got)) | ((got.double() - want).abs() <= tol)
    assert bool(same.all()), [(float(b[i]), float(got[j, i]), float(want[i])) for j, i in (~same).nonzero()[:5].tolist()]


@pytest.mark.gpu
def test_what_lies_outside_the_operands_is_not_read_into_the_sums():
    # NaN behind the rows, columns and depth of every operand
    for M, N, K in ((5, 70, 72), (130, 200, 100), (1030, 600, 136), (2570, 2100, 100)):
        full = [torch.full((n + 40, K + 40 + (-K) % 8), math.nan, dtype=torch.bfloat16, device="cuda") for n in (M, N, N)]
        ops = [f[:n, :K] for f, n in zip(full, (M, N, N))]
        for o, src in zip(ops, operands(M, N, K)):
            o.copy_(src)
        check(ops[0], ops[1], None, "silu", None, ops[2])


@pytest.mark.gpu
def test_infinities_and_nan_stay_in_their_row_and_column():
    M, N, K = 40, 200, 128
    x, w, _ = operands(M, N, K)
    x, w = x.clone(), w.clone()
    x[3, 5] = math.nan
    w[17, 9] = math.nan
    out = api.moe_linear(x, w, None, "relu")
    nan = torch.isnan(out)
    assert bool(nan[3].all()) and bool(nan[:, 17].all())
    nan[3] = False
    nan[:, 17] = False
    assert not bool(nan.any())
    y = api.moe_linear(x * 0, w * 0, torch.full((N,), -math.inf, device="cuda"), "relu")
    assert bool((y[:3, :17] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(1, 520), (24, 520), (200, 520), (1300, 520), (3000, 1500)])
def test_repeatable_streams_and_replay(M, N):
    x, w, u = operands(M, N, 776)
    b = mat(1, N, 4, dtype=torch.float32)[0]
    ws = api.linear_workspace("cuda")
    ref = api.moe_linear(x, w, b, "gelu", w_up=u, ws=ws)
    assert torch.equal(ref, api.moe_linear(x, w, b, "gelu", w_up=u, ws=ws))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = [api.moe_linear(x, w, b, "gelu", w_up=u, stream=s) for _ in range(3)]
    here = [api.moe_linear(x, w, b, "gelu", w_up=u, ws=ws) for _ in range(3)]
    s.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(ref, o) for o in other + here)
    out = torch.empty_like(ref)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:  # two graphs on one workspace
        with torch.cuda.graph(g):
            api.moe_linear(x, w, b, "gelu", w_up=u, ws=ws, out=out)
    x.copy_(mat(M, 776, 21))
    for g in graphs:
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        check(x, w, b, "gelu", w_up=u)
        assert torch.equal(out, api.moe_linear(x, w, b, "gelu", w_up=u))
    assert api.moe_get_device_status(ws) == api.MOE_OK


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(8, 512), (100, 512), (2000, 512), (5000, 1024)])
def test_a_wait_that_runs_out_is_reported_and_recoverable(M, N):
    x, w, _ = operands(M, N, 1024)
    ws = api.linear_workspace("cuda")
    ref = api.moe_linear(x, w, ws=ws)
    api.set_wait_limit_us(20000, stall_test=True)
    try:
        api.moe_linear(x, w, ws=ws)
        assert api.moe_get_device_status(ws) == 5
    finally:
        api.set_wait_limit_us(0)
    assert torch.equal(ref, api.moe_linear(x, w, ws=ws))
    assert api.moe_get_device_status(ws) == api.MOE_OK


@pytest.mark.gpu
def test_python_refusals():
    x, w, u = operands(4, 16, 32)
    b = torch.zeros(16, device="cuda")
    for bad in (lambda: api.moe_linear(x.float(), w), lambda: api.moe_linear(x, w[:, :24]), lambda: api.moe_linear(x, w.cpu()),
                lambda: api.moe_linear(x, w, b.bfloat16()), lambda: api.moe_linear(x, w, b[:8]), lambda: api.moe_linear(x, w, act="tanh"),
                lambda: api.moe_linear(x, w, residual=torch.zeros(4, 16, device="cuda")),
                lambda: api.moe_linear(x, w, w_up=torch.zeros(16, 40, device="cuda").bfloat16()[:, :32]),
                lambda: api.moe_linear(x, w, out=torch.zeros(16, 4, device="cuda").bfloat16().t()),
                lambda: api.moe_linear(x.t(), x.t()), lambda: api.moe_linear(x, w, out_dtype=torch.float16)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: api.moe_linear(x, w, bias_up=b), lambda: api.moe_linear(x[:, 4:20], w[:, 4:20]),
                lambda: api.moe_linear(x.expand(2, 4, 32)[0][:1].expand(4, 32), w),
                lambda: api.moe_linear(mat(4, 30, 1), mat(16, 30, 1)),
                lambda: api.moe_linear(x, w, ws=torch.zeros(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(api.MoEError):
            bad()
    assert api.moe_linear(x[:0], w).shape == (0, 16)


@pytest.mark.gpu
def test_sizes_past_32_bits_are_refused():
    # 2^32 + 4 rows are not 4
    big = torch.empty(1, 8, dtype=torch.bfloat16, device="cuda").expand(2 ** 32 + 4, 8)
    for bad in (lambda: api.moe_linear(big, big[:1]), lambda: api.moe_linear(big[:1], big)):
        with pytest.raises(api.MoEError) as e:
            bad()
        assert e.value.code == 2


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 5, 300])
def test_one_column_whose_gate_and_up_rows_lie_apart(M):
    # of a single row no stride is read: w a row of a wide matrix, w_up one of its own
    x, w, u = mat(M, 64, 1), mat(1, 64, 2, 24), mat(1, 64, 3)
    check(x, w, None, "silu", None, u)
    check(x, u, None, "silu", None, w)


@pytest.mark.gpu
@pytest.mark.parametrize("M,K", [(1000, 72), (257, 1100), (2600, 40)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_columns_behind_rows_that_end_inside_16_bytes(M, K, dtype):
    # rows 16-byte aligned, N any: out a slice of a wider buffer whose other columns stay as they were,
    # down to the last row's, behind which a buffer may end
    for N in (2043, 2044, 2045, 2046, 2047, 2049, 2050, 2082, 4100):
        x, w, u = operands(M, N, K)
        b = mat(1, N, 4, dtype=torch.float32)[0]
        pad = (-N) % 8 + 8
        for gate, act, res in ((None, "gelu", None), (u, "silu", None), (None, "none", "apart"), (u, "relu", "in place")):
            big = torch.full((M + 1, N + pad), 7.0, dtype=dtype, device="cuda")
            out, r = big[:M, :N], None
            if res == "apart":
                r = mat(M, N, 8, pad, dtype)
            elif res:
                out.copy_(mat(M, N, 9, 0, dtype))
                r = out
            check(x, w, b, act, r, gate, out_dtype=dtype, out=out)
            assert bool((big[M:] == 7.0).all()) and bool((big[:, N:] == 7.0).all()), (N, gate is not None, res)
