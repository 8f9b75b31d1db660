"""The gated linear layer (w8a8_gemm_glu, w8a8_linear_glu, their FP8 forms and a chain's gated layer) on the GPU
against out = act(g) * u in 64 bits on the same codes.

Tolerance.  g = (acc * sa) * sw + b: acc is exact (int8) or off by at most K * 2^-23 * sum |products| (E4M3, the
library's bound for its accumulator); its conversion, two products and the sum round once each, so g is off by
e_g <= 2^-22 (|acc sa sw| + |b|) + (accumulator's error) * sa sw, and u likewise.  SiLU and GELU change by at
most 1.13 per unit of g, and are themselves evaluated to 2^-15 of their value; the result rounds once to bf16
(half a step, 2^-8).  In sum |out - exact| <= (2^-8 + 2^-15) |exact| + 1.2 e_g (|u| + e_u) + |act(g)| e_u,
plus 1e-30 for activations below binary32's normal range."""
import math

import numpy as np
import pytest
import torch

import oracle
from tests.util import bf16_bits_to_torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def w8():
    import w8a8_int8_gemm_b200 as mod
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return mod


def act64(g, act, w8):
    a = 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3) if act == w8.ACT_GELU else g
    return torch.where(a > -700, g / (1 + torch.exp(-a.clamp(min=-700))), torch.zeros_like(g))


def check(w8, got, xq, wq, sa, sw, bias, act):
    """got against the definition on these codes (int8, or E4M3 in uint8)."""
    f = torch.float64
    fp8 = wq.dtype == torch.uint8
    x, w = [(c.view(torch.float8_e4m3fn) if fp8 else c).to(f) for c in (xq, wq)]
    N, K = wq.shape[0] // 2, wq.shape[1]
    s = sa.to(f)[:, None] * sw.to(f)
    b = torch.zeros(2 * N, dtype=f, device=DEV) if bias is None else bias.to(f)
    acc = x @ w.T
    y = acc * s + b
    e = (acc * s).abs() * 2.0 ** -22 + b.abs() * 2.0 ** -22
    if fp8:
        e = e + K * 2.0 ** -23 * (x.abs() @ w.abs().T) * s
    g, u, eg, eu = y[:, :N], y[:, N:], e[:, :N], e[:, N:]
    a = act64(g, act, w8)
    want = a * u
    tol = want.abs() * (2.0 ** -8 + 2.0 ** -15) + 1.2 * eg * (u.abs() + eu) + a.abs() * eu + 1e-30
    off = (got.to(f) - want).abs()
    assert bool((off <= tol).all()), f"off by up to {float((off / tol).max())} tolerances"


def inputs(w8, M, N, K, fp8, seed=0, std=0.5):
    rng = np.random.default_rng([seed, M, N, K])
    x = torch.from_numpy((rng.standard_normal((M, K)) * 2).astype(np.float32)).bfloat16().to(DEV)
    w = torch.from_numpy((rng.standard_normal((2 * N, K)) * std / math.sqrt(K)).astype(np.float32)).to(DEV)
    bias = torch.from_numpy((rng.standard_normal(2 * N) * 0.5).astype(np.float32)).bfloat16().to(DEV)
    wq, sw = (w8.w8a8_quantize_weight_fp8 if fp8 else w8.w8a8_quantize_weight)(w)
    return x, wq, sw, bias


def quantize(w8, x, fp8):
    return (w8.w8a8_quantize_act_fp8 if fp8 else w8.w8a8_quantize_act)(x)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 8, 16), (1, 136, 256), (3, 64, 48), (64, 128, 256), (127, 72, 144),
                                   (129, 256, 128), (130, 264, 2064), (300, 1032, 512), (1000, 520, 1008),
                                   (257, 2048, 384)])
def test_linear_glu(w8, M, N, K, fp8):
    x, wq, sw, bias = inputs(w8, M, N, K, fp8)
    linear = w8.w8a8_linear_glu_fp8 if fp8 else w8.w8a8_linear_glu
    xq0, sa0 = quantize(w8, x, fp8)
    for act in (w8.ACT_SILU, w8.ACT_GELU):
        xq = torch.empty((M, K), dtype=torch.uint8 if fp8 else torch.int8, device=DEV)
        sa = torch.empty(M, device=DEV)
        out = linear(x, wq, sw, bias, act=act, ws_xq=xq, ws_scale_a=sa)
        assert torch.equal(xq, xq0) and torch.equal(sa, sa0)  # the workspaces hold w8a8_quantize_act's results
        check(w8, out, xq, wq, sa, sw, bias, act)
    check(w8, linear(x, wq, sw, act=w8.ACT_SILU), xq0, wq, sa0, sw, None, w8.ACT_SILU)


# every tile shape, ring depth and grid, half-width tail items and several tiles per CTA among them; guard rows
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("cfg", [dict(block_m=128, block_n=256, stages=4, grid=3, raster_group=2),
                                 dict(block_m=128, block_n=128, stages=6, grid=5, raster_group=1),
                                 dict(block_m=128, block_n=128, stages=2, grid=148, raster_group=8),
                                 dict(block_m=256, block_n=256, stages=6, grid=16, raster_group=1),
                                 dict(block_m=256, block_n=256, stages=3, grid=4, raster_group=2),
                                 dict(block_m=256, block_n=128, stages=8, grid=6, raster_group=8),
                                 dict(block_m=256, block_n=128, stages=2, grid=148, raster_group=1)])
@pytest.mark.parametrize("M,N,K", [(300, 328, 384), (513, 456, 272)])
def test_every_tile_configuration(w8, M, N, K, cfg, fp8):
    x, wq, sw, bias = inputs(w8, M, N, K, fp8, seed=1)
    xq, sa = quantize(w8, x, fp8)
    gemm = w8.w8a8_gemm_glu_fp8_ex if fp8 else w8.w8a8_gemm_glu_ex
    buf = torch.full((M + 2, N), 3.0, dtype=torch.bfloat16, device=DEV)
    out = gemm(xq, wq, sa, sw, bias, out=buf[1:-1], act=w8.ACT_SILU, config=cfg)
    check(w8, out, xq, wq, sa, sw, bias, w8.ACT_SILU)
    assert bool((buf[0] == 3).all()) and bool((buf[-1] == 3).all())
    again = gemm(xq, wq, sa, sw, bias, act=w8.ACT_SILU)  # the selected configuration: the same bits for int8
    if not fp8:
        assert torch.equal(again, out)


def test_gate_over_its_range(w8):
    """A gate from far below to far above 0, zero rows and the largest accumulators: one-hot codes make g and u
    plain numbers."""
    K, N, M = 256, 256, 256
    vals = torch.linspace(-120, 120, M, device=DEV)
    xq = torch.zeros((M, K), dtype=torch.int8, device=DEV)
    xq[:, 0] = 1
    xq[0] = 0
    xq[1] = 127
    wq = torch.zeros((2 * N, K), dtype=torch.int8, device=DEV)
    wq[:, 0] = torch.randint(-127, 128, (2 * N,), device=DEV, dtype=torch.int8)
    wq[:2] = 127
    wq[N + 1] = -127
    sa = vals / 127
    sw = torch.ones(2 * N, device=DEV)
    for act in (w8.ACT_SILU, w8.ACT_GELU):
        check(w8, w8.w8a8_gemm_glu(xq, wq, sa, sw, act=act), xq, wq, sa, sw, None, act)


def test_against_two_linear_layers(w8):
    """The gate's two projections are w8a8_linear's: identity weights on one of them give the other's value."""
    M, N, K = 200, 264, 512
    x, wq, sw, bias = inputs(w8, M, N, K, False, seed=3)
    half = w8.w8a8_linear(x, wq[N:].contiguous(), sw[N:].contiguous(), bias[N:].contiguous())
    wq2, bias2 = wq.clone(), bias.clone()
    wq2[:N] = 0
    bias2[:N] = 100.0                               # silu(100) = 100 in binary32
    got = w8.w8a8_linear_glu(x, wq2, sw, bias2)
    assert bool(((got.double() - 100 * half.double()).abs() <= (100 * half.double()).abs() * 2.0 ** -7).all())


def test_against_the_oracle(w8):
    """Codes, scales and accumulators of the CPU oracle, the gate in 64 bits on the host."""
    M, N, K = 70, 72, 144
    rng = np.random.default_rng(5)
    xb = oracle.f32_to_bf16_bits((rng.standard_normal((M, K)) * 3).astype(np.float32))
    wq, sw = oracle.quantize_weight((rng.standard_normal((2 * N, K)) * 0.1).astype(np.float32))
    xq, sa = oracle.quantize_act(xb)
    y = oracle.gemm_i64(xq, wq).astype(np.float64) * sa.astype(np.float64)[:, None] * sw.astype(np.float64)
    g, u = y[:, :N], y[:, N:]
    want = g / (1 + np.exp(-g)) * u
    got = w8.w8a8_linear_glu(bf16_bits_to_torch(xb, DEV), torch.from_numpy(wq).to(DEV), torch.from_numpy(sw).to(DEV))
    off = np.abs(got.double().cpu().numpy() - want)
    e = np.abs(y) * 2.0 ** -22
    tol = np.abs(want) * (2.0 ** -8 + 2.0 ** -15) + 1.2 * e[:, :N] * (np.abs(u) + e[:, N:]) + np.abs(g) * e[:, N:]
    assert bool((off <= tol + 1e-30).all())


def test_chain_with_a_gated_layer(w8):
    """A gated MLP as one graph: up (gated), then down; the same bits as the two calls, on two launches."""
    M, H, F = 333, 256, 528
    x, wq, sw, bias = inputs(w8, M, F, H, False, seed=6)
    _, wd, sd, bd = inputs(w8, 1, H // 2, F, False, seed=7)  # a plain weight of H rows
    up = w8.linear_layer(x, wq, sw, bias, output_glu=w8.ACT_SILU)
    down = w8.linear_layer(up["out"], wd, sd, bd)
    chain = w8.w8a8_chain_create([up, down])
    for seed in (8, 9):
        x.copy_(inputs(w8, M, F, H, False, seed=seed)[0])
        chain.launch()
        h = w8.w8a8_linear_glu(x, wq, sw, bias)
        want = w8.w8a8_linear(h, wd, sd, bd)
        torch.cuda.synchronize()
        assert torch.equal(up["out"], h) and torch.equal(down["out"], want)
    chain.close()


def test_captured_and_other_stream(w8):
    x, wq, sw, bias = inputs(w8, 150, 200, 256, False, seed=10)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.zeros((150, 200), dtype=torch.bfloat16, device=DEV)
    ws, sa = torch.empty_like(x, dtype=torch.int8), torch.empty(150, device=DEV)
    w8.w8a8_linear_glu(x, wq, sw, bias, out=out, ws_xq=ws, ws_scale_a=sa, stream=s)
    s.synchronize()
    want = w8.w8a8_linear_glu(x, wq, sw, bias)
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w8.w8a8_linear_glu(x, wq, sw, bias, out=out, ws_xq=ws, ws_scale_a=sa)
    x.copy_(inputs(w8, 150, 200, 256, False, seed=11)[0])
    g.replay()
    torch.cuda.synchronize()
    check(w8, out, ws, wq, sa, sw, bias, w8.ACT_SILU)


def test_workspace_of_a_call_on_another_stream(w8):
    """A workspace allocated inside the call belongs to the call's stream: the current stream may not get its memory
    back while the other stream still has the call ahead of it."""
    x, wq, sw, bias = inputs(w8, 512, 256, 1024, False, seed=12)
    want = w8.w8a8_linear_glu(x, wq, sw, bias)
    busy = torch.randn(8192, 8192, device=DEV).bfloat16()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for as_number in (False, True):
        with torch.cuda.stream(s):
            for _ in range(20):
                busy = (busy @ busy) * 1e-3
        out = w8.w8a8_linear_glu(x, wq, sw, bias, stream=s.cuda_stream if as_number else s)
        for n in (512 * 1024, 512 * 1024 + 2048, 2048, 512 * 256 * 2):  # the sizes that could be handed out again
            torch.full((n,), 77, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_empty_and_refusals(w8):
    x, wq, sw, bias = inputs(w8, 4, 16, 32, False)
    assert w8.w8a8_linear_glu(x[:0], wq, sw, bias).shape == (0, 16)
    for act in (0, 3, -1):
        with pytest.raises(w8.W8A8Error) as e:
            w8.w8a8_linear_glu(x, wq, sw, bias, act=act)
        assert e.value.status == 1
    with pytest.raises(ValueError):
        w8.w8a8_linear_glu(x, wq[:31].contiguous(), sw[:31].contiguous())   # an odd number of rows
    with pytest.raises(ValueError):
        w8.w8a8_linear_glu(x, wq, sw[:16].contiguous())
    with pytest.raises(TypeError):
        w8.w8a8_linear_glu_fp8(x, wq, sw)
    with pytest.raises(w8.W8A8Error):
        w8.w8a8_linear_glu(x, wq[:24].contiguous(), sw[:24].contiguous())   # N = 12
    with pytest.raises(w8.W8A8Error):
        w8.w8a8_chain_create([w8.linear_layer(x, wq, sw, bias, input_act=w8.ACT_GELU, output_glu=w8.ACT_SILU)])
