"""The gated GEMM's output where a warp's consecutive stores are of the same step of their tiles: tiles with one step
(block_n 128), and outputs that end inside a tile of two (N mod 128 in 1..32 or 65..96), many tiles to a CTA, short
K.  The accumulators are integers, so every configuration gives the same bits; the widest tile on full columns is
checked against 64 bits elsewhere."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def w8():
    import w8a8_int8_gemm_b200 as mod
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return mod


def operands(M, N, K, fp8, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    if fp8:  # small whole numbers: every sum is exact in binary32
        xq, wq = [torch.randint(-8, 9, s, generator=g, device=DEV).float().to(torch.float8_e4m3fn).view(torch.uint8)
                  for s in ((M, K), (2 * N, K))]
    else:
        xq, wq = [torch.randint(-127, 128, s, generator=g, device=DEV, dtype=torch.int8) for s in ((M, K), (2 * N, K))]
    sa = torch.rand(M, generator=g, device=DEV) * 1e-2
    sw = torch.rand(2 * N, generator=g, device=DEV) * 1e-2
    return xq, wq, sa, sw


def padded(wq, sw, N, to):
    """The same weights with zero columns up to `to`, a multiple of 128: no store is left out."""
    w = torch.zeros((2 * to, wq.shape[1]), dtype=wq.dtype, device=DEV)
    s = torch.zeros(2 * to, device=DEV)
    w[:N], w[to:to + N] = wq[:N], wq[N:]
    s[:N], s[to:to + N] = sw[:N], sw[N:]
    return w, s


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("N", [8, 24, 32, 72, 96, 136, 200, 264, 328, 5640])
@pytest.mark.parametrize("block_m,block_n,grid", [(128, 128, 2), (128, 256, 2), (256, 128, 4), (256, 256, 4),
                                                  (128, 128, 148), (128, 256, 148), (256, 256, 148)])
def test_consecutive_stores_of_one_step(w8, block_m, block_n, grid, N, fp8):
    K = 32
    M = 2305 if N > 1000 else 20480 if grid < 148 else 128000  # many tiles to a CTA
    xq, wq, sa, sw = operands(M, N, K, fp8, seed=N)
    gemm = w8.w8a8_gemm_glu_fp8_ex if fp8 else w8.w8a8_gemm_glu_ex
    cfg = dict(block_m=block_m, block_n=block_n, stages=2, grid=grid, raster_group=1)
    full_wq, full_sw = padded(wq, sw, N, (N + 127) // 128 * 128)
    full = gemm(xq, full_wq, sa, full_sw, config=dict(cfg, block_m=128, block_n=256, grid=148))
    want = full[:, :N].contiguous()
    for _ in range(3):
        out = torch.full((M, N), 3.0, dtype=torch.bfloat16, device=DEV)
        gemm(xq, wq, sa, sw, out=out, config=cfg)
        assert torch.equal(out, want)
    assert w8.w8a8_read_device_error() == 0
