"""Calls on a stream other than the current one: the workspaces, outputs and counters that a call makes for itself belong
to its stream, so the current stream gets their memory neither back nor under way while the other one still has the
call ahead of it."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def w8():
    import w8a8_int8_gemm_b200 as mod
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return mod


def layer(w8, fp8):
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(512, 1024, generator=g, device=DEV).bfloat16()
    w = torch.randn(256, 1024, generator=g, device=DEV)
    wq, sw = (w8.w8a8_quantize_weight_fp8 if fp8 else w8.w8a8_quantize_weight)(w)
    return x, wq, sw, torch.randn(256, generator=g, device=DEV).bfloat16()


@pytest.mark.parametrize("name", ["w8a8_linear", "w8a8_linear_fp8", "w8a8_linear_fused", "w8a8_linear_gelu"])
def test_a_layer_behind_other_work(w8, name):
    x, wq, sw, bias = layer(w8, "fp8" in name)
    call = getattr(w8, name)
    want = call(x, wq, sw, bias)
    busy = torch.randn(8192, 8192, device=DEV).bfloat16()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        with torch.cuda.stream(s):
            for _ in range(20):
                busy = (busy @ busy) * 1e-3
        out = call(x, wq, sw, bias, stream=stream)
        for n in (512 * 1024, 2048, 512 * 256 * 2, 20):  # the sizes that could be handed out again
            torch.full((n,), 77, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert w8.w8a8_read_device_error() == 0


def test_the_default_stream_by_its_handle(w8):
    """A handle of 0 is the default stream, for allocations too."""
    x, wq, sw, bias = layer(w8, False)
    want = w8.w8a8_linear(x, wq, sw, bias)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with w8._on(0, x.device):
            assert torch.cuda.current_stream().cuda_stream == 0
        out = w8.w8a8_linear(x, wq, sw, bias, stream=0)
        xq, _ = w8.w8a8_quantize_act(x, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(xq, w8.w8a8_quantize_act(x)[0])
