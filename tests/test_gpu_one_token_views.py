"""One token of a large head-major buffer: the stride of a dimension of one is free, however long the others are."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
HEADS, TOKENS, D = 32, 2 ** 20, 64  # 2^31 values


@pytest.fixture(scope="module")
def buffer():
    b = torch.empty(HEADS, TOKENS, D, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    b[:, 77] = torch.randn(HEADS, D, generator=g, device=DEV).bfloat16()
    return b


@pytest.fixture(scope="module")
def w8():
    import w8a8_int8_gemm_b200 as mod
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return mod


def test_attention(w8, buffer):
    one = buffer[:, 77:78].transpose(0, 1)  # [1, heads, D]
    packed = one.contiguous()
    many = torch.randn(40, HEADS, D, device=DEV).bfloat16()
    out = torch.zeros(HEADS, 3, D, dtype=torch.bfloat16, device=DEV)
    for kernel in (w8.ATTENTION_ROWS, w8.ATTENTION_TILES):
        for q, k, v in ((0, 1, 1), (1, 0, 0), (0, 0, 0)):
            a = [one if x == 0 else many for x in (q, k, v)]
            b = [packed if x == 0 else many for x in (q, k, v)]
            assert torch.equal(w8.w8a8_attention(*a, kernel=kernel), w8.w8a8_attention(*b, kernel=kernel))
        w8.w8a8_attention(one, many, many, out=out[:, 1:2].transpose(0, 1), kernel=kernel)
        assert torch.equal(out[:, 1], w8.w8a8_attention(packed, many, many, kernel=kernel)[0])
        assert not bool(out[:, 0].any()) and not bool(out[:, 2].any())


def test_norm_and_rotation(w8, buffer):
    one = buffer[:, 77:78].transpose(0, 1)
    cos, sin = torch.rand(1, D // 2, device=DEV), torch.rand(1, D // 2, device=DEV)
    packed = one[:, :4].contiguous()
    want = w8.w8a8_qk_norm_rope(one.contiguous(), packed, cos=cos, sin=sin)
    got = w8.w8a8_qk_norm_rope(one, one[:, :4], cos=cos, sin=sin)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    w8.w8a8_qk_norm_rope(one, packed, cos=cos, sin=sin, q_out=one)  # in place
    assert torch.equal(one, want[0])
