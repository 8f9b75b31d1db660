"""A work item that takes longer than the limit of a wait: the warps that have nothing to do in it, and the one that waits
for its end, do not give up."""
import pytest
import torch

from tests.test_gpu_attention import check, tensor

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("queries", [100, 256])
def test_an_item_of_thousands_of_tiles(queries, D):
    import w8a8_int8_gemm_b200 as w8
    keys = 400_003  # some 3 and 5 ms
    q, k, v = tensor(queries, 2, D), tensor(keys, 1, D, seed=2), tensor(keys, 1, D, seed=3)
    lse = torch.empty(queries, 2, device=DEV)
    w8.w8a8_attention(q, k[:5], v[:5], kernel=w8.ATTENTION_TILES)
    torch.cuda.synchronize()
    w8.w8a8_set_wait_timeout_ns(1_000_000)
    try:
        out = w8.w8a8_attention(q, k, v, lse=lse, kernel=w8.ATTENTION_TILES)
        assert w8.w8a8_read_device_error() == 0
    finally:
        w8.w8a8_set_wait_timeout_ns(2_000_000_000)
    rows = list(range(0, queries, 37))
    check(out[rows], lse[rows], q[rows], k, v, [0, len(rows)], [0, keys], D ** -0.5)
