"""The tile kernel on hundreds of causal documents with more queries than keys: work items whose first 128 queries see
no key follow items with fewer than 128 queries, each ending inside a tile of keys, and each CTA takes several.
Against the definition in 64 bits, within the tolerance of tests/test_gpu_attention.py."""
import pytest
import torch

from tests.test_gpu_attention import check, starts, tensor

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def w8():
    import w8a8_int8_gemm_b200 as mod
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return mod


MORE_QUERIES = {
    "300 over 50": [(300, 50)] * 200,
    "200 over 50": [(200, 50)] * 400,
    "by turns": [(100, 30), (200, 60), (256, 100), (128, 127), (300, 1), (250, 33)] * 100,
    "no keys between": [(200, 50), (130, 0), (300, 70), (0, 9), (1, 1)] * 100,
}


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("name", list(MORE_QUERIES))
def test_more_queries_than_keys_in_many_items(w8, name, D):
    docs, H = MORE_QUERIES[name], 4
    lq, lk = [a for a, _ in docs], [b for _, b in docs]
    cu_q, cu_k = starts(lq), starts(lk)
    q, k, v = tensor(sum(lq), H, D, seed=7), tensor(sum(lk), 2, D, seed=8), tensor(sum(lk), 2, D, seed=9)
    got = []
    for _ in range(3):
        lse = torch.full((sum(lq), H), 9.0, device=DEV)
        got.append((w8.w8a8_attention(q, k, v, cu_q=cu_q, cu_k=cu_k, causal=True, lse=lse, kernel=w8.ATTENTION_TILES),
                    lse))
    torch.cuda.synchronize()
    assert w8.w8a8_read_device_error() == 0
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
    at = list(range(0, len(docs), 13)) + [len(docs) - 1]
    for d in at:
        (a, b), (c, e) = (int(cu_q[d]), int(cu_q[d + 1])), (int(cu_k[d]), int(cu_k[d + 1]))
        check(got[0][0][a:b], got[0][1][a:b], q[a:b], k[c:e], v[c:e], [0, b - a], [0, e - c], D ** -0.5, causal=True)
