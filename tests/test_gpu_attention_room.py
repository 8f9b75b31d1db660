"""Caches with room to grow in one buffer: the unused room between them is stated as documents without queries, and may
hold anything.  Each sequence against itself alone, within the tolerance of tests/test_gpu_attention.py."""
import pytest
import torch

from tests.test_gpu_attention import check, tensor

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kernel", [0, 1, 2])
@pytest.mark.parametrize("new", [1, 3, 150])
def test_caches_in_place(new, kernel, D):
    import w8a8_int8_gemm_b200 as w8
    used, room, Hq, Hk = [700, 150, 1999, 2000, 256], 2000, 8, 2
    n = len(used)
    k, v = tensor(n * room, Hk, D, seed=2), tensor(n * room, Hk, D, seed=3)
    q = tensor(n * new, Hq, D, seed=1)
    cu_q, cu_k = [0], [0]
    for i, u in enumerate(used):  # document 2 i: the cache; 2 i + 1: its room
        k[i * room + u:(i + 1) * room] = float("nan")
        v[i * room + u:(i + 1) * room] = float("nan")
        cu_q += [(i + 1) * new] * 2
        cu_k += [i * room + u, (i + 1) * room]
    starts = [torch.tensor(c, dtype=torch.int32, device=DEV) for c in (cu_q, cu_k)]
    lse = torch.empty(n * new, Hq, device=DEV)
    out = w8.w8a8_attention(q, k, v, causal=True, cu_q=starts[0], cu_k=starts[1], lse=lse, kernel=kernel)
    for i, u in enumerate(used):
        a, c = i * new, i * room
        check(out[a:a + new], lse[a:a + new], q[a:a + new], k[c:c + u], v[c:c + u], [0, new], [0, u], D ** -0.5,
              causal=True)
    assert w8.w8a8_read_device_error() == 0
