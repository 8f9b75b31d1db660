"""The tile that the gated GEMM selects where K is no multiple of 128: the launch on single CTAs makes no half-width
items, so a short last round of them costs a whole one, and CTA pairs with fewer rounds are taken.  (Every
configuration gives the same bits: the kernels are compared as a captured graph names them.)"""
import re

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
SINGLE = dict(block_m=128, block_n=256, stages=4, grid=148, raster_group=1)
PAIR = dict(block_m=256, block_n=256, stages=6, grid=148, raster_group=1)


@pytest.fixture(scope="module")
def w8():
    import w8a8_int8_gemm_b200 as mod
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return mod


def kernel(w8, path, M, N, K, config):
    """The name of the kernel that the call launches."""
    xq = torch.zeros((M, K), dtype=torch.int8, device=DEV)
    wq = torch.zeros((2 * N, K), dtype=torch.int8, device=DEV)
    sa, sw = torch.ones(M, device=DEV), torch.ones(2 * N, device=DEV)
    out = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
    w8.w8a8_gemm_glu_ex(xq, wq, sa, sw, out=out, config=config)
    g = torch.cuda.CUDAGraph(keep_graph=True)
    g.enable_debug_mode()
    with torch.cuda.graph(g):
        w8.w8a8_gemm_glu_ex(xq, wq, sa, sw, out=out, config=config)
    g.debug_dump(str(path))
    text = path.read_text()
    name = re.search(r"_Z\w*gemm_w8a8_kernel\w*", text)
    assert name is not None, text
    return name[0]


@pytest.mark.parametrize("M,N,K", [(1463, 4864, 1936), (248, 9968, 2320), (4363, 600, 2544)])
def test_pairs_where_single_ctas_need_a_whole_round_more(w8, tmp_path, M, N, K):
    kinds = [kernel(w8, tmp_path / f"{i}.dot", M, N, K, c) for i, c in enumerate((None, SINGLE, PAIR))]
    assert kinds[1] != kinds[2]
    assert kinds[0] == kinds[2]
