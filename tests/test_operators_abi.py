"""Refusals of the operators beside the linear layers, at the C entry points on the host: every argument is
checked before any device is touched (no GPU needed)."""
import ctypes

import pytest
import torch

import __graft_entry__

A = 0x10000  # a 16-byte-aligned address that is never dereferenced on these paths


@pytest.fixture(scope="module")
def w8():
    __graft_entry__.build()
    import w8a8_int8_gemm_b200 as mod
    return mod


def qk(w8, **change):
    d = w8.QkDesc(q=A, k=A, q_out=A, k_out=A, q_weight=A, k_weight=None, cos=A, sin=A, positions=None, M=4,
                  table_rows=4, ldq=256, hsq=64, ldk=256, hsk=64, ldq_out=128, hsq_out=64, ldk_out=128, hsk_out=64,
                  heads_q=2, heads_k=2, head_dim=64, rot_dim=64, layout=0, eps=1e-6)
    for name, value in change.items():
        setattr(d, name, value)
    return w8.raw_lib().w8a8_qk_norm_rope(ctypes.byref(d), None)


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), 1), (dict(heads_q=-1), 1), (dict(heads_k=65537), 1), (dict(head_dim=8), 1), (dict(head_dim=264), 1),
    (dict(head_dim=60), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(layout=2), 1), (dict(sin=None), 1), (dict(cos=None), 1), (dict(cos=None, sin=None, positions=A), 1),
    (dict(rot_dim=0), 1), (dict(rot_dim=24), 1), (dict(rot_dim=80), 1), (dict(table_rows=3), 1),
    (dict(table_rows=-1, positions=A), 1), (dict(q=None), 1), (dict(k_out=None), 1), (dict(ldq=-8), 1),
    (dict(hsq_out=32), 1), (dict(ldq_out=64), 1), (dict(ldq_out=0), 1), (dict(ldq=2 ** 31), 1),
    (dict(q=A + 8), 2), (dict(k_out=A + 2), 2), (dict(q_weight=A + 4), 2), (dict(cos=A + 4), 2),
    (dict(positions=A + 2), 2), (dict(ldq=260), 2), (dict(hsk=68), 2),
    (dict(M=0), 0), (dict(heads_q=0, heads_k=0), 0), (dict(M=0, table_rows=0), 0),
])
def test_qk_norm_rope(w8, change, status):
    assert qk(w8, **change) == status


def test_qk_norm_rope_needs_arguments(w8):
    assert w8.raw_lib().w8a8_qk_norm_rope(None, None) == 1


def glu(w8, fn="w8a8_linear_glu", M=4, N=8, K=32, act=2, x=A, wq=A, sw=A, bias=None, out=A, xq=A, sa=A):
    return getattr(w8.raw_lib(), fn)(x, wq, sw, bias, out, xq, sa, M, N, K, act, None)


@pytest.mark.parametrize("fn", ["w8a8_linear_glu", "w8a8_linear_glu_fp8"])
@pytest.mark.parametrize("change,status", [
    (dict(act=0), 1), (dict(act=3), 1), (dict(act=0, M=0), 1), (dict(N=12), 1), (dict(K=24), 1), (dict(M=-1), 1),
    (dict(N=2 ** 30), 1), (dict(x=None), 1), (dict(sw=None), 1), (dict(sa=None), 1), (dict(out=None), 1),
    (dict(wq=A + 8), 2), (dict(bias=A + 2), 2), (dict(xq=A + 4), 2), (dict(M=0), 0), (dict(N=0, act=1), 0),
])
def test_linear_glu(w8, fn, change, status):
    assert glu(w8, fn, **change) == status


@pytest.mark.parametrize("fn", ["w8a8_gemm_glu", "w8a8_gemm_glu_fp8"])
def test_gemm_glu(w8, fn):
    call = getattr(w8.raw_lib(), fn)
    assert call(A, A, A, A, None, A, 4, 8, 32, 0, None) == 1
    assert call(A, A, None, A, None, A, 4, 8, 32, 2, None) == 1
    assert call(A, A, A, None, None, A, 4, 8, 32, 2, None) == 1
    assert call(A, A, A, A, None, A, 4, 2 ** 30, 32, 2, None) == 1
    assert call(A, A, A, A, A + 2, A, 4, 8, 32, 1, None) == 2
    assert call(A, A, A, A, None, A, 0, 8, 32, 1, None) == 0
    cfg = w8.GemmConfig(block_m=256, block_n=256, stages=7, grid=2, raster_group=1)
    assert getattr(w8.raw_lib(), fn + "_ex")(A, A, A, A, None, A, 4, 8, 32, 2, ctypes.byref(cfg), None) == 1


def test_chain_with_gated_layers(w8):
    h = ctypes.c_void_p(None)
    for extra in ((0, 3), (1, 2), (0, -1)):  # (input_act, output_glu): unknown gates, GELU before a gated layer
        d = (w8.LinearDesc * 1)(w8.LinearDesc(A, A, A, None, A, A, A, 4, 8, 32, *extra))
        assert w8.raw_lib().w8a8_chain_create(d, 1, ctypes.byref(h)) == 1 and not h.value
    d = (w8.LinearDesc * 1)(w8.LinearDesc(A, A, A, None, A, A + 4, A, 4, 8, 32, 0, 2))
    assert w8.raw_lib().w8a8_chain_create(d, 1, ctypes.byref(h)) == 2 and not h.value


def attention(w8, **change):
    d = w8.AttentionDesc(q=A, k=A, v=A, out=A, lse=A, cu_q=A, cu_k=A, prefix=None, slopes=None, tokens_q=4,
                         tokens_k=8, ldq=128, hsq=64, ldk=64, hsk=64, ldv=64, hsv=64, ldo=128, hso=64, docs=2,
                         heads_q=2, heads_k=1, head_dim=64, causal=0, scale=0.125, cap=0.0)
    for name, value in change.items():
        setattr(d, name, value)
    return w8.raw_lib().w8a8_attention(ctypes.byref(d), None)


@pytest.mark.parametrize("change,status", [
    (dict(tokens_q=-1), 1), (dict(tokens_k=-1), 1), (dict(tokens_q=2 ** 30 + 1), 1), (dict(docs=0), 1),
    (dict(docs=2 ** 24 + 1), 1), (dict(heads_k=0), 1), (dict(heads_q=1, heads_k=2), 1), (dict(heads_q=3, heads_k=2), 1),
    (dict(heads_q=65537), 1), (dict(head_dim=96), 1), (dict(head_dim=256), 1), (dict(cu_q=None, tokens_q=5), 1),
    (dict(cu_k=None, tokens_k=7), 1), (dict(causal=2), 1), (dict(kernel=3), 1), (dict(kernel=-1), 1), (dict(prefix=A), 1), (dict(scale=0.0), 1),
    (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(cap=-1.0), 1),
    (dict(cap=float("nan")), 1), (dict(cap=2e6), 1), (dict(cap=1e-7), 1), (dict(scale=1e-13), 1), (dict(scale=2e6), 1), (dict(q=None), 1), (dict(v=None), 1), (dict(out=None), 1),
    (dict(ldq=32), 1), (dict(ldk=0), 1), (dict(hsq=0), 1), (dict(ldo=64), 1), (dict(hso=8), 1), (dict(ldv=2 ** 31), 1),
    (dict(ldk=-64), 1), (dict(k=A + 8), 2), (dict(out=A + 2), 2), (dict(ldv=68), 2), (dict(hsq=68, ldq=136), 2),
    (dict(cu_q=A + 2), 2), (dict(lse=A + 1), 2), (dict(slopes=A + 2), 2),
    (dict(tokens_q=0), 0), (dict(tokens_q=0, q=None, out=None), 0),
])
def test_attention(w8, change, status):
    assert attention(w8, **change) == status


def test_attention_needs_arguments(w8):
    assert w8.raw_lib().w8a8_attention(None, None) == 1


def test_binding_refuses_what_are_no_cuda_tensors(w8):
    """The native part of the binding names the argument (no device is touched)."""
    x = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    for f in (w8.w8a8_attention, lambda q, k, v: w8.w8a8_qk_norm_rope(q, k)):
        with pytest.raises(TypeError, match="q must be a torch.Tensor"):
            f(None, x, x)
        with pytest.raises(ValueError, match="q must be a CUDA tensor"):
            f(x, x, x)
    for f in (w8.w8a8_linear_glu, w8.w8a8_linear_glu_fp8):
        with pytest.raises(TypeError, match="x must be a torch.Tensor"):
            f([1.0], x, x)
        with pytest.raises(ValueError, match="x must be a CUDA tensor"):
            f(x[0], x[0], x[0])


def test_native_part_of_the_binding_matches_torch(w8):
    assert w8._calls.torch_version == torch.__version__.split("+")[0]
