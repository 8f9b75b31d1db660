"""Where the Python binding allocates: every tensor that a call makes for itself belongs to the stream the call is given
(memory of another stream could be handed out again, or be written, before the call's kernels have run).  On the host,
with the library, the layout checks and the allocator replaced; the calls whose binding is native are tested on a GPU."""
import pytest
import torch

import __graft_entry__


@pytest.fixture(scope="module")
def w8():
    __graft_entry__.build()
    import w8a8_int8_gemm_b200 as mod
    return mod


class Library:
    """Every function succeeds; the pointers it was given are kept."""

    def __init__(self, real):
        self.real, self.pointers = real, []

    def __getattr__(self, name):
        if name in ("w8a8_linear_sync_words", "w8a8_status_string"):
            return getattr(self.real, name)

        def call(*args):
            self.pointers.extend(a for a in args if isinstance(a, int) and a > 2 ** 20)
            return 0
        return call


BF, I8, U8, F32 = torch.bfloat16, torch.int8, torch.uint8, torch.float32
M, N, K = 4, 8, 32
x, w = torch.zeros(M, K, dtype=BF), torch.zeros(N, K)
xq, wq, xe, we = [torch.zeros(n, K, dtype=t) for t in (I8, U8) for n in (M, N)]
sa, sw, bias = torch.zeros(M), torch.zeros(N), torch.zeros(N, dtype=BF)
wg, wge, sg = torch.zeros(2 * N, K, dtype=I8), torch.zeros(2 * N, K, dtype=U8), torch.zeros(2 * N)
CALLS = {
    "w8a8_quantize_act": (x,), "w8a8_quantize_weight": (w,), "w8a8_gemm": (xq, wq, sa, sw, bias),
    "w8a8_gemm_ex": (xq, wq, sa, sw), "w8a8_gemm_i32": (xq, wq), "w8a8_gemm_i32_ex": (xq, wq),
    "w8a8_linear": (x, wq, sw, bias), "w8a8_linear_fused": (x, wq, sw, bias), "w8a8_linear_noalloc": (x, wq, sw, bias),
    "w8a8_quantize_act_fp8": (x,), "w8a8_quantize_weight_fp8": (w,), "w8a8_gemm_fp8": (xe, we, sa, sw),
    "w8a8_gemm_fp8_ex": (xe, we, sa, sw), "w8a8_gemm_fp8_f32": (xe, we), "w8a8_gemm_fp8_f32_ex": (xe, we),
    "w8a8_linear_fp8": (x, we, sw, bias), "w8a8_quantize_act_gelu": (x,), "w8a8_gelu": (x,),
    "w8a8_linear_gelu": (x, wq, sw, bias), "w8a8_gemm_glu": (xq, wg, sa, sg), "w8a8_gemm_glu_ex": (xq, wg, sa, sg),
    "w8a8_gemm_glu_fp8": (xe, wge, sa, sg), "w8a8_gemm_glu_fp8_ex": (xe, wge, sa, sg),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_a_calls_tensors_belong_to_its_stream(w8, name, monkeypatch):
    lib = Library(w8._lib)
    made = []
    streams = []

    def empty(like, shape, dtype, stream):
        t = torch.zeros(shape, dtype=dtype)
        streams.append(stream)
        made.append(t)
        return t

    monkeypatch.setattr(w8, "_lib", lib)
    monkeypatch.setattr(w8, "_empty", empty)
    monkeypatch.setattr(w8, "_need", lambda *a: None)
    monkeypatch.setattr(w8, "_need_contig", lambda *a: None)
    monkeypatch.setattr(w8, "_stream", lambda stream, device: None)
    monkeypatch.setattr(w8, "_one_device", lambda *a: torch.device("cpu"))
    monkeypatch.setattr(w8, "_call", lambda dev, fn, *a: fn(*a))
    stream = object()
    if name == "w8a8_linear_fused":  # (its counters are zeroed: on the same stream, by a helper of their own)
        monkeypatch.setattr(w8, "_zeros", empty)
    out = getattr(w8, name)(*CALLS[name], stream=stream)
    known = {t.data_ptr() for t in (*CALLS[name], *made)}
    assert made and all(s is stream for s in streams)
    assert all(p in known for p in lib.pointers), "the call made a tensor on another stream"
    for t in out if isinstance(out, tuple) else (out,):
        assert any(t is m for m in made)


def test_every_wrapper_that_allocates_is_covered(w8):
    native = {"w8a8_linear_glu", "w8a8_linear_glu_fp8", "w8a8_qk_norm_rope", "w8a8_attention"}
    none_made = {"w8a8_status_string", "w8a8_abi_version", "w8a8_linear_sync_words", "w8a8_select_config",
                 "w8a8_read_device_error", "w8a8_set_wait_timeout_ns", "w8a8_selftest_wait_timeout", "w8a8_chain_create",
                 "w8a8_chain_launch", "w8a8_chain_layers", "w8a8_chain_destroy"}
    assert set(CALLS) | native | none_made == set(w8.exported_names())
