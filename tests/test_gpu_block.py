"""A whole transformer block through the library, as a user runs it: QKV linear -> norms and rotation (in place in
the QKV buffer) -> attention over packed documents -> attention-output linear -> gated MLP up -> down, eagerly,
and as one CUDA graph replayed on other inputs.

Every step is compared with its own definition on the inputs that it got (each step's test holds its tolerance);
here the steps' wiring is what is tested: views, documents, workspaces shared between layers, streams."""
import pytest
import torch

from tests import test_gpu_attention as attention_test
from tests import test_gpu_glu as glu_test
from tests import test_gpu_qk_norm_rope as qk_test

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def w8():
    import w8a8_int8_gemm_b200 as mod
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return mod


class Block:
    """One block's weights, buffers and calls.  Hq query heads share Hk key/value heads of D values."""

    def __init__(self, w8, Hq, Hk, D, F, lengths, causal):
        self.w8, self.Hq, self.Hk, self.D, self.F, self.causal = w8, Hq, Hk, D, F, causal
        self.T, H = sum(lengths), Hq * D
        self.H = H
        g = torch.Generator(device=DEV).manual_seed(3)

        def weight(n, k):
            return w8.w8a8_quantize_weight(torch.randn((n, k), generator=g, device=DEV) / k ** 0.5)

        def bias(n):
            return (torch.randn(n, generator=g, device=DEV) * 0.1).bfloat16()

        n_qkv = (Hq + 2 * Hk) * D
        self.qkv_w, self.out_w, self.up_w, self.down_w = weight(n_qkv, H), weight(H, H), weight(2 * F, H), weight(H, F)
        self.qkv_b, self.out_b, self.up_b, self.down_b = bias(n_qkv), bias(H), bias(2 * F), bias(H)
        self.qw, self.kw = [(1 + 0.1 * torch.randn(D, generator=g, device=DEV)).bfloat16() for _ in range(2)]
        self.cos, self.sin = qk_test.table(max(lengths), D)
        self.pos = torch.cat([torch.arange(n, device=DEV) for n in lengths]).to(torch.int32)
        self.cu = attention_test.starts(lengths)
        new = dict(dtype=torch.bfloat16, device=DEV)
        self.qkv = torch.empty((self.T, Hq + 2 * Hk, D), **new)
        self.a, self.o = torch.empty((self.T, Hq, D), **new), torch.empty((self.T, H), **new)
        self.h, self.y = torch.empty((self.T, F), **new), torch.empty((self.T, H), **new)
        self.lse = torch.empty((self.T, Hq), device=DEV)
        self.ws = torch.empty((self.T, max(H, F)), dtype=torch.int8, device=DEV)  # one workspace for every linear
        self.sa = torch.empty(self.T, device=DEV)

    def run(self, x, stream=None):
        w8, Hq, Hk = self.w8, self.Hq, self.Hk
        flat = self.ws.view(-1)
        ws_h, ws_f = flat[:self.T * self.H].view(self.T, self.H), flat[:self.T * self.F].view(self.T, self.F)
        how = dict(ws_scale_a=self.sa, stream=stream)
        w8.w8a8_linear(x, *self.qkv_w, self.qkv_b, out=self.qkv.view(self.T, -1), ws_xq=ws_h, **how)
        q, k, v = self.qkv[:, :Hq], self.qkv[:, Hq:Hq + Hk], self.qkv[:, Hq + Hk:]
        w8.w8a8_qk_norm_rope(q, k, self.qw, self.kw, self.cos, self.sin, positions=self.pos, q_out=q, k_out=k,
                             stream=stream)
        w8.w8a8_attention(q, k, v, causal=self.causal, cu_q=self.cu, cu_k=self.cu, out=self.a, lse=self.lse,
                          stream=stream)
        w8.w8a8_linear(self.a.view(self.T, -1), *self.out_w, self.out_b, out=self.o, ws_xq=ws_h, **how)
        w8.w8a8_linear_glu(self.o, *self.up_w, self.up_b, out=self.h, ws_xq=ws_h, **how)
        w8.w8a8_linear(self.h, *self.down_w, self.down_b, out=self.y, ws_xq=ws_f, **how)
        return self.y

    def check(self, x):
        w8, Hq, Hk, D = self.w8, self.Hq, self.Hk, self.D
        raw = w8.w8a8_linear(x, *self.qkv_w, self.qkv_b).view(self.T, Hq + 2 * Hk, D)
        q, k, v = self.qkv[:, :Hq], self.qkv[:, Hq:Hq + Hk], self.qkv[:, Hq + Hk:]
        qk_test.check(q, raw[:, :Hq], self.qw, self.cos, self.sin, self.pos.long(), 1e-6, False)
        qk_test.check(k, raw[:, Hq:Hq + Hk], self.kw, self.cos, self.sin, self.pos.long(), 1e-6, False)
        assert torch.equal(v, raw[:, Hq + Hk:])
        attention_test.check(self.a, self.lse, q, k, v, self.cu, self.cu, D ** -0.5, causal=self.causal)
        assert torch.equal(self.o, w8.w8a8_linear(self.a.view(self.T, -1), *self.out_w, self.out_b))
        xq, sa = w8.w8a8_quantize_act(self.o)
        glu_test.check(w8, self.h, xq, self.up_w[0], sa, self.up_w[1], self.up_b, w8.ACT_SILU)
        assert torch.equal(self.y, w8.w8a8_linear(self.h, *self.down_w, self.down_b))
        assert w8.w8a8_read_device_error() == 0


def activations(T, H, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn((T, H), generator=g, device=DEV).bfloat16()


@pytest.mark.parametrize("Hq,Hk,D,F,lengths,causal", [(4, 4, 128, 1024, [300, 77, 513], False),
                                                      (8, 2, 64, 768, [129, 1, 640], True),
                                                      (2, 1, 64, 256, [3, 5], True)])
def test_block(w8, Hq, Hk, D, F, lengths, causal):
    b = Block(w8, Hq, Hk, D, F, lengths, causal)
    x = activations(b.T, b.H, 1)
    b.run(x)
    torch.cuda.synchronize()
    b.check(x)
    # the block as one graph, on a stream of its own, replayed on other activations
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        b.run(x, stream=s)
    for seed in (2, 3):
        x.copy_(activations(b.T, b.H, seed))
        g.replay()
        torch.cuda.synchronize()
        got = b.y.clone()
        b.check(x)
        b.run(x)
        torch.cuda.synchronize()
        assert torch.equal(b.y, got)


def test_two_threads_with_streams_of_their_own(w8):
    """Calls from two threads at once, each on a stream by handle or object and with outputs and workspaces of the
    call's own, give the bits of calls one after the other."""
    import threading
    q, k = attention_test.tensor(300, 4, 64, seed=1), attention_test.tensor(300, 2, 64, seed=2)
    x = attention_test.tensor(70, 256, seed=3)
    wq, sw = w8.w8a8_quantize_weight(torch.randn((2 * 128, 256), device=DEV))

    def calls(stream):
        return [w8.w8a8_attention(q, k, k, causal=True, stream=stream), *w8.w8a8_qk_norm_rope(q, k, stream=stream),
                w8.w8a8_linear_glu(x, wq, sw, stream=stream)]

    want = calls(None)
    torch.cuda.synchronize()
    got, streams = {}, [torch.cuda.Stream(), torch.cuda.Stream()]

    def work(i):
        stream = streams[i] if i else streams[i].cuda_stream
        got[i] = [calls(stream) for _ in range(50)]

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert w8.w8a8_read_device_error() == 0
    for i in range(2):
        for outs in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(outs, want))
