"""What a query does not see leaves its bits alone, with a cap and a bias too: keys, values and queries of other
documents, and keys that a mask hides, are made large or NaN, and out and lse compared with a clean run."""
import math

import pytest
import torch

from tests.test_gpu_attention import starts, tensor

pytestmark = pytest.mark.gpu

DEV = "cuda"
KERNELS = [0, 1, 2]  # chosen, for few queries, for many
HOW = {"plain": {}, "cap 2.5": dict(cap=2.5), "cap 30": dict(cap=30.0), "cap 1e4": dict(cap=1e4), "bias": dict(slopes=True),
       "cap and bias": dict(cap=30.0, slopes=True)}


@pytest.fixture(scope="module")
def w8():
    import w8a8_int8_gemm_b200 as mod
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return mod


def attention(w8, q, k, v, how, **more):
    how = dict(HOW[how], **more)
    if how.get("slopes"):
        how["slopes"] = 2.0 ** -torch.arange(1, q.shape[1] + 1, device=DEV, dtype=torch.float32)
    lse = torch.zeros(q.shape[:2], device=DEV)
    return w8.w8a8_attention(q, k, v, lse=lse, **how), lse


@pytest.mark.parametrize("what", [float("nan"), float("inf"), 1e4])
@pytest.mark.parametrize("how", list(HOW))
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("D", [64, 128])
def test_a_neighbour_document(w8, D, kernel, how, what):
    """(Multiplied where it is finite, so that scores of every size appear.)"""
    for lens in ([(1, 130), (1, 70), (1, 200)], [(130, 130), (70, 70), (200, 200)], [(9, 40), (16, 16), (140, 33)]):
        lq, lk = [a for a, _ in lens], [b for _, b in lens]
        q, k, v = tensor(sum(lq), 2, D), tensor(sum(lk), 2, D, seed=2), tensor(sum(lk), 2, D, seed=3)
        cu_q, cu_k = starts(lq), starts(lk)
        args = dict(cu_q=cu_q, cu_k=cu_k, kernel=kernel)
        want, want_lse = attention(w8, q, k, v, how, **args)
        (a, b), (c, d) = cu_q[1:3].tolist(), cu_k[1:3].tolist()
        for t in (q[a:b], k[c:d], v[c:d]):
            t.copy_(t * what if math.isfinite(what) else torch.full_like(t, what))
        got, lse = attention(w8, q, k, v, how, **args)
        for x, y in ((got, want), (lse, want_lse)):
            assert torch.equal(x[:a], y[:a]) and torch.equal(x[b:], y[b:])


@pytest.mark.parametrize("what", [float("nan"), float("-inf"), 1e4, -300.0])
@pytest.mark.parametrize("how", list(HOW))
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("D", [64, 128])
def test_keys_that_a_mask_hides(w8, D, kernel, how, what):
    """Causal: a key in the middle that the queries before it do not see, and its value, large but finite."""
    for L, at in ((150, 100), (150, 3), (300, 290)):
        q, k, v = tensor(L, 2, D), tensor(L, 2, D, seed=2), tensor(L, 2, D, seed=3)
        want, want_lse = attention(w8, q, k, v, how, causal=True, kernel=kernel)
        k[at] = k[at] * what if math.isfinite(what) else what
        v[at] = 1e30
        got, lse = attention(w8, q, k, v, how, causal=True, kernel=kernel)
        assert torch.equal(got[:at], want[:at]) and torch.equal(lse[:at], want_lse[:at])


@pytest.mark.parametrize("how", list(HOW))
@pytest.mark.parametrize("kernel", KERNELS)
def test_other_queries_of_the_document(w8, kernel, how):
    """A query's bits do not depend on the values of the queries beside it."""
    for L in (5, 150):
        q, k, v = tensor(L, 2, 64), tensor(L, 2, 64, seed=2), tensor(L, 2, 64, seed=3)
        want, want_lse = attention(w8, q, k, v, how, causal=True, kernel=kernel)
        q[L // 2] *= 1e3
        q[L // 2 + 1] = float("nan")
        got, lse = attention(w8, q, k, v, how, causal=True, kernel=kernel)
        rest = [i for i in range(L) if i not in (L // 2, L // 2 + 1)]
        assert torch.equal(got[rest], want[rest]) and torch.equal(lse[rest], want_lse[rest])


def test_values_behind_a_slots_keys(w8):
    """The kernel for few queries weighs no key behind the last one that any of its 16 rows sees, not even by 0."""
    L = 150
    q, k, v = tensor(L, 2, 64), tensor(L, 2, 64, seed=2), tensor(L, 2, 64, seed=3)
    want, _ = attention(w8, q, k, v, "plain", causal=True, kernel=w8.ATTENTION_ROWS)
    v[130] = float("nan")
    got, _ = attention(w8, q, k, v, "plain", causal=True, kernel=w8.ATTENTION_ROWS)
    assert torch.equal(got[:128], want[:128]) and bool(torch.isnan(got[130:]).all())
