"""The cap cap * tanh(s / cap) on scores far inside it, around it and far beyond it, in one row: both kernels against
64 bits, with the cap's error relative to the capped score.

Tolerance.  A score s has an error e of its own (the products' sum in binary32 within head_dim * 2^-23 of the sum of
magnitudes; 4 roundings, 2^-22 each of its magnitude), and capping it a relative one of 1e-6 (tanh is computed to
7e-7 of its value; tanh' <= 1 does not enlarge e).  So e_j = dot_j + 2^-20 |s_j| + 1e-6 |cap tanh(s_j / cap)|, a weight
w_j changes by a factor between exp(-e_j) / sum_k w_k exp(e_k) and exp(e_j) / sum_k w_k exp(-e_k), and as in
tests/test_gpu_attention.py weights enter the product in bf16 (2^-8; 2^-16 in two parts), numerator and sum are within
2^-20, the weighted sum adds n * 2^-23, and out rounds once.  Likewise for the logarithm of the sum."""
import math

import pytest
import torch

from tests.test_gpu_attention import tensor

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def w8():
    import w8a8_int8_gemm_b200 as mod
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return mod


def check(out, lse, q, k, v, scale, cap, r):
    f = torch.float64
    (_, Hq, D), (Lk, Hk) = q.shape, k.shape[:2]
    q = q.to(f)
    k, v = [x.to(f).repeat_interleave(Hq // Hk, 1) for x in (k, v)]
    raw = torch.einsum("ihd,jhd->ihj", q, k) * scale
    s = cap * torch.tanh(raw / cap)
    e = torch.einsum("ihd,jhd->ihj", q.abs(), k.abs()) * scale * D * 2.0 ** -23
    e = torch.minimum(e + 2.0 ** -20 * raw.abs(), 2 * s.abs() + e) + 1e-6 * s.abs()
    want_lse = torch.logsumexp(s, -1)
    w = torch.exp(s - want_lse[..., None])
    up, down = (w * torch.exp(e)).sum(-1), (w * torch.exp(-e)).sum(-1)
    factor = torch.exp(e) / down[..., None] - 1
    want = torch.einsum("ihj,jhd->ihd", w, v)
    tol = want.abs() * 2.0 ** -8 + torch.einsum("ihj,jhd->ihd", w * (factor + r + 2.0 ** -20 + Lk * 2.0 ** -23), v.abs())
    off = (out.to(f) - want).abs()
    assert bool((off <= tol).all()), f"out off by {float((off / tol).max())} tolerances"
    tol = torch.maximum(torch.log(up), -torch.log(down)) + 2.0 ** -20 + Lk * 2.0 ** -24 + 2.0 ** -22 * want_lse.abs()
    off = (lse.to(f) - want_lse).abs()
    assert bool((off <= tol).all()), f"lse off by {float((off / tol).max())} tolerances"


def kernels(w8):
    return [(w8.ATTENTION_ROWS, 2.0 ** -16), (w8.ATTENTION_TILES, 2.0 ** -8)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap", [1e-4, 0.05, 2.0, 30.0, 700.0, 1e4, 1e5, 1e6])
@pytest.mark.parametrize("Lq", [2, 150])
def test_relative_to_the_score(w8, Lq, cap, D):
    """Scores of unit size under every cap: those far inside a large one keep their relative accuracy."""
    q, k, v = tensor(Lq, 2, D), tensor(450, 2, D, seed=2), tensor(450, 2, D, seed=3)
    for kernel, r in kernels(w8):
        lse = torch.empty(Lq, 2, device=DEV)
        out = w8.w8a8_attention(q, k, v, cap=cap, lse=lse, kernel=kernel)
        check(out, lse, q, k, v, D ** -0.5, cap, r)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap", [0.05, 2.0, 30.0, 700.0, 1e4, 1e5])
@pytest.mark.parametrize("Lq", [3, 150])
def test_a_score_beyond_the_cap_beside_small_ones(w8, Lq, cap, D):
    """Keys whose scores lie at -5, -1.1, -0.9, -0.3 and -0.2 of the cap, in every stretch of 32 keys, do not take
    accuracy from the others."""
    q, k, v = tensor(Lq, 2, D), tensor(400, 2, D, seed=2), tensor(400, 2, D, seed=3)
    q[..., 0] = 4.0
    k[..., 0] = 0.0
    for n, part in enumerate((-5.0, -1.1, -0.9, -0.3, -0.2)):
        k[5 * n::32] = 0.0
        k[5 * n::32, :, 0] = part * cap / 4.0 * D ** 0.5
    for kernel, r in kernels(w8):
        lse = torch.empty(Lq, 2, device=DEV)
        out = w8.w8a8_attention(q, k, v, cap=cap, lse=lse, kernel=kernel)
        check(out, lse, q, k, v, D ** -0.5, cap, r)


@pytest.mark.parametrize("scale,cap", [(1e-12, 1e6), (1e6, 1e-6), (1e6, 1e6), (1e-12, 1e-6)])
def test_ends_of_the_ranges(w8, scale, cap):
    q, k, v = tensor(140, 2, 64), tensor(200, 2, 64, seed=2), tensor(200, 2, 64, seed=3)
    for kernel, r in kernels(w8):
        lse = torch.empty(140, 2, device=DEV)
        out = w8.w8a8_attention(q, k, v, scale=scale, cap=cap, lse=lse, kernel=kernel)
        if cap * min(1.0, scale / cap) < 1:
            check(out, lse, q, k, v, scale, cap, r)
        assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
