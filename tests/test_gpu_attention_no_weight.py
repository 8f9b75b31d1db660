"""Rows whose scores are all -inf: no key weighs anything, as where a mask leaves none."""
import math

import pytest
import torch

from tests.test_gpu_attention import tensor

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kernel", [0, 1, 2])
@pytest.mark.parametrize("Lq", [1, 40, 300])
@pytest.mark.parametrize("causal", [False, True])
def test_scores_of_minus_infinity(causal, Lq, kernel, D):
    import w8a8_int8_gemm_b200 as w8
    q, k, v = tensor(Lq, 2, D), tensor(333, 2, D, seed=2), tensor(333, 2, D, seed=3)
    rows = torch.zeros(Lq, dtype=torch.bool, device=DEV)
    rows[::3] = True
    k[..., 0] = 2.0
    base_lse = torch.empty(Lq, 2, device=DEV)
    q[..., 0] = 0.0
    base = w8.w8a8_attention(q, k, v, causal=causal, lse=base_lse, kernel=kernel)
    q[rows, :, 0] = float("-inf")  # every score of the row is -inf
    lse = torch.empty(Lq, 2, device=DEV)
    out = w8.w8a8_attention(q, k, v, causal=causal, lse=lse, kernel=kernel)
    assert bool((out[rows] == 0).all()) and bool((lse[rows] == -math.inf).all())
    assert torch.equal(out[~rows], base[~rows]) and torch.equal(lse[~rows], base_lse[~rows])
    q[rows, :, 0] = -3e38          # the products overflow
    k[..., 0] = 3e38
    q[~rows, :, 0] = 0.0
    out = w8.w8a8_attention(q, k, v, causal=causal, lse=lse, kernel=kernel)
    assert bool((out[rows] == 0).all()) and bool((lse[rows] == -math.inf).all())
    q[0, 0, 0] = float("nan")      # a NaN stays one
    out = w8.w8a8_attention(q, k, v, causal=causal, lse=lse, kernel=kernel)
    assert bool(torch.isnan(out[0, 0]).all()) and bool(torch.isnan(lse[0, 0]))
