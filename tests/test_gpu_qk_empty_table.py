"""A table of angles without rows, or without angles, is a table: it does not turn the rotation off."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


def test_tables_without_rows_and_without_angles():
    import w8a8_int8_gemm_b200 as w8
    g = torch.Generator(device=DEV).manual_seed(1)
    q, k = [torch.randn(5, h, 64, generator=g, device=DEV).bfloat16() for h in (4, 2)]
    none = torch.empty(0, 16, device=DEV)
    with pytest.raises(w8.W8A8Error) as e:  # fewer rows than tokens
        w8.w8a8_qk_norm_rope(q, k, cos=none, sin=none)
    assert e.value.status == 1
    with pytest.raises(w8.W8A8Error) as e:  # rot_dim 0
        w8.w8a8_qk_norm_rope(q, k, cos=torch.empty(5, 0, device=DEV), sin=torch.empty(5, 0, device=DEV))
    assert e.value.status == 1
    # every position lies outside: rotated values are NaN, the others the norm's
    pos = torch.zeros(5, dtype=torch.int32, device=DEV)
    got = w8.w8a8_qk_norm_rope(q, k, cos=none, sin=none, positions=pos)
    for x, y in zip(got, w8.w8a8_qk_norm_rope(q, k)):
        assert bool(torch.isnan(x[..., :32]).all()) and torch.equal(x[..., 32:], y[..., 32:])
    # no tokens need no rows
    assert w8.w8a8_qk_norm_rope(q[:0], k[:0], cos=none, sin=none)[0].shape == (0, 4, 64)
    assert w8.w8a8_qk_norm_rope(q[:0], k[:0], cos=none, sin=none, positions=pos[:0])[1].shape == (0, 2, 64)
