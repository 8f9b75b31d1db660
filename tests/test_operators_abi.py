"""Refusals of the operators beside the linear layers, at the C entry points on the host: every argument is
checked before any device is touched (no GPU needed)."""
import ctypes

import pytest

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
