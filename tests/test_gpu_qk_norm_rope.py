"""Norms of queries and keys with the position rotation (w8a8_qk_norm_rope) on the GPU against the formula in
64 bits.

Tolerance.  The kernel computes in binary32 and rounds once to bf16 (half a step: 2^-8 of the value).  In
binary32 the sum of D <= 256 squares is 8 serial additions and 5 of the tree (relative error below 14 * 2^-24,
halved by the square root), rsqrt adds 2^-22, the two products by it and by the weight 2 * 2^-24, and the
rotation's products and sum 3 * 2^-24 of the terms: below 2^-20 of |n_a cos| + |n_b sin| in all."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def w8():
    import w8a8_int8_gemm_b200 as mod
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return mod


def reference(x, weight, cos, sin, row, eps, pairs):
    """The formula in float64 -> (value, sum of the magnitudes that were added)."""
    f = torch.float64
    x = x.to(f)
    n = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    if weight is not None:
        n = n * weight.to(f)
    y, mag = n.clone(), n.abs()
    if cos is not None:
        h = cos.shape[1]
        t = torch.arange(h, device=x.device)
        a, b = (2 * t, 2 * t + 1) if pairs else (t, t + h)
        c, s = cos.to(f)[row][:, None], sin.to(f)[row][:, None]
        y[..., a] = n[..., a] * c - n[..., b] * s
        y[..., b] = n[..., b] * c + n[..., a] * s
        mag[..., a] = (n[..., a] * c).abs() + (n[..., b] * s).abs()
        mag[..., b] = (n[..., b] * c).abs() + (n[..., a] * s).abs()
    return y, mag


def check(got, x, weight, cos, sin, row, eps, pairs):
    want, mag = reference(x, weight, cos, sin, row, eps, pairs)
    off = (got.double() - want).abs()
    tol = want.abs() * 2.0 ** -8 + mag * 2.0 ** -20 + 1e-38
    assert bool((off <= tol).all()), f"off by {float((off - tol).max())} beyond the tolerance"


def table(rows, rot, seed=0):
    g = torch.Generator().manual_seed(seed)
    ang = torch.rand((rows, rot // 2), generator=g, dtype=torch.float64) * 6.28318
    return ang.cos().float().to(DEV), ang.sin().float().to(DEV)


def tensor(*shape, seed=1, std=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).bfloat16().to(DEV)


# every lane count per head, ragged head counts, one and many tokens, full and partial rotation
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("M,hq,hk,D,R", [(1, 1, 1, 128, 128), (1, 32, 8, 128, 128), (7, 24, 24, 128, 128),
                                         (333, 5, 3, 64, 64), (65, 9, 1, 64, 16), (40, 3, 3, 96, 96),
                                         (31, 2, 2, 80, 32), (17, 7, 2, 256, 256), (19, 4, 4, 200, 112),
                                         (23, 3, 1, 16, 16), (29, 11, 5, 24, 16), (50, 13, 13, 32, 32),
                                         (21, 1, 2, 40, 32), (2305, 4, 4, 128, 64)])
def test_against_the_formula(w8, M, hq, hk, D, R, pairs):
    q, k = tensor(M, hq, D), tensor(M, hk, D, seed=2)
    qw, kw = tensor(D, seed=3), tensor(D, seed=4)
    cos, sin = table(M + 3, R)
    layout = w8.ROPE_PAIRS if pairs else w8.ROPE_HALVES
    qo, ko = w8.w8a8_qk_norm_rope(q, k, qw, kw, cos, sin, layout=layout)
    row = torch.arange(M, device=DEV)
    check(qo, q, qw, cos, sin, row, 1e-6, pairs)
    check(ko, k, kw, cos, sin, row, 1e-6, pairs)
    # gathered positions, repeated ones among them, no weights
    pos = torch.randint(0, M + 3, (M,), dtype=torch.int32, device=DEV)
    qo, ko = w8.w8a8_qk_norm_rope(q, k, None, None, cos, sin, positions=pos, eps=0.5, layout=layout)
    check(qo, q, None, cos, sin, pos.long(), 0.5, pairs)
    check(ko, k, None, cos, sin, pos.long(), 0.5, pairs)


def test_norm_alone(w8):
    q, k, qw = tensor(37, 6, 128), tensor(37, 2, 128, seed=5), tensor(128, seed=6)
    qo, ko = w8.w8a8_qk_norm_rope(q, k, qw, None)
    check(qo, q, qw, None, None, None, 1e-6, False)
    check(ko, k, None, None, None, None, 1e-6, False)


@pytest.mark.parametrize("pairs", [False, True])
def test_views_of_one_buffer_in_place_and_head_major(w8, pairs):
    M, hq, hk, D = 77, 6, 2, 64
    layout = w8.ROPE_PAIRS if pairs else w8.ROPE_HALVES
    buf = tensor(M, hq + 2 * hk + 1, D)
    cos, sin = table(M, D)
    q, k, rest = buf[:, :hq], buf[:, hq:hq + hk], buf[:, hq + hk:]
    q0, k0, rest0 = q.clone(), k.clone(), rest.clone()
    want_q, want_k = w8.w8a8_qk_norm_rope(q0, k0, None, None, cos, sin, layout=layout)
    # head-major outputs, in a buffer with guard rows around them
    hm = torch.full((hq + 2, M, D), 7.0, dtype=torch.bfloat16, device=DEV)
    qo, _ = w8.w8a8_qk_norm_rope(q, k, None, None, cos, sin, layout=layout, q_out=hm[1:-1].transpose(0, 1))
    assert torch.equal(qo.contiguous(), want_q)
    assert bool((hm[0] == 7).all()) and bool((hm[-1] == 7).all())
    # head-major inputs
    qi, _ = w8.w8a8_qk_norm_rope(hm[1:-1].transpose(0, 1), k, None, None)
    check(qi, want_q, None, None, None, None, 1e-6, pairs)
    # in place in the QKV buffer: the values are left as they were
    w8.w8a8_qk_norm_rope(q, k, None, None, cos, sin, layout=layout, q_out=q, k_out=k)
    assert torch.equal(q, want_q) and torch.equal(k, want_k) and torch.equal(rest, rest0)


def test_rows_that_can_go_wrong(w8):
    q, k = tensor(6, 4, 128), tensor(6, 4, 128, seed=8)
    cos, sin = table(6, 128)
    q[0] = 0.0                                    # zero row: 0 * rsqrt(eps)
    q[1] = 3e19                                   # squares overflow binary32: rsqrt(inf) = 0
    q[2, 0, 5] = float("inf")
    q[3, 1, 7] = float("nan")
    q[4] = 1e-30                                  # squares vanish beside eps
    qo, ko = w8.w8a8_qk_norm_rope(q, k, None, None, cos, sin)
    assert bool((qo[0] == 0).all()) and bool((qo[1] == 0).all())
    assert bool(torch.isnan(qo[2, 0, 5])) and bool(torch.isnan(qo[3, 1]).all())
    clean = torch.ones((6, 4), dtype=torch.bool, device=DEV)
    clean[1] = clean[2, 0] = clean[3, 1] = False  # the other heads of those tokens are untouched by it
    row = torch.arange(6, device=DEV)
    for m in range(6):
        h = clean[m].nonzero()[:, 0]
        if len(h):
            check(qo[m:m + 1, h], q[m:m + 1, h], None, cos, sin, row[m:m + 1], 1e-6, False)
    check(ko, k, None, cos, sin, row, 1e-6, False)


@pytest.mark.parametrize("pairs", [False, True])
def test_positions_outside_the_table(w8, pairs):
    """They read nothing; the rotated values are NaN, the others and the other tokens as always."""
    q, k = tensor(5, 2, 64), tensor(5, 1, 64, seed=9)
    cos, sin = table(8, 32)
    pos = torch.tensor([3, -1, 8, 7, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    qo, ko = w8.w8a8_qk_norm_rope(q, k, None, None, cos, sin, positions=pos,
                                  layout=w8.ROPE_PAIRS if pairs else w8.ROPE_HALVES)
    good, bad = torch.tensor([0, 3], device=DEV), torch.tensor([1, 2, 4], device=DEV)
    for o, x in ((qo, q), (ko, k)):
        check(o[good], x[good], None, cos, sin, pos[good].long(), 1e-6, pairs)
        assert bool(torch.isnan(o[bad][..., :32]).all())
        n, mag = reference(x[bad], None, None, None, None, 1e-6, pairs)
        assert bool(((o[bad].double() - n).abs() <= n.abs() * 2.0 ** -8 + mag * 2.0 ** -20)[..., 32:].all())


def test_empty(w8):
    e = torch.empty((0, 4, 64), dtype=torch.bfloat16, device=DEV)
    qo, ko = w8.w8a8_qk_norm_rope(e, e)
    assert qo.shape == (0, 4, 64)
    q, none = tensor(3, 2, 64), torch.empty((3, 0, 64), dtype=torch.bfloat16, device=DEV)
    qo, ko = w8.w8a8_qk_norm_rope(q, none)
    check(qo, q, None, None, None, None, 1e-6, False)
    assert ko.shape == (3, 0, 64)


def test_offsets_beyond_32_bits(w8):
    """A token stride that puts the last token's offset past 2^32 bytes and 2^31 elements."""
    ld = 2 ** 30 + 64
    buf = torch.empty(2 * ld + 2 * 64, dtype=torch.bfloat16, device=DEV)
    x = buf.as_strided((3, 2, 64), (ld, 64, 1))
    x.copy_(tensor(3, 2, 64, seed=11))
    cos, sin = table(3, 64)
    qo, ko = w8.w8a8_qk_norm_rope(x, x, None, None, cos, sin)
    check(qo, x, None, cos, sin, torch.arange(3, device=DEV), 1e-6, False)
    assert torch.equal(qo, ko)
    want = qo.clone()
    w8.w8a8_qk_norm_rope(x, tensor(3, 1, 64), None, None, cos, sin, q_out=x)
    assert torch.equal(x, want)


def test_other_stream_and_captured(w8):
    q, k = tensor(130, 8, 128), tensor(130, 2, 128, seed=12)
    cos, sin = table(130, 128)
    want = w8.w8a8_qk_norm_rope(q, k, None, None, cos, sin)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = w8.w8a8_qk_norm_rope(q, k, None, None, cos, sin, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w8.w8a8_qk_norm_rope(q, k, None, None, cos, sin, q_out=qo, k_out=ko)
    for _ in range(2):
        q.copy_(tensor(130, 8, 128, seed=13))
        g.replay()
        torch.cuda.synchronize()
        check(qo, q, None, cos, sin, torch.arange(130, device=DEV), 1e-6, False)
        assert torch.equal(ko, want[1])


def test_refusals(w8):
    q, k = tensor(4, 2, 64), tensor(4, 2, 64)
    cos, sin = table(4, 64)
    with pytest.raises(ValueError):
        w8.w8a8_qk_norm_rope(q, k[:3])
    with pytest.raises(ValueError):
        w8.w8a8_qk_norm_rope(q, k, cos=cos)
    with pytest.raises(TypeError):
        w8.w8a8_qk_norm_rope(q.float(), k)
    with pytest.raises(TypeError):
        w8.w8a8_qk_norm_rope(q, k, None, None, cos, sin, positions=torch.zeros(4, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        w8.w8a8_qk_norm_rope(q, k, torch.ones(32, dtype=torch.bfloat16, device=DEV))
    for bad in (dict(cos=cos[:3], sin=sin[:3]), dict(cos=cos[:, :12].contiguous(), sin=sin[:, :12].contiguous()),
                dict(eps=-1.0), dict(eps=float("nan")), dict(layout=2)):
        with pytest.raises(w8.W8A8Error) as e:
            w8.w8a8_qk_norm_rope(q, k, **bad)
        assert e.value.status == 1
    wide = tensor(4, 2, 68)
    with pytest.raises(w8.W8A8Error) as e:
        w8.w8a8_qk_norm_rope(wide[..., :64], k)    # head stride 68
    assert e.value.status == 2
    with pytest.raises(w8.W8A8Error) as e:           # outputs that overlap one another
        w8.w8a8_qk_norm_rope(q, k, q_out=torch.zeros_like(q[:, :1]).expand(4, 2, 64))
    assert e.value.status == 1
