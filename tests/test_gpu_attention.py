"""w8a8_attention on the GPU against the definition in 64 bits.

Tolerance, per query: with e_s the error of a score (the products' sum in binary32 within head_dim * 2^-23 of the
sum of magnitudes, the library's bound for its tensor-core sums; 4 roundings of the score and of its exponent's
argument in units of log2, 2^-22 of the largest magnitude a score or bias takes; 1e-6 * cap), a weight is off by
a factor within 2 e_s + 2^-20 (numerator and sum), and it enters the product with v rounded to bf16 (half a step:
2^-8; 2^-16 where it enters in two parts).  The weighted sum of n terms in binary32 adds n * 2^-23, and out
rounds once:  |out - exact| <= 2^-8 |exact| + (r + 2 e_s + 2^-20 + n 2^-23) sum_j w_j |v_j|.  The logarithm of the
sum:  |lse - exact| <= e_s + 2^-20 + n 2^-24 + 2^-22 |lse|."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def w8():
    import w8a8_int8_gemm_b200 as mod
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return mod


def tensor(*shape, seed=1, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * std).bfloat16()


def starts(lengths, first=0):
    return torch.tensor([first] + list(lengths), device=DEV).cumsum(0).to(torch.int32)


def reference(q, k, v, scale, cap=0.0, causal=False, prefix=0, slopes=None):
    """One document in float64: out, lse, sum of |w v|, error of a score per query, keys per query."""
    f = torch.float64
    q, k, v = q.to(f), k.to(f), v.to(f)
    (Lq, Hq, D), (Lk, Hk) = q.shape, k.shape[:2]
    k, v = [x.repeat_interleave(Hq // Hk, 1) for x in (k, v)]
    s = torch.einsum("ihd,jhd->ihj", q, k) * scale
    e = torch.einsum("ihd,jhd->ihj", q.abs(), k.abs()).amax(-1) * scale * D * 2.0 ** -23 if Lk else torch.zeros(Lq, Hq, device=DEV)
    big = s.abs()
    if cap:
        s = cap * torch.tanh(s / cap)
    i = torch.arange(Lq, device=DEV)[:, None] + Lk - Lq
    j = torch.arange(Lk, device=DEV)[None]
    if slopes is not None:
        b = slopes.to(f)[None, :, None] * (i - j).abs()[:, None]
        s, big = s - b, big + b
    seen = torch.ones(Lq, Lk, dtype=torch.bool, device=DEV)
    if causal:
        seen = (j <= i) | (j < prefix)
    s = s.masked_fill(~seen[:, None], -math.inf)
    lse = torch.logsumexp(s, -1) if Lk else torch.full((Lq, Hq), -math.inf, dtype=f, device=DEV)
    w = torch.exp(s - lse[..., None]).masked_fill(~seen[:, None], 0.0)
    if Lk:
        e = e + 2.0 ** -22 * big.masked_fill(~seen[:, None], 0.0).amax(-1) * 4
    return (torch.einsum("ihj,jhd->ihd", w, v), lse, torch.einsum("ihj,jhd->ihd", w, v.abs()), e + 1e-6 * cap,
            seen.sum(-1))


def check(out, lse, q, k, v, cu_q, cu_k, scale, cap=0.0, causal=False, prefix=None, slopes=None, r=2.0 ** -8):
    for d in range(len(cu_q) - 1):
        a, b, c, e = int(cu_q[d]), int(cu_q[d + 1]), int(cu_k[d]), int(cu_k[d + 1])
        if a == b:
            continue
        want, want_lse, mag, es, n = reference(q[a:b], k[c:e], v[c:e], scale, cap, causal,
                                               0 if prefix is None else int(prefix[d]), slopes)
        n = n[:, None].double()
        none = (n == 0).expand_as(want_lse)
        got, got_lse = out[a:b].double(), lse[a:b].double()
        assert bool((got[none] == 0).all()) and bool((got_lse[none] == -math.inf).all()), "queries that see no key"
        tol = want.abs() * 2.0 ** -8 + (r + 2 * es + 2.0 ** -20 + n * 2.0 ** -23)[..., None] * mag + 1e-37
        off = (got - want).abs()
        assert bool((off <= tol)[~none].all()), f"document {d}: out off by {float((off / tol)[~none].max())} tolerances"
        tol = es + 2.0 ** -20 + n * 2.0 ** -24 + 2.0 ** -22 * want_lse.abs()
        off = (got_lse - want_lse).abs()
        assert bool((off <= tol)[~none].all()), f"document {d}: lse off by {float((off / tol)[~none].max())} tolerances"


KERNELS = [0, 1, 2]  # chosen, for few queries, for many


def case(w8, docs, Hq, Hk, D, seed=0, r=2.0 ** -8, std=1.0, kernel=0, **how):
    lq, lk = [x for x, _ in docs], [y for _, y in docs]
    q = tensor(sum(lq), Hq, D, seed=seed + 1, std=std)
    k = tensor(sum(lk), Hk, D, seed=seed + 2, std=std)
    v = tensor(sum(lk), Hk, D, seed=seed + 3)
    cu_q, cu_k = starts(lq), starts(lk)
    lse = torch.full((sum(lq), Hq), 9.0, device=DEV)
    out = w8.w8a8_attention(q, k, v, cu_q=cu_q, cu_k=cu_k, lse=lse, kernel=kernel, **how)
    torch.cuda.synchronize()
    assert w8.w8a8_read_device_error() == 0
    check(out, lse, q, k, v, cu_q, cu_k, how.pop("scale", D ** -0.5), r=r, **how)
    return out


DOCS = {
    "one token, one key": [(1, 1)],
    "one token, long caches": [(1, 4097), (1, 3), (1, 129), (1, 128), (1, 16)],
    "empty documents": [(0, 5), (3, 0), (0, 0), (5, 5), (2, 0)],
    "small": [(2, 2), (3, 3), (17, 17), (33, 33)],
    "tile edges": [(127, 127), (128, 128), (129, 129), (255, 255), (256, 256), (257, 257)],
    "more queries than keys": [(200, 50), (300, 1), (40, 39)],
    "extending a cache": [(5, 1000), (40, 640), (130, 777), (300, 1111)],
    "long": [(1111, 1111), (64, 64), (769, 769)],
}


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("how", ["plain", "causal", "prefix", "cap", "bias", "all"])
@pytest.mark.parametrize("docs", list(DOCS))
@pytest.mark.parametrize("kernel", KERNELS)
def test_masks_and_lengths(w8, kernel, docs, how, D):
    shapes = DOCS[docs]
    Hq, Hk = {"plain": (3, 3), "causal": (6, 2), "prefix": (4, 1), "cap": (2, 2), "bias": (8, 4), "all": (5, 1)}[how]
    args = {}
    if how in ("causal", "prefix", "all"):
        args["causal"] = True
    if how in ("prefix", "all"):
        args["prefix"] = torch.tensor([(37 * i) % 300 for i in range(len(shapes))], dtype=torch.int32, device=DEV)
    if how in ("cap", "all"):
        args["cap"] = 2.5 if how == "cap" else 30.0
    if how in ("bias", "all"):
        args["slopes"] = 2.0 ** -torch.arange(1, Hq + 1, device=DEV, dtype=torch.float32)
    case(w8, shapes, Hq, Hk, D, seed=len(docs), kernel=kernel, **args)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 3, 8, 16, 40])
def test_shared_heads_single_tokens(w8, G, D):
    """One to four tokens per sequence over ragged caches, in the row kernel: weights in two parts (r = 2^-16)."""
    how = dict(r=2.0 ** -16, causal=True, kernel=w8.ATTENTION_ROWS)
    case(w8, [(1, 700), (1, 5000), (1, 1), (1, 15), (1, 17), (1, 0), (1, 2049)], 2 * G, 2, D, **how)
    case(w8, [(4, 700), (3, 33), (2, 2), (4, 1025)], 2 * G, 2, D, **how)
    case(w8, [(1, 1000 * i + 1) for i in range(40)], 2 * G, 2, D, causal=True)  # the chosen kernel


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("scale,std", [(1.0, 2.0), (0.01, 1.0), (30.0, 1.0)])
def test_sharp_and_flat_weights(w8, scale, std, kernel):
    case(w8, [(300, 300), (1, 300)], 2, 2, 64, scale=scale, std=std, kernel=kernel)
    case(w8, [(140, 400), (3, 300)], 2, 1, 128, scale=scale, std=std, causal=True, kernel=kernel)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap", [1e-3, 0.3, 4.0, 50.0, 700.0, 1e5])
@pytest.mark.parametrize("kernel", KERNELS)
def test_cap_over_its_range(w8, kernel, cap, D):
    """Scores far inside the cap, around it and far beyond it, in the same tile and in tiles of their own."""
    for Lq in (2, 150):
        q, k, v = tensor(Lq, 2, D), tensor(450, 2, D, seed=2), tensor(450, 2, D, seed=3)
        q[: Lq // 2] *= 0.02
        k[:130] *= 0.05
        k[300:] *= 4.0
        lse = torch.empty(Lq, 2, device=DEV)
        out = w8.w8a8_attention(q, k, v, cap=cap, lse=lse, kernel=kernel)
        check(out, lse, q, k, v, [0, Lq], [0, 450], D ** -0.5, cap=cap)


@pytest.mark.parametrize("kernel", KERNELS)
def test_scores_that_climb(w8, kernel):
    """The running maximum grows with every tile of keys, by more and less than a power of 2^8 at a time."""
    for step in (0.02, 0.5):
        for Lq in (1, 200):
            D, L = 64, 900
            q = torch.zeros(Lq, 1, D, device=DEV).bfloat16()
            k = torch.zeros(L, 1, D, device=DEV).bfloat16()
            q[..., 0] = 8.0
            k[:, 0, 0] = torch.arange(L, device=DEV) * step
            v = tensor(L, 1, D, seed=5)
            lse = torch.empty(Lq, 1, device=DEV)
            for kk in (k, k.flip(0)):
                out = w8.w8a8_attention(q, kk, v, scale=1.0, lse=lse, kernel=kernel)
                check(out, lse, q, kk, v, [0, Lq], [0, L], 1.0)


@pytest.mark.parametrize("kernel", KERNELS)
def test_views_gaps_and_garbage(w8, kernel):
    """Strided views of one buffer; NaN and infinities in every token outside the documents; rows of out and lse
    outside them stay as they were."""
    for lens in ([(1, 130), (1, 257), (1, 3)], [(150, 150), (70, 70), (300, 300)]):
        Hq, Hk, D = 6, 2, 128
        lq, lk = [a for a, _ in lens], [b for _, b in lens]
        fq, fk = 5, 9
        Tq, Tk = fq + sum(lq) + 7, fk + sum(lk) + 11
        cu_q, cu_k = starts(lq, fq), starts(lk, fk)
        kv = tensor(Tk, 2, Hk + 1, D, seed=3)
        k, v = kv[:, 0, :Hk], kv[:, 1, 1:]
        for t in (slice(0, fk), slice(int(cu_k[-1]), Tk)):
            k[t], v[t] = float("nan"), float("inf")
        q = tensor(Hq, Tq, D, seed=4).transpose(0, 1)  # head-major
        q[:fq], q[int(cu_q[-1]):] = float("nan"), float("inf")
        buf = torch.full((Tq, Hq + 2, D), 3.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((Tq, Hq), 5.0, device=DEV)
        w8.w8a8_attention(q, k, v, causal=True, cu_q=cu_q, cu_k=cu_k, out=buf[:, 1:-1], lse=lse, kernel=kernel)
        check(buf[:, 1:-1], lse, q, k, v, cu_q, cu_k, D ** -0.5, causal=True)
        assert bool((buf[:, 0] == 3).all()) and bool((buf[:, -1] == 3).all())
        for t in (slice(0, fq), slice(int(cu_q[-1]), Tq)):
            assert bool((buf[t] == 3).all()) and bool((lse[t] == 5).all())


@pytest.mark.parametrize("kernel", KERNELS)
def test_a_neighbour_full_of_nan(w8, kernel):
    """NaN in one document's keys and values stays in that document."""
    for lens in ([(1, 130), (1, 70), (1, 200)], [(130, 130), (70, 70), (200, 200)]):
        lq, lk = [a for a, _ in lens], [b for _, b in lens]
        q, k, v = tensor(sum(lq), 2, 64), tensor(sum(lk), 2, 64, seed=2), tensor(sum(lk), 2, 64, seed=3)
        cu_q, cu_k = starts(lq), starts(lk)
        clean = w8.w8a8_attention(q, k, v, cu_q=cu_q, cu_k=cu_k, kernel=kernel)
        k[int(cu_k[1]):int(cu_k[2])] = float("nan")
        v[int(cu_k[1]):int(cu_k[2])] = float("nan")
        out = w8.w8a8_attention(q, k, v, cu_q=cu_q, cu_k=cu_k, kernel=kernel)
        a, b = int(cu_q[1]), int(cu_q[2])
        assert torch.equal(out[:a], clean[:a]) and torch.equal(out[b:], clean[b:])
        assert bool(torch.isnan(out[a:b]).all())


@pytest.mark.parametrize("kernel", KERNELS)
def test_hidden_keys_may_hold_anything(w8, kernel):
    """Keys past every query's limit: NaN scores and values that nothing sees."""
    for Lq, Lk in ((1, 300), (150, 150)):
        q, k, v = tensor(Lq, 2, 128), tensor(Lk, 2, 128, seed=2), tensor(Lk, 2, 128, seed=3)
        k[100] = float("nan")  # a NaN key that is seen makes its queries NaN
        out = w8.w8a8_attention(q, k, v, causal=True, kernel=kernel)
        sees = torch.arange(Lq, device=DEV) + Lk - Lq >= 100
        assert bool(torch.isnan(out[sees]).all()) and bool(torch.isfinite(out[~sees]).all())


@pytest.mark.parametrize("kernel", KERNELS)
def test_head_major_everything(w8, kernel):
    """[heads, tokens, D] tensors: a token stride below the head stride, for every operand."""
    q, k, v = [tensor(h, n, 64, seed=i).transpose(0, 1) for i, (h, n) in enumerate([(4, 333), (2, 401), (2, 401)])]
    out = torch.full((6, 333, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(333, 4, device=DEV)
    w8.w8a8_attention(q, k, v, causal=True, out=out[1:-1].transpose(0, 1), lse=lse, kernel=kernel)
    check(out[1:-1].transpose(0, 1), lse, q, k, v, [0, 333], [0, 401], 64 ** -0.5, causal=True)
    assert bool((out[0] == 3).all()) and bool((out[-1] == 3).all())


@pytest.mark.parametrize("kernel", KERNELS)
def test_queries_in_equal_parts_keys_ragged(w8, kernel):
    """One of the two streams with starts, the other in equal parts; key and value streams of their own strides."""
    lk = [5, 200, 0, 131]
    q, k = tensor(4 * 9, 2, 128), tensor(sum(lk), 2, 128, seed=2)
    v = tensor(sum(lk), 3, 128, seed=3)[:, :2]
    lse = torch.empty(36, 2, device=DEV)
    out = w8.w8a8_attention(q, k, v, cu_k=starts(lk), lse=lse, kernel=kernel)
    check(out, lse, q, k, v, starts([9] * 4), starts(lk), 128 ** -0.5)


@pytest.mark.parametrize("kernel", KERNELS)
def test_biases_that_grow_and_vanish(w8, kernel):
    """Negative, zero and steep slopes, keys on both sides of a query."""
    slopes = torch.tensor([-0.01, 0.0, 3.0, 0.25], device=DEV)
    case(w8, [(150, 150), (7, 260), (1, 33)], 4, 2, 64, slopes=slopes, kernel=kernel)
    prefix = torch.tensor([100, 7, 0], dtype=torch.int32, device=DEV)
    case(w8, [(150, 150), (7, 260), (1, 33)], 4, 2, 128, slopes=slopes, causal=True, prefix=prefix, kernel=kernel)


def test_equal_parts_without_starts(w8):
    q, k, v = tensor(6 * 50, 4, 64), tensor(6 * 70, 2, 64, seed=2), tensor(6 * 70, 2, 64, seed=3)
    got = w8.w8a8_attention(q, k, v, docs=6, causal=True)
    want = w8.w8a8_attention(q, k, v, cu_q=starts([50] * 6), cu_k=starts([70] * 6), causal=True)
    assert torch.equal(got, want)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("most", [3, 40])
def test_thousands_of_documents(w8, most, kernel):
    n = 2500
    lens = [1 + (7 * i) % most for i in range(n)]
    q, k, v = tensor(sum(lens), 2, 64), tensor(sum(lens), 1, 64, seed=2), tensor(sum(lens), 1, 64, seed=3)
    cu = starts(lens)
    lse = torch.empty(sum(lens), 2, device=DEV)
    out = w8.w8a8_attention(q, k, v, cu_q=cu, cu_k=cu, causal=True, lse=lse, kernel=kernel)
    at = list(range(0, n, 97)) + [n - 2, n - 1]
    for d in at:
        a, b = int(cu[d]), int(cu[d + 1])
        check(out[a:b], lse[a:b], q[a:b], k[a:b], v[a:b], [0, b - a], [0, b - a], 64 ** -0.5, causal=True)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("Lq", [1, 140])
def test_offsets_beyond_32_bits(w8, Lq, kernel):
    """A cache whose token stride puts keys past 2^32 elements."""
    L, ld = 300, 2 ** 24 + 64
    buf = torch.empty((L - 1) * ld + 192, dtype=torch.bfloat16, device=DEV)
    k, v = buf.as_strided((L, 1, 64), (ld, 64, 1)), buf.as_strided((L, 1, 64), (ld, 64, 1), 64)
    k.copy_(tensor(L, 1, 64, seed=2))
    v.copy_(tensor(L, 1, 64, seed=3))
    q = tensor(Lq, 2, 64)
    lse = torch.empty(Lq, 2, device=DEV)
    out = w8.w8a8_attention(q, k, v, lse=lse, kernel=kernel)
    check(out, lse, q, k, v, [0, Lq], [0, L], 64 ** -0.5)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("docs", [[(1, 3000), (1, 100)], [(300, 300), (77, 200)]])
def test_streams_graphs_and_repeats(w8, docs, kernel):
    lq, lk = [a for a, _ in docs], [b for _, b in docs]
    q, k, v = tensor(sum(lq), 4, 128), tensor(sum(lk), 2, 128, seed=2), tensor(sum(lk), 2, 128, seed=3)
    cu_q, cu_k = starts(lq), starts(lk)
    how = dict(causal=True, cu_q=cu_q, cu_k=cu_k, kernel=kernel)
    want = w8.w8a8_attention(q, k, v, **how)
    for _ in range(3):
        assert torch.equal(w8.w8a8_attention(q, k, v, **how), want)   # the same bits every time
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(q) for _ in streams]
    torch.cuda.synchronize()
    for s, o in zip(streams, outs):                                     # two calls at once
        w8.w8a8_attention(q, k, v, out=o, stream=s, **how)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    o = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w8.w8a8_attention(q, k, v, out=o, **how)
    q.copy_(tensor(sum(lq), 4, 128, seed=9))
    k.copy_(tensor(sum(lk), 2, 128, seed=10))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, w8.w8a8_attention(q, k, v, **how))


@pytest.mark.parametrize("kernel", KERNELS)
def test_no_queries_and_no_keys(w8, kernel):
    k = tensor(5, 2, 64)
    assert w8.w8a8_attention(k[:0], k, k).shape == (0, 2, 64)
    lse = torch.zeros(5, 2, device=DEV)
    for q in (k, tensor(200, 2, 64)):
        lse = torch.zeros(q.shape[0], 2, device=DEV)
        out = w8.w8a8_attention(q, k[:0], k[:0], lse=lse, kernel=kernel)
        assert bool((out == 0).all()) and bool((lse == -math.inf).all())


@pytest.mark.parametrize("kernel", KERNELS)
def test_starts_that_decrease_stay_in_bounds(w8, kernel):
    """Starts out of order or out of range give some rows or none, inside the arrays they are given."""
    q, k = tensor(64, 2, 64), tensor(64, 2, 64, seed=2)
    buf = torch.full((66, 2, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    for cu in ([0, 60, 20, 64], [-5, 30, 90, 10 ** 9], [64, 32, 16, 0], [2 ** 31 - 1, -2 ** 31, 5, 7]):
        c = torch.tensor(cu, dtype=torch.int32, device=DEV)
        w8.w8a8_attention(q, k, k, cu_q=c, cu_k=c.flip(0).contiguous(), out=buf[1:-1], causal=True,
                          kernel=kernel)
        torch.cuda.synchronize()
        assert bool((buf[0] == 3).all()) and bool((buf[-1] == 3).all())
    assert w8.w8a8_read_device_error() == 0


def test_refusals(w8):
    q, k = tensor(4, 4, 64), tensor(6, 2, 64)
    cu = starts([4])
    with pytest.raises(ValueError):
        w8.w8a8_attention(q, k, k[:5])
    with pytest.raises(ValueError):
        w8.w8a8_attention(q, k, tensor(6, 2, 128))
    with pytest.raises(TypeError):
        w8.w8a8_attention(q.float(), k, k)
    with pytest.raises(TypeError):
        w8.w8a8_attention(q, k, k, cu_q=cu.long())
    with pytest.raises(ValueError):
        w8.w8a8_attention(q, k, k, cu_q=cu, cu_k=starts([3, 3]))
    with pytest.raises(ValueError):
        w8.w8a8_attention(q, k, k, lse=torch.empty(4, 2, device=DEV))
    with pytest.raises(ValueError):
        w8.w8a8_attention(q, k, k, slopes=torch.ones(2, device=DEV))
    for bad in (dict(docs=3), dict(cap=-1.0), dict(scale=0.0), dict(scale=float("nan")), dict(cap=float("inf")),
                dict(prefix=torch.zeros(1, dtype=torch.int32, device=DEV)), dict(kernel=3)):
        with pytest.raises(w8.W8A8Error) as e:
            w8.w8a8_attention(q, k, k, **bad)
        assert e.value.status == 1
    with pytest.raises(w8.W8A8Error) as e:
        w8.w8a8_attention(tensor(4, 3, 64), k, k)     # 3 heads over 2
    assert e.value.status == 1
    with pytest.raises(w8.W8A8Error) as e:
        w8.w8a8_attention(tensor(4, 4, 96), tensor(6, 2, 96), tensor(6, 2, 96))
    assert e.value.status == 1
    wide = tensor(6, 2, 68)
    with pytest.raises(w8.W8A8Error) as e:
        w8.w8a8_attention(q, wide[..., :64], k)
    assert e.value.status == 2


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("how", ["plain", "causal bias", "prefix cap"])
def test_more_items_than_sms(w8, how, D):
    """The tile kernel's CTAs take several items each, one after the other, of long documents that end inside a tile
    (some of the heads are checked); twice in a row, with the same bits."""
    lengths, H = [2047, 15, 2223], 24
    q, k, v = [tensor(sum(lengths), H, D, seed=50 + i) for i in range(3)]
    cu = starts(lengths)
    slopes = 2.0 ** -(torch.arange(H, device=DEV) / 3.0)
    prefix = torch.tensor([700, 15, 1], dtype=torch.int32, device=DEV)
    args = {"plain": {}, "causal bias": dict(causal=True, slopes=slopes),
            "prefix cap": dict(causal=True, prefix=prefix, cap=20.0)}[how]
    got = []
    for _ in range(2):
        lse = torch.full((sum(lengths), H), 9.0, device=DEV)
        got.append((w8.w8a8_attention(q, k, v, cu_q=cu, cu_k=cu, lse=lse, kernel=w8.ATTENTION_TILES, **args), lse))
    torch.cuda.synchronize()
    assert w8.w8a8_read_device_error() == 0
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    for h in (0, 3, 11, 23):
        one = slice(h, h + 1)
        sub = dict(args, slopes=args["slopes"][one]) if "slopes" in args else args
        check(got[0][0][:, one], got[0][1][:, one], q[:, one], k[:, one], v[:, one], cu, cu, D ** -0.5, **sub)
