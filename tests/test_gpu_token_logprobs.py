"""token_logprobs on the GPU against its definition in binary64.

Bounds (e = 2^-24, half a binary32 step): a weight 2^y has relative error 2^-22 (ex2) + 16 e
(y's rounding, weighed by the weight itself); a thread adds up to n of them one after the
other, so s and t are within ds = 2^-21 + (n + 32) e.  lse: ds + 4 e |lse|.  log p: ds + 4 e
(|x| + |lse|).  entropy: ds (2 + H) + 8 e (1 + H).  The top tokens' indices are exact."""
import math

import pytest
import torch

from tests._decode_ref import DEV, logprobs_reference

pytestmark = pytest.mark.gpu
E = 2.0 ** -24


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import __graft_entry__
    __graft_entry__.build()
    import int8_weight_quantized_int4_gb300 as q
    return q


def check(q, x, tokens, k, **kw):
    r = q.token_logprobs(x, tokens, k=k, **kw)
    assert q.device_error() == 0
    tok = tokens[:, None] if tokens.dim() == 1 else tokens
    lp, ent, lse, top, idx = logprobs_reference(x, tok, k)
    ds = 2.0 ** -21 + (x.shape[1] / 256 + 9 + 32) * E

    def near(got, want, tol, what):
        got = got.double()
        same = torch.isinf(want) & (got == want)
        bad = ~(same | ((got - want).abs() <= tol))
        assert not bool(bad.any()), (what, got[bad][:4], want[bad][:4], tol[bad][:4])
    big = torch.where(lse.isinf(), 0.0, lse.abs())[:, None]
    xs = x.double().gather(1, tok.long()).abs().clamp_max(1e30)
    near(r.lse, lse, ds + 4 * E * big[:, 0], "lse")
    near(r.entropy, ent, ds * (2 + ent) + 8 * E * (1 + ent), "entropy")
    near(r.logprob.view(tok.shape), lp, ds + 4 * E * (xs + big), "logprob")
    if k:
        assert torch.equal(r.top_idx, idx), (r.top_idx[:2], idx[:2])
        xt = x.double().gather(1, idx.long()).abs().clamp_max(1e30)
        near(r.top_logprob, top, ds + 4 * E * (xt + big), "top")
    else:
        assert r.top_logprob is None and r.top_idx is None
    return r


def rand(M, N, dtype, seed=0, scale=3.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = (torch.randn(M, N, generator=g, device=DEV) * scale).to(dtype)
    return x, torch.randint(0, N, (M,), generator=g, device=DEV)


TYPES = [torch.float16, torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N", [(1, 1), (2, 7), (3, 64), (5, 1000), (1, 4097), (64, 2048), (2, 50257), (1, 248320),
                                 (800, 300), (900, 5001), (70, 128257)])
def test_shapes(q, dtype, M, N):
    x, tok = rand(M, N, dtype, seed=M + N)
    for k in sorted({0, 1, min(5, N), min(20, N), min(64, N)}):
        check(q, x, tok if k % 2 else tok.int(), k)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,off", [(3, 0), (5, 1), (8, 3), (1, 7)])
def test_strided_and_unaligned_rows(q, dtype, pad, off):
    """Rows of a padded matrix that start anywhere; the padding holds NaN."""
    M, N = 6, 3001
    buf = torch.full((M, N + pad + off), float("nan"), device=DEV, dtype=dtype)
    x, tok = rand(M, N, dtype, seed=pad)
    view = buf[:, off:off + N]
    view.copy_(x)
    check(q, view, tok, 10)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N", [(2, 5000), (1, 248320), (780, 20001)])
def test_ties(q, dtype, M, N):
    """Equal logits come by index: all equal, a handful of values, and zeros of both signs."""
    tok = torch.zeros(M, dtype=torch.int64, device=DEV)
    check(q, torch.full((M, N), 1.25, device=DEV, dtype=dtype), tok, 64)
    g = torch.Generator(device=DEV).manual_seed(N)
    few = torch.randint(0, 3, (M, N), generator=g, device=DEV).to(dtype)
    check(q, few, tok, 64)
    x = torch.where(torch.rand(M, N, generator=g, device=DEV) < 0.5, -0.0, 0.0).to(dtype)
    check(q, x, tok, 20)
    x, _ = rand(M, N, torch.bfloat16, seed=2, scale=1.0)        # bf16 values: many ties
    check(q, x.to(dtype), tok, 64)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("left", [0, 1, 3, 19, 20, 21, 200])
def test_masked_vocabulary(q, dtype, left):
    """-inf, or the type's lowest value, everywhere but at `left` tokens."""
    for M, N in ((3, 40000), (770, 2001)):
        x, tok = rand(M, N, dtype, seed=left)
        g = torch.Generator(device=DEV).manual_seed(left)
        keep = torch.zeros(M, N, dtype=torch.bool, device=DEV)
        keep.scatter_(1, torch.argsort(torch.rand(M, N, generator=g, device=DEV))[:, :left], True)
        check(q, x.masked_fill(~keep, float("-inf")), tok, 20)
        if dtype != torch.float32 or left:
            # binary32's lowest value times log2(e) is -inf: still a probability of 0
            low = x.masked_fill(~keep, torch.finfo(dtype).min if dtype == torch.float16 else -3.0e4)
            check(q, low, tok, 20)


def test_all_masked_row(q):
    x, tok = rand(4, 3000, torch.float16)
    x[1] = float("-inf")
    r = check(q, x, tok, 5)
    assert r.lse[1] == -math.inf and r.logprob[1] == -math.inf and r.entropy[1] == 0
    assert r.top_idx[1].tolist() == [0, 1, 2, 3, 4] and bool((r.top_logprob[1] == -math.inf).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("left", [0, 1, 20, 200])
@pytest.mark.parametrize("low", ["lowest", -1.0e9, -1.0e30])
def test_masked_with_large_finite_values(q, dtype, left, low):
    """Masks of the type's lowest value or another large one: with `left` tokens besides, the
    others have no probability; alone, they are equally likely."""
    low = torch.finfo(dtype).min if low == "lowest" else low
    for M, N in ((3, 40000), (770, 2001)):
        x, tok = rand(M, N, dtype, seed=left)
        g = torch.Generator(device=DEV).manual_seed(left)
        keep = torch.zeros(M, N, dtype=torch.bool, device=DEV)
        keep.scatter_(1, torch.argsort(torch.rand(M, N, generator=g, device=DEV))[:, :left], True)
        check_far(q, x.masked_fill(~keep, low), tok, 20)


def check_far(q, x, tok, k):
    """Against logits less their row's maximum, m (exact in binary64): log p = (x - m) - log s
    has one rounding of x - m (2 e |x - m|, <= 2 e (|log p| + log N)), the others' as in check."""
    r = q.token_logprobs(x, tok, k=k)
    assert q.device_error() == 0
    m = x.double().amax(1, keepdim=True)
    lp, ent, lse, top, idx = logprobs_reference(x.double() - m, tok[:, None], k)
    ds = 2.0 ** -21 + (x.shape[1] / 256 + 41) * E
    far = math.log(x.shape[1]) + 2

    def near(got, want, tol, what):
        err = (got.double() - want).abs()
        assert bool((err <= tol).all()), (what, float((err / tol).max()))
    near(r.lse, lse + m[:, 0], ds + 4 * E * (lse + m[:, 0]).abs() + 4 * E * m[:, 0].abs(), "lse")
    near(r.entropy, ent, ds * (2 + ent) + 8 * E * (1 + ent), "entropy")
    near(r.logprob, lp[:, 0], ds + 4 * E * (lp[:, 0].abs() + far), "logprob")
    near(r.top_logprob, top, ds + 4 * E * (top.abs() + far), "top")
    assert torch.equal(r.top_idx, idx)


@pytest.mark.parametrize("shift", [1.0e6, -1.0e6, 1.0e8, -1.0e12])
def test_far_from_zero(q, shift):
    """binary32 logits a long way from zero: the differences between them are what counts."""
    step = max(1.0, 2.0 ** math.ceil(math.log2(abs(shift) * 2.0 ** -23)))       # distinct after rounding
    for M, N in ((2, 30000), (770, 2001)):
        x, tok = rand(M, N, torch.float32, seed=4)
        check_far(q, (x.double() * step + shift).float(), tok, 20)


@pytest.mark.parametrize("dtype", TYPES)
def test_large_values_in_few_places(q, dtype):
    """The best logits crowded where one thread reads them (its list overflows and the
    threshold rises), and sorted rows."""
    ve = 16 // torch.empty(0, dtype=dtype).element_size()
    M, N = 800, 100000
    x = torch.zeros(M, N, device=DEV, dtype=dtype)
    base = torch.randn(M, N, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)) * 0.1
    col = torch.arange(N, device=DEV)
    crowd = (col // ve) % 256 < 19
    ramp = (col % 2039).float() / 64
    x = torch.where(crowd, 4 + ramp, base).to(dtype)
    tok = torch.full((M,), 5, device=DEV)
    check(q, x, tok, 64)
    check(q, x, tok, 20)
    up = torch.linspace(-8, 8, 30000, device=DEV).to(dtype).expand(3, -1).contiguous()
    check(q, up, tok[:3], 64)
    check(q, up.flip(1).contiguous(), tok[:3], 64)


def test_peaked_rows_keep_small_entropies(q):
    """One token holds nearly all probability: entropy and log p near 0 without cancellation."""
    x = torch.zeros(5, 5000, device=DEV)
    for i, v in enumerate((10.0, 20.0, 25.0, 30.0, 60.0)):
        x[i, 77 * i + 3] = v
    tok = torch.tensor([3, 80, 157, 234, 311], device=DEV)
    check(q, x, tok, 3)
    check(q, x + 1000.0, tok, 3)


def test_several_tokens_and_bad_ones(q):
    x, _ = rand(7, 999, torch.bfloat16)
    tok = torch.randint(0, 999, (7, 6), device=DEV)
    check(q, x, tok, 2)
    check(q, x, tok[:, :0], 2)
    tok[2, 3], tok[5, 0] = 999, -1
    r = q.token_logprobs(x, tok)
    assert q.device_error() == q.QW_ERR_BAD_INDEX and q.device_error() == 0
    nan = torch.isnan(r.logprob)
    assert nan.sum() == 2 and bool(nan[2, 3]) and bool(nan[5, 0])


def test_nan_and_inf(q):
    x, tok = rand(3, 4000, torch.float32)
    x[0, 1000], x[1, 17] = float("nan"), float("inf")
    r = q.token_logprobs(x, tok, k=4)
    assert q.device_error() == 0
    assert bool(torch.isnan(r.lse[:2]).all()) and bool(torch.isfinite(r.lse[2]))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,k", [(3, 20, 20), (2, 4097, 64), (1, 248320, 20), (800, 3000, 7)])
@pytest.mark.parametrize("left", [0, 1, 5, 70])
def test_indices_of_nan_rows_are_columns(q, dtype, M, N, k, left):
    """Rows of NaN of either sign but for `left` logits: sums are NaN, and the indices are k
    different columns, so that a gather with them stays inside the row."""
    g = torch.Generator(device=DEV).manual_seed(left)
    word = {2: torch.int16, 4: torch.int32}[torch.empty(0, dtype=dtype).element_size()]
    for sign in (1.0, -1.0, 0.0):
        nan = torch.full((M, N), float("nan"), dtype=dtype, device=DEV).view(word)
        low = torch.iinfo(word).min
        if sign < 0:
            nan |= low
        elif sign == 0:
            nan |= torch.randint(0, 2, (M, N), generator=g, device=DEV).to(word) * low
        x = nan.view(dtype)
        at = torch.argsort(torch.rand(M, N, generator=g, device=DEV))[:, :min(left, N - 1)]
        x.scatter_(1, at, torch.randn(M, N, generator=g, device=DEV).to(dtype)[:, :at.shape[1]])
        r = q.token_logprobs(x, torch.zeros(M, dtype=torch.int32, device=DEV), k=k)
        assert q.device_error() == 0
        assert bool(torch.isnan(r.lse).all()) and bool(torch.isnan(r.top_logprob).all())
        idx = torch.sort(r.top_idx, dim=1).values
        assert int(idx.min()) >= 0 and int(idx.max()) < N, (sign, r.top_idx[0])
        assert bool((idx[:, 1:] > idx[:, :-1]).all())
        # the numbers first, largest first, then NaN by index
        v = x.double()
        order = torch.sort(torch.where(torch.isnan(v), float("inf"), -v), dim=1, stable=True).indices[:, :k]
        assert torch.equal(r.top_idx.long(), order)


def test_workspace_is_shared_by_calls_of_any_shape(q):
    ws = q.Workspace(torch.device("cuda:0"))
    for M, N, k in ((700, 3000, 64), (3, 248320, 20), (1, 50000, 64), (200, 9000, 5), (700, 3000, 1), (64, 128257, 20)):
        x, tok = rand(M, N, torch.float16, seed=M)
        check(q, x, tok, k, ws=ws)


def test_repeats_bitwise_streams_and_graph(q):
    x, tok = rand(16, 100003, torch.float16)
    a = check(q, x, tok, 20)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(10):
            b = q.token_logprobs(x, tok, k=20)
    s.synchronize()
    for u, v in zip(a, b):
        assert torch.equal(u, v)
    g = torch.cuda.CUDAGraph()
    ws = q.Workspace(torch.device("cuda:0"))
    q.token_logprobs(x, tok, k=20, ws=ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        c = q.token_logprobs(x, tok, k=20, ws=ws)
    x.copy_(rand(16, 100003, torch.float16, seed=5)[0])
    g.replay()
    torch.cuda.synchronize()
    want = q.token_logprobs(x, tok, k=20)
    for u, v in zip(c, want):
        assert torch.equal(u, v)


def test_rows_past_2_to_31_elements(q):
    M, N = 9000, 248320
    x = torch.zeros(M, N, dtype=torch.float16, device=DEV)
    x[-1, 200000] = 9.0
    tok = torch.zeros(M, dtype=torch.int32, device=DEV)
    r = q.token_logprobs(x, tok, k=1)
    assert q.device_error() == 0
    assert int(r.top_idx[-1, 0]) == 200000 and int(r.top_idx[0, 0]) == 0
    assert abs(float(r.lse[-1]) - math.log(N - 1 + math.exp(9.0))) < 1e-5


def test_binding_refusals(q):
    x, tok = rand(2, 100, torch.float16)
    with pytest.raises(TypeError):
        q.token_logprobs(x.double(), tok)
    with pytest.raises(ValueError):
        q.token_logprobs(x.t(), tok)
    with pytest.raises(TypeError):
        q.token_logprobs(x, tok.float())
    with pytest.raises(ValueError):
        q.token_logprobs(x, tok[:1])
    with pytest.raises(q.QgemmError):
        q.token_logprobs(x, tok, k=65)
    r = q.token_logprobs(x[:0], tok[:0], k=3)
    assert r.logprob.shape == (0,) and r.top_idx.shape == (0, 3)
