"""sample_tokens against its definition in binary64 (tests/_tree_ref.py).

Tolerances.  A weight from 2^-12 on is a whole number of 2^-40 within 2e-11 of its value, a lighter
one within 4e-6 of it (binary32; thousands of them that round differently, so that less than
1e-7 of their sum is left), and so is a running sum of the total (N 2^-41 / total <= 2^20 2^-41 <
5e-7 only if all N weights were rounded to whole numbers the same way; independent, below 1e-9);
the sum that top-p takes its share of is within 1e-7 of the part below the border.  So the draw has to be the definition's for some number within 1e-7 of u
and of top_p (relative); its log probability, that answer's within 2^-22 (relative; absolute
below 1): one rounding of the quotient, one of log1p (2 ulp), the weights."""
import ctypes
import math

import numpy as np
import pytest
import torch

import int8_weight_quantized_int4_gb300 as q
from tests import _tree_ref as ref

pytestmark = pytest.mark.gpu
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def check(logits, u, **kw):
    r = q.sample_tokens(logits, u, **kw)
    again = q.sample_tokens(logits, u, **kw)
    assert torch.equal(r.token, again.token) and torch.equal(r.logprob, again.logprob)
    assert q.device_error() == 0
    x, uu = logits.double().cpu().numpy(), u.double().cpu().numpy()
    rows = {n: v.double().cpu().numpy() if torch.is_tensor(v) else np.full(len(uu), np.float64(np.float32(v)))
            for n, v in kw.items()}
    token, lp = r.token.tolist(), r.logprob.double().tolist()
    for i in range(len(uu)):
        f = {n: (int(v[i]) if n == "top_k" else v[i]) for n, v in rows.items()}
        ok = ref.draws(x[i], uu[i], **f)
        assert token[i] in ok, (i, token[i], ok, f, uu[i])
        assert any(lp[i] == e or abs(lp[i] - e) <= 2 ** -22 * max(1.0, abs(e)) for e in ok[token[i]]), (i, lp[i], ok, f)
    return r


def make(M, N, dtype, seed, spread=2.5, peaks=32):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, N, generator=g) * spread
    if peaks:
        at = torch.randint(0, N, (M, peaks), generator=g)
        x.scatter_(1, at, torch.rand(M, peaks, generator=g) * 10 + 3)
    return x.to(TYPES[dtype]).cuda(), torch.rand(M, generator=g).cuda()


FILTERS = [dict(), dict(top_k=1), dict(top_k=40), dict(temperature=0.7, top_p=0.9), dict(min_p=0.03),
           dict(temperature=1.3, top_k=100, top_p=0.8, min_p=0.02), dict(temperature=0.0), dict(top_p=0.999),
           dict(top_k=3000, top_p=0.97), dict(temperature=2.0, top_k=700)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("M,N", [(1, 1), (3, 2), (5, 7), (4, 33), (9, 1000), (6, 4097), (3, 50257), (700, 513), (2, 131073),
                                 (1, 262144), (640, 2049)])
def test_filters(M, N, dtype):
    x, u = make(M, N, dtype, M * 7 + N)
    for kw in FILTERS if M < 100 else FILTERS[:6]:
        check(x, u, **kw)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_a_setting_a_row(dtype):
    x, u = make(48, 6000, dtype, 3)
    g = torch.Generator().manual_seed(4)

    def pick(v, t=torch.float32):
        return torch.tensor(v, dtype=t)[torch.randint(0, len(v), (48,), generator=g)].cuda()
    check(x, u, temperature=pick([0.0, 0.5, 1.0, 1.7, -1.0]), top_k=pick([0, 1, 7, 300, 5999, 6000, 9000, -3], torch.int32),
          top_p=pick([1.0, 0.9, 0.3, 0.0, 1.5]), min_p=pick([0.0, 0.1, 1.0, -0.5]))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("N", [100, 3001, 40000])
def test_flat_rows_and_ties(N, dtype):
    """Lists that overflow: all equal, few values, a wide and flat distribution."""
    g = torch.Generator().manual_seed(N)
    few = torch.round(torch.randn(4, N, generator=g) * 2) / 2
    flat = torch.randn(4, N, generator=g) * 0.05
    same = torch.full((2, N), -7.25)
    x = torch.cat([few, flat, same]).to(TYPES[dtype]).cuda()
    u = torch.rand(10, generator=g).cuda()
    for kw in (dict(), dict(top_k=N // 3), dict(top_p=0.6), dict(top_k=N // 2, top_p=0.5), dict(min_p=0.9), dict(temperature=0.0),
               dict(top_k=5, top_p=0.5), dict(top_p=0.99, min_p=0.3), dict(top_k=N // 3, min_p=1.0)):
        check(x, u, **kw)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("N", [65, 20011])
def test_masked_places(N, dtype):
    x, u = make(12, N, dtype, N)
    g = torch.Generator().manual_seed(9)
    hide = (torch.rand(12, N, generator=g) < 0.97).cuda()
    hide[:, 3] = False
    low = torch.finfo(x.dtype).min
    for v in (float("-inf"), low, float("nan")):
        y = x.masked_fill(hide, v)
        y[1] = v                                       # a row of nothing else
        y[2, : N // 2] = v
        y[3] = float("-inf")
        y[4] = low
        y[5] = float("nan")
        for kw in (dict(), dict(top_k=20), dict(top_p=0.9), dict(min_p=0.05), dict(temperature=0.0),
                   dict(top_k=50, top_p=0.7, min_p=0.01), dict(temperature=1e-3), dict(top_k=N - 1)):
            check(y, u, **kw)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_infinite_logits(dtype):
    x, u = make(6, 3000, dtype, 1)
    x[0, 17] = x[0, 2900] = float("inf")
    x[1, 5] = float("inf")
    x[2, ::3] = float("inf")
    x[3, 100] = float("inf")
    x[3, 101] = float("-inf")
    x[3, 102] = float("nan")
    for kw in (dict(), dict(top_k=20), dict(top_p=0.9), dict(min_p=0.05), dict(temperature=0.0), dict(top_k=2, top_p=0.4)):
        check(x, u, **kw)


def test_strided_rows_and_borders_of_u():
    x, _ = make(8, 5001, "bf16", 5)
    wide = torch.zeros(8, 9001, dtype=torch.bfloat16, device="cuda")
    wide[:, 2001:7002] = x
    u = torch.tensor([0.0, 1.0 - 2 ** -24, 0.5, 1e-30, 0.999, 0.25, 0.75, 1.0], device="cuda")
    for kw in (dict(), dict(top_k=30), dict(top_p=0.8)):
        r = check(wide[:, 2001:7002], u, **kw)
        s = check(x, u, **kw)
        assert torch.equal(r.token, s.token) and torch.equal(r.logprob, s.logprob)
    one = q.sample_tokens(x[2:3], u[2:3], top_p=0.8)          # a row alone: spread over more CTAs
    assert one.token.item() == s.token[2].item()
    # out-of-range numbers draw the first or the last of what stays
    odd = q.sample_tokens(x[:4], torch.tensor([-1.0, 2.0, float("nan"), float("inf")], device="cuda"), top_k=3)
    best = torch.topk(x[:4].float(), 3).indices.sort(1).values
    assert odd.token.tolist() == [best[0, 0], best[1, 2], best[2, 0], best[3, 2]]


def test_greedy_takes_the_first_of_equals():
    x = torch.zeros(3, 9000, device="cuda")
    x[0, 8000] = x[0, 4000] = x[0, 4001] = 2.0
    x[1, 1:] = -0.0
    r = q.sample_tokens(x, torch.rand(3, device="cuda"), temperature=0)
    assert r.token.tolist() == [4000, 0, 0] and r.logprob.tolist() == [0, 0, 0]


def test_largest_row():
    N = 1 << 20
    x, u = make(2, N, "bf16", 8)
    for kw in (dict(), dict(top_k=64), dict(top_p=0.9), dict(top_k=5000)):
        check(x, u, **kw)


def test_shares_follow_the_probabilities():
    """The u's of an even grid draw each token as often as its probability says, within one."""
    x, _ = make(1, 300, "fp32", 12, spread=1.0, peaks=0)
    n = 4096
    u = ((torch.arange(n, dtype=torch.float32) + 0.5) / n).cuda()
    r = q.sample_tokens(x.expand(n, 300), u, top_k=50)
    w = torch.softmax(torch.topk(x[0].double(), 50).values, 0)
    got = torch.bincount(r.token.long(), minlength=300)[torch.topk(x[0], 50).indices]
    assert (got - w * n).abs().max() <= 1.0 + 1e-3 and int(got.sum()) == n


def test_streams_graphs_and_empty():
    x, u = make(16, 7000, "fp16", 2)
    want = q.sample_tokens(x, u, top_p=0.9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = q.sample_tokens(x, u, top_p=0.9)
    side.synchronize()
    assert torch.equal(other.token, want.token)
    p = torch.full((16,), 0.9, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = q.sample_tokens(x, u, top_p=p)
    for _ in range(2):
        g.replay()
        assert torch.equal(r.token, want.token) and torch.equal(r.logprob, want.logprob)
    x.copy_(make(16, 7000, "fp16", 77)[0])
    p.fill_(0.5)
    g.replay()
    assert torch.equal(r.token, q.sample_tokens(x, u, top_p=0.5).token)
    none = q.sample_tokens(x[:0], u[:0])
    assert none.token.shape == (0,)


def test_binding_refusals():
    x, u = make(4, 50, "fp16", 2)
    with pytest.raises(TypeError):
        q.sample_tokens(x.double(), u)
    with pytest.raises(TypeError):
        q.sample_tokens(x.cpu(), u)
    with pytest.raises(ValueError):
        q.sample_tokens(x.T, u)
    with pytest.raises(ValueError):
        q.sample_tokens(x, u[:3])
    with pytest.raises(TypeError):
        q.sample_tokens(x, u.double())
    with pytest.raises(TypeError):
        q.sample_tokens(x, u, top_k=torch.ones(4, device="cuda"))
    with pytest.raises(ValueError):
        q.sample_tokens(x, u, top_p=torch.ones(5, device="cuda"))
    with pytest.raises(ValueError):
        q.sample_tokens(x, u, top_k=1 << 40)
    with pytest.raises(q.QgemmError):
        q.sample_tokens(x[:, :0], u)


@pytest.mark.parametrize("N", [33, 50257])
def test_one_row_for_all(N):
    """Logits broadcast over the rows (a stride of 0), in two streams at once."""
    g = torch.Generator(device="cuda").manual_seed(N)
    x = torch.randn(1, N, generator=g, device="cuda").half() * 3
    u = torch.rand(40, generator=g, device="cuda")
    kw = dict(temperature=0.9, top_k=100, top_p=0.9, min_p=0.01)
    want = q.sample_tokens(x.repeat(40, 1), u, **kw)
    got = [q.sample_tokens(x.expand(40, N), u, **kw)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(q.sample_tokens(x.expand(40, N), u, **kw))
    torch.cuda.synchronize()
    assert all(torch.equal(want.token, y.token) and torch.equal(want.logprob, y.logprob) for y in got)


@pytest.mark.parametrize("n", [30, 63, 64, 65, 127, 128, 129, 255, 256, 257, 400, 1023, 1024, 1025])
@pytest.mark.parametrize("ties", [False, True])
def test_lists_of_every_length(n, ties):
    """n logits far above the rest, all different or many alike, cut in every way."""
    rng = np.random.default_rng(n)
    N, M = 20000, 24
    x = np.full((M, N), -40.0)
    for r in range(M):
        at = rng.choice(N, n, replace=False)
        x[r, at] = rng.choice([0.0, 0.5, 1.0], n) if ties else rng.permutation(n) / n * 3
    x = torch.tensor(x, dtype=torch.float32, device="cuda")
    u = torch.tensor(rng.random(M), dtype=torch.float32, device="cuda")
    for kw in (dict(top_k=n), dict(top_k=max(n // 2, 1)), dict(top_k=7), dict(top_k=max(n - 1, 1), top_p=0.7), dict(top_p=0.5),
               dict(top_p=0.97), dict(min_p=0.2), dict(top_k=n // 3, top_p=0.9, min_p=0.3)):
        check(x, u, **kw)


@pytest.mark.parametrize("temperature", [1e-38, 1e-30, 1e-6, 1e6, 1e30, float("inf")])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_extreme_temperatures(temperature, dtype):
    """From the largest logit alone to equal weights, which no list holds; a tenth of the places masked."""
    x, u = make(7, 20011, dtype, 41)
    x[:, ::10] = -math.inf
    for kw in (dict(), dict(top_k=700), dict(top_k=5000), dict(top_p=0.9), dict(top_k=9000, top_p=0.7), dict(min_p=0.5)):
        check(x, u, temperature=temperature, **kw)


@pytest.mark.parametrize("top_p", [0.0, -0.1, -math.inf])
def test_a_top_p_not_above_0_leaves_the_first(top_p):
    """Also of rows that no list holds."""
    g = torch.Generator().manual_seed(50)
    x = torch.cat([torch.full((2, 40000), 1.5), torch.randn(2, 40000, generator=g) * 0.01]).half().cuda()
    x[1, :7] = 0.0
    u = torch.tensor([0.3, 0.9, 0.0, 0.999], device="cuda")
    for kw in (dict(), dict(top_k=30), dict(top_k=3000), dict(top_k=30000, min_p=0.5)):
        r = check(x, u, top_p=top_p, **kw)
        assert r.token.tolist() == [0, 7, *x[2:].float().argmax(1).tolist()]
        per_row = torch.full((4,), top_p, device="cuda")
        assert torch.equal(q.sample_tokens(x, u, top_p=per_row, **kw).token, r.token)


def test_every_row_is_drawn_where_weights_lie_at_the_bar_of_min_p():
    """200 logits within 1e-5 to 1e-9 of where the weight is min_p: some weights of logits next to each other
    round the other way round there.  Every row's token is written, and its weight reaches min_p within 4e-6."""
    g = torch.Generator().manual_seed(60)
    M, N = 1 << 17, 200
    for width in (1e-6, 1e-8, 1e-9):
        mp = torch.exp(torch.rand(M, generator=g, dtype=torch.float64) * -8.3).float()
        t = (torch.rand(M, generator=g) * 3 + 0.2)
        top = -t.double() * mp.double().log()
        x = torch.randn(M, N, generator=g) * width - (top - top.float().double()).float()[:, None]
        x[:, 0] = top.float()
        u = torch.rand(M, generator=g)
        x, u, t, mp = (v.cuda() for v in (x, u, t, mp))
        token, lp = torch.full((M,), -7777, dtype=torch.int32, device="cuda"), torch.full((M,), 1.0, device="cuda")
        s = q.SamplingDesc(temperature=1.0, top_p=1.0, temperatures=t.data_ptr(), min_ps=mp.data_ptr())
        ptr = [ctypes.c_void_p(v.data_ptr()) for v in (x, u, token, lp)]
        assert q.lib().sample_tokens(ptr[0], q.QW_F32, M, N, N, ptr[1], s, *ptr[2:], ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
        torch.cuda.synchronize()
        assert bool(((token >= 0) & (token < N)).all()) and bool((lp <= 0).all())
        w = torch.exp((x.gather(1, token.long()[:, None])[:, 0].double() - x[:, 0].double()) / t.double())
        assert bool((w >= mp.double() * (1 - 4e-6)).all())


def log_shares(x, token, temperature=1.0, top_k=0):
    """Log probabilities of the tokens (one a row of x, binary64) among the top_k."""
    t = float(np.float32(temperature))
    w = np.exp((x - x.max(1, keepdims=True)) / t)
    total = np.sort(w, 1)[:, -top_k:].sum(1) if top_k else w.sum(1)
    at = np.arange(len(x)), token
    return (x[at] - x.max(1)) / t - np.log(total)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("kw", [dict(), dict(temperature=1.1), dict(top_k=149999), dict(temperature=0.9, top_k=100000)])
def test_log_probabilities_of_far_tokens(dtype, kw):
    """A vocabulary far below one logit, drawn from.  The logarithm: the distance of the logit (exact), its
    quotient and log1p of the total (an ulp each) and their difference, all below 2^-22 of the result."""
    N, gaps, parts = 150000, (12.0, 17.0, 19.0, 20.5), (0.02, 0.2, 0.45, 0.7, 0.95)
    g = torch.Generator().manual_seed(51)
    x = (torch.randn(len(gaps), N, generator=g) * 0.5).to(TYPES[dtype])
    x[:, 70000] = torch.tensor(gaps)
    x = x.repeat_interleave(len(parts), 0)
    y = x.double().numpy()
    w = np.exp((y - y.max(1, keepdims=True)) / float(np.float32(kw.get("temperature", 1.0))))
    far = w[:, 70001:].sum(1) / w.sum(1)
    u = torch.tensor(1 - far * np.tile(parts, len(gaps)), dtype=torch.float32).cuda()
    r = q.sample_tokens(x.cuda(), u, **kw)
    want = log_shares(y, r.token.cpu().numpy(), **kw)
    err = np.abs(r.logprob.double().cpu().numpy() - want)
    assert q.device_error() == 0 and (want < -12).sum() >= 15
    assert (err <= 2 ** -22 * np.maximum(1, np.abs(want))).all(), (err / np.abs(want)).max()


def beside_borders(x, lo, hi, inside=(0.0, 1.0), temperature=1.0, most=400):
    """Numbers (float32) whose nearest border between two tokens' shares of the row x (binary64) is between lo
    and hi away, within `inside`; and the tokens that they draw."""
    w = np.exp((x - x.max()) / float(np.float32(temperature)))
    sums = np.cumsum(w.astype(np.longdouble))
    sums = (sums / sums[-1]).astype(np.float64)
    b = sums[(sums > inside[0]) & (sums < inside[1])]
    near = b.astype(np.float32)
    step = int(math.ceil(hi / 2 ** -25))
    grid = np.unique(np.concatenate([near + np.float32(i * 2 ** -25) for i in range(-step, step + 1)]).astype(np.float32)).astype(np.float64)
    at = np.searchsorted(sums, grid)
    gap = np.minimum(np.abs(sums[np.minimum(at, len(sums) - 1)] - grid), np.abs(grid - sums[np.maximum(at - 1, 0)]))
    grid = grid[(gap >= lo) & (gap <= hi)]
    grid = grid[np.random.default_rng(0).permutation(len(grid))[:most]]
    return torch.tensor(grid, dtype=torch.float32), torch.tensor(np.searchsorted(sums, grid, side="right"), dtype=torch.int32)


def check_borders(x, lo, hi, fewest, temperature=1.0, inside=(0.35, 0.65), filters=(dict(), dict(min_p=1e-9))):
    u, want = beside_borders(x.double().numpy(), lo, hi, inside, temperature)
    assert len(u) >= fewest, len(u)
    rows = x.cuda()[None].expand(len(u), -1)
    for kw in filters:
        got = q.sample_tokens(rows, u.cuda(), temperature=temperature, **kw).token.cpu()
        assert torch.equal(got, want), (kw, int((got != want).sum()), len(u))
    assert q.device_error() == 0


@pytest.mark.parametrize("dtype,top,rest", [("fp16", 7.8984375, 2.4438e-4), ("fp16", 4.5, 3 * 2.0 ** -24), ("bf16", 7.90625, 0.9 * 2.0 ** -22),
                                            ("fp32", 7.8984375, 2.4438e-4)])
def test_weights_of_logits_near_zero(dtype, top, rest):
    """A difference from the largest logit that binary32 does not hold: draws 3e-9 from a border, where weights within
    2e-11 and half a unit (1.2e-13 of the largest) move it by 1e-10."""
    n = int(round(math.exp(top)))
    x = torch.full((n + 1,), rest).to(TYPES[dtype])
    x[0] = top
    check_borders(x, 3e-9, 2.5e-8, 10)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("gap", [6.5625, 6.4375, 6.0, 5.875])
def test_weights_of_a_rounded_exponent(dtype, gap):
    """Differences whose product with log2(e) is rounded far: draws 2.5e-10 from a border, where weights of 1.4e-3
    within 4e-11 and a unit of 2^-40 (6.5e-10 of them) move it by 1.8e-10."""
    x = torch.zeros(int(round(math.exp(gap))) + 1).to(TYPES[dtype])
    x[0] = gap
    check_borders(x, 2.5e-10, 1.5e-9, 2)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("gap", [8.25, 7.5])
def test_weights_are_rounded_to_fine_units(dtype, gap):
    """Thousands of equal weights, all rounded alike: draws 1.5e-10 from a border, where weights of 2^-12 within 4e-11
    and half a unit of 2^-42 (4.4e-10 of them) move it by a quarter of that, 1.2e-10."""
    x = torch.zeros(int(round(math.exp(gap))) + 1).to(TYPES[dtype])
    x[0] = gap
    check_borders(x, 1.5e-10, 4.5e-10, 6)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("gap", [18.0, 22.0])
def test_a_flat_vocabulary_far_below_one_logit(dtype, gap):
    """2^20 - 1 equal tokens: the draw is the definition's for some number within 1e-7 (weights within 3e-7 of an even
    part of all) and half a unit of 2^-42 a token (1.2e-7) of u."""
    N = 1 << 20
    x = torch.zeros(1, N)
    x[0, 0] = gap
    x = x.to(TYPES[dtype])
    w = math.exp(-gap)
    share = (N - 1) * w / (1 + (N - 1) * w)
    u = torch.tensor([1 - share * f for f in (0.999, 0.97, 0.8, 0.5, 0.1)], dtype=torch.float32)
    eps = 1e-7 + N * 2.0 ** -43
    for kw in (dict(), dict(top_k=N - 1)):
        r = q.sample_tokens(x.cuda().expand(5, N), u.cuda(), **kw)
        total = 1 + (N - 1 - bool(kw)) * w
        for token, lp, v in zip(r.token.tolist(), r.logprob.tolist(), u.double().tolist()):
            assert token >= 1 and v - eps < (1 + token * w) / total and v + eps >= (1 + (token - 1) * w) / total, (kw, token, v)
            assert abs(lp + gap + math.log(total)) <= 2 ** -22 * gap


@pytest.mark.parametrize("dtype", list(TYPES))
def test_light_weights_have_no_common_error(dtype):
    """Half of the sum in weights of 2^-17 to 2^-20, at a temperature whose log2(e) / t rounds far: within 2^-22 (ex2)
    and four sums' 2^-24, all alike at the worst, they move a border by a quarter of 4.8e-7, and rounding 320,000 of
    them to units of 2^-42 by 3.6e-8."""
    g = torch.Generator().manual_seed(53)
    n = 320000
    x = -1.1 * math.log(2) * (17 + 3 * torch.rand(n + 1, generator=g))
    x[0] = 0.0
    check_borders(x.to(TYPES[dtype]), 1.58e-7, 1.78e-7, 50, temperature=1.1)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_top_p_counts_what_lies_far_below(dtype):
    """Half of the sum in 320,000 tokens far below the border of top_p, the other in 30: which of these stay.  An
    error that the far ones' weights share (log2(e) / t rounded: 5.5e-7) would move the border by a quarter of it; ex2's
    2^-22, and what sums of independent roundings leave of 2^-24 a step (1e-7), by 8e-8."""
    g = torch.Generator().manual_seed(54)
    n, few, t = 320000, 30, 1.1
    x = torch.cat([-torch.arange(few) * 0.03125, -t * math.log(2) * (13.5 + torch.rand(n, generator=g))]).to(TYPES[dtype])
    y = x.double().numpy()
    w = np.exp((y - y.max()) / float(np.float32(t)))
    total = w.sum()
    assert 0.35 < w[few:].sum() / total < 0.65
    sums = np.cumsum(w[:few]) / total
    p, want = [], []
    for j, s in enumerate(sums):
        if 0.3 < s < 0.5:
            near = np.float32(s)
            for i in range(-8, 9):
                v = float(near + np.float32(i * 2 ** -25))
                if 0.8e-7 <= abs(v - s) <= 1.3e-7:
                    p.append(v)
                    want.append(j + (v > s))
    assert len(p) >= 10
    u = torch.full((len(p),), 1 - 2 ** -24, device="cuda")
    got = q.sample_tokens(x.cuda()[None].expand(len(p), -1), u, temperature=t, top_p=torch.tensor(p, device="cuda")).token.tolist()
    assert got == want


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("temperature", [0.8, 1.1, 3.0, math.inf])
def test_infinite_logits_at_any_temperature(dtype, temperature):
    """Two of three weights of 1 stay, or one: nothing else counts towards top_p."""
    x, _ = make(8, 3000, dtype, 61)
    x[:, 17] = x[:, 1500] = x[:, 2900] = math.inf
    u = torch.tensor([0.0, 0.2, 0.4, 0.6, 0.8, 0.9, 0.95, 0.999], device="cuda")
    for p, n in ((0.5, 2), (0.3, 1), (0.9, 3)):
        for kw in (dict(), dict(min_p=0.1), dict(top_k=2999)):
            r = q.sample_tokens(x, u, temperature=temperature, top_p=p, **kw)
            assert r.token.tolist() == [(17, 1500, 2900)[int(v * n)] for v in u.tolist()]
            assert bool(((r.logprob.double() + math.log(n)).abs() <= 2 ** -22 * max(1.0, math.log(n))).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("temperature", [0.8, 1.1, 1e30])
@pytest.mark.parametrize("N", [65, 3000])
def test_logits_further_apart_than_any_number(dtype, temperature, N):
    """The largest finite value beside the lowest."""
    x = torch.full((8, N), torch.finfo(TYPES[dtype]).min, dtype=TYPES[dtype], device="cuda")
    x[:, 17] = x[:, 30] = x[:, 60] = torch.finfo(TYPES[dtype]).max
    x[:, 40:50] = 0.0
    u = torch.tensor([0.0, 0.2, 0.4, 0.6, 0.8, 0.9, 0.95, 0.999], device="cuda")
    for kw in (dict(top_p=0.5), dict(top_p=0.3), dict(top_p=0.9), dict(), dict(min_p=0.1), dict(top_k=2), dict(top_k=20, top_p=0.6)):
        r = q.sample_tokens(x, u, temperature=temperature, **kw)
        n = kw.get("top_k", 3) if kw.get("top_k", 3) < 3 else {0.5: 2, 0.3: 1, 0.6: 2}.get(kw.get("top_p"), 3)
        assert r.token.tolist() == [(17, 30, 60)[int(v * n)] for v in u.tolist()], kw
        assert bool(((r.logprob.double() + math.log(n)).abs() <= 2 ** -22 * max(1.0, math.log(n))).all())
