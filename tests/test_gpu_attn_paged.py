"""attn_paged on the GPU against its definition in binary64, with error bounds derived in
_decode_ref.Cache.tolerances.  Every slot of the cache that holds no key of the batch is NaN
(and, int8, has a NaN scale)."""
import math

import pytest
import torch

from tests._decode_ref import DEV, Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import __graft_entry__
    __graft_entry__.build()
    import int8_weight_quantized_int4_gb300 as q
    return q


def check(q, c, window=0, sinks=0, max_new=None, scale=None, **kw):
    ref = c.reference(window, sinks, scale)
    tol, lse_tol = c.tolerances(ref)
    lse = torch.full((c.T, c.Hq), 7.0, device=DEV)
    out, got_lse = q.attn_paged(c.q, *c.args(), max_new=max_new or max(c.news + [1]), window=window, sinks=sinks,
                                scale=scale, lse=lse, **c.kw, **kw)
    assert q.device_error() == 0
    assert got_lse is lse
    err = (out.double() - ref[0]).abs()
    assert bool((err <= tol).all()), (float((err / tol).max()), float(err.max()))
    empty = torch.isinf(ref[1])
    assert torch.equal(torch.isneginf(lse), empty)
    assert bool((out[empty] == 0).all())
    d = (lse.double() - ref[1])[~empty].abs()
    assert bool((d <= lse_tol[~empty]).all()), float((d / lse_tol[~empty]).max())
    return out, lse


HEADS = [("fp16", 256, 24, 4, 16, False), ("bf16", 128, 32, 8, 64, True), ("int8", 256, 24, 4, 16, False),
         ("fp16", 64, 64, 8, 1, False), ("bf16", 256, 8, 8, 48, False), ("int8", 128, 16, 1, 7, False),
         ("int8", 64, 6, 2, 32, False), ("fp16", 128, 40, 10, 33, True), ("bf16", 64, 16, 1, 128, False)]


@pytest.mark.parametrize("kind,d,Hq,Hkv,page,nhd", HEADS)
@pytest.mark.parametrize("lens", [[1], [15], [16], [17], [129], [1003], [0, 1, 2, 63, 64, 65, 300]])
def test_one_token(q, kind, d, Hq, Hkv, page, nhd, lens):
    c = Cache(lens, [min(1, n) for n in lens], Hq, Hkv, d, page, kind, nhd, seed=len(lens) + d)
    check(q, c)


@pytest.mark.parametrize("kind,d,Hq,Hkv,page,nhd", HEADS)
@pytest.mark.parametrize("lens,news", [
    ([5, 77, 300, 9, 18], [5, 3, 6, 1, 2]), ([40, 0, 33], [40, 0, 2]), ([130], [130]), ([700, 10], [9, 10])])
def test_several_tokens(q, kind, d, Hq, Hkv, page, nhd, lens, news):
    c = Cache(lens, news, Hq, Hkv, d, page, kind, nhd, seed=sum(news) + d)
    out, _ = check(q, c)
    # a wrong hint changes the work's split, not the result
    check(q, c, max_new=1)


@pytest.mark.parametrize("kind,d,Hq,Hkv,page,nhd", HEADS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (100, 0), (100, 1), (130, 64), (64, 300), (5000, 4)])
def test_window_and_sinks(q, kind, d, Hq, Hkv, page, nhd, window, sinks):
    c = Cache([1, 100, 101, 260, 777], [1, 3, 1, 2, 4], Hq, Hkv, d, page, kind, nhd, seed=window)
    check(q, c, window, sinks)


@pytest.mark.parametrize("kind,d,Hq,Hkv,page", [("fp16", 256, 24, 4, 16), ("bf16", 128, 8, 2, 64), ("int8", 256, 6, 1, 16),
                                               ("int8", 64, 4, 4, 16), ("fp16", 64, 2, 1, 80)])
def test_long_context_is_split_and_joined(q, kind, d, Hq, Hkv, page):
    """One long sequence over every SM, beside short ones: items cut across CTAs."""
    c = Cache([20011, 3, 70, 1], [1, 1, 2, 1], Hq, Hkv, d, page, kind, seed=3)
    a, la = check(q, c)
    for _ in range(5):                                   # joined in a fixed order: the same bits
        lse = torch.empty_like(la)
        b, lb = q.attn_paged(c.q, *c.args(), max_new=2, lse=lse, **c.kw)
        assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and torch.equal(la, lb)
    check(q, c, window=9000, sinks=500)


@pytest.mark.parametrize("kind,d,G,new", [("bf16", 128, 16, 1), ("fp16", 256, 16, 3), ("int8", 128, 12, 4),
                                          ("fp16", 64, 7, 2), ("int8", 256, 5, 1)])
def test_long_context_of_one_head(q, kind, d, G, new):
    """One KV head over every SM: its parts are joined in groups, and the groups."""
    for n in (2999, 33000):
        c = Cache([n], [new], G, 1, d, 16, kind, seed=n)
        a, la = check(q, c)
        for _ in range(5):
            lse = torch.empty_like(la)
            b, lb = q.attn_paged(c.q, *c.args(), max_new=new, lse=lse, **c.kw)
            assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and torch.equal(la, lb)


@pytest.mark.parametrize("kind,d", [("fp16", 128), ("bf16", 256), ("int8", 64)])
@pytest.mark.parametrize("window", [128, 129, 1 << 30, 2 ** 31 - 2, 2 ** 31 - 1])
def test_windows_past_every_key(q, kind, d, window):
    """A window that reaches every key hides none, however large, also where a sequence has more
    new tokens than positions (those before the first see nothing)."""
    c = Cache([3, 100, 60], [10, 2, 90], 8, 2, d, 16, kind, seed=3)
    a, la = check(q, c, window=window)
    b, lb = check(q, c)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and torch.equal(la, lb)


@pytest.mark.parametrize("past", [2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63 - 1, 2 ** 70])
def test_sizes_past_32_bits(q, past):
    """Sizes that no C int holds count as the largest, not modulo 2^32; negative ones are refused."""
    c = Cache([300, 40], [5, 1], 8, 2, 64, 16, "fp16", seed=3)
    check(q, c, window=past)
    check(q, c, window=past, sinks=past)
    check(q, c, window=7, sinks=past)
    check(q, c, max_new=past)
    for kw in (dict(window=-past), dict(sinks=-past, window=5), dict(max_new=-past)):
        with pytest.raises(q.QgemmError):
            q.attn_paged(c.q, *c.args(), **kw)


def count_case(kind, d, lens, news, Hkv, G, page, seed=0):
    """A batch whose scores are all 0 and whose values count: strip s (16 keys) of a sequence is 1
    in channel s % d of even heads and s // d % d of odd ones, else 0.  Returns (q, args, scales)."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pid = torch.randperm(sum(need) + 2, generator=g).to(DEV)
    act = torch.bfloat16 if kind == "bf16" else torch.float16
    store = torch.int8 if kind == "int8" else act
    v = torch.zeros(sum(need) + 2, Hkv, page, d, dtype=store, device=DEV)
    k = torch.randint(-3, 4, v.shape, device=DEV).to(store)
    table = torch.zeros(len(lens), max(need), dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = pid[at:at + need[b]]
        strip = torch.arange(need[b] * page, device=DEV) // 16
        for h in range(Hkv):
            one = torch.nn.functional.one_hot((strip // d if h % 2 else strip) % d, d).to(store)
            v[pid[at:at + need[b]], h] = one.view(need[b], page, d)
        at += need[b]
    cu = [0]
    for x in news:
        cu.append(cu[-1] + x)
    qq = torch.randn(cu[-1], Hkv * G, d, generator=g).to(act).to(DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    kw = {}
    if kind == "int8":
        kw = {s: torch.full(v.shape[:3], 1.0, device=DEV) for s in ("k_scale", "v_scale")}
    return qq, (k, v, table, torch.tensor(lens, **i32), torch.tensor(cu, **i32)), kw


@pytest.mark.parametrize("kind,d,Hkv,G,new", [("bf16", 128, 2, 8, 1), ("fp16", 256, 4, 6, 1), ("fp16", 256, 2, 6, 6),
                                              ("int8", 256, 2, 6, 1), ("int8", 128, 2, 9, 7), ("fp16", 64, 2, 16, 4)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (9000, 500)])
def test_every_strip_counts_once(q, kind, d, Hkv, G, new, window, sinks):
    """With scores of 0 every visible key weighs 1 / n.  A strip that is skipped or taken twice
    moves its channel by 16 keys of at most 2060 (n / d or 16 d of them), 2^-8, and the log of the sum by
    16 / n >= 2^-13.  All sums are of whole numbers below 2^24, scaled by powers of two; what rounds is
    the output (u), the quotient and the logarithms (a few 2^-24)."""
    u = torch.finfo(torch.bfloat16 if kind == "bf16" else torch.float16).eps / 2
    for lens in ([20011], [33000], [131071], [20011, 3, 33000, 700, 16], [3001] * 60):
        news = [min(new, n) for n in lens]
        qq, args, kw = count_case(kind, d, lens, news, Hkv, G, 32, seed=len(lens))
        lse = torch.empty(qq.shape[:2], device=DEV)
        out, _ = q.attn_paged(qq, *args, max_new=new, window=window, sinks=sinks, scale=0.0, lse=lse, **kw)
        assert q.device_error() == 0
        t = 0
        for n, m in zip(lens, news):
            for at in range(n - m, n):
                key = torch.arange(at + 1, device=DEV)
                if window:
                    key = key[(key > at - window) | (key < sinks)]
                for h in range(Hkv):
                    c = (key // 16 // d if h % 2 else key // 16) % d
                    want = torch.bincount(c, minlength=d).double() / key.numel()
                    got = out[t, h * G:(h + 1) * G].double()
                    assert bool(((got - want).abs() <= u * want * 1.01 + 2.0 ** -25).all()), (n, at, h)
                ln = torch.tensor(float(key.numel()), dtype=torch.float64).log().item()
                assert float((lse[t].double() - ln).abs().max()) <= 16 * 2.0 ** -24 * (1 + ln), (n, at)
                t += 1


@pytest.mark.parametrize("kind,d,G,new", [("fp16", 256, 6, 1), ("bf16", 128, 4, 13), ("int8", 64, 16, 2), ("int8", 128, 8, 1)])
@pytest.mark.parametrize("extra", [1 << 15, 1 << 18, (1 << 20) - 64])
def test_wide_page_tables(q, kind, d, G, new, extra):
    """Tables that could name up to 2^30 keys: the schedule counts places in larger units."""
    lens = [1 + (i * 37) % 90 for i in range(30)] + [5200, 1, 700]
    news = [min(n, 1 + (i * 5) % new) for i, n in enumerate(lens)]
    c = Cache(lens, news, 2 * G, 2, d, 1024, kind, seed=d + new, extra_pages=extra)
    a, la = check(q, c, max_new=new)
    b, lb = check(q, c, max_new=new)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and torch.equal(la, lb)
    check(q, c, window=300, sinks=3, max_new=new)


@pytest.mark.parametrize("kind,d", [(k, d) for k in ("fp16", "bf16", "int8") for d in (64, 128, 256)])
@pytest.mark.parametrize("G,new", [(6, 1), (4, 4), (5, 13)])
def test_many_sequences(q, kind, d, G, new):
    """More items than a third of the SMs: several CTAs an SM, of 8, 16 and up to 64 columns;
    long and short contexts, so that ranges cut items and hold many."""
    lens = [1 + (i * 37) % 90 for i in range(40)] + [2200, 1, 700]
    news = [min(n, 1 + (i * 5) % new) for i, n in enumerate(lens)]
    c = Cache(lens, news, 2 * G, 2, d, 16 if d == 64 else 48, kind, nhd=d == 128, seed=d + new)
    a, la = check(q, c, max_new=new)
    b, lb = check(q, c, max_new=new)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and torch.equal(la, lb)
    check(q, c, window=70, sinks=3, max_new=new)


@pytest.mark.parametrize("lens", [[700], [3, 900, 0, 45, 2100, 1, 16], [1 + (i * 131) % 700 for i in range(32)]])
def test_short_schedules_repeat(q, lens):
    """Up to 32 sequences, whose schedule one warp makes: every launch lists all its work, so
    rows that were NaN before are the same each time."""
    c = Cache(lens, [min(1, n) for n in lens], 16, 4, 128, 16, "bf16", seed=len(lens))
    want, _ = check(q, c)
    out = torch.empty(100, *want.shape, dtype=want.dtype, device=DEV)
    for _ in range(3):
        out.fill_(float("nan"))
        for o in out:
            q.attn_paged(c.q, *c.args(), out=o)
        assert bool((out.view(torch.int16) == want.contiguous().view(torch.int16)).all())
    assert q.device_error() == 0


def test_many_short_sequences(q):
    """More items than a CTA lists at a time (several lists a CTA)."""
    lens = [1 + (i * 7) % 40 for i in range(1500)]
    c = Cache(lens, [1] * 1500, 16, 8, 64, 16, "fp16", seed=5)
    check(q, c)


@pytest.mark.parametrize("kind", ["fp16", "bf16", "int8"])
def test_large_scores_and_scale(q, kind):
    """Scores that differ by hundreds (the reference moves many times), another scale, and a
    negative one."""
    c = Cache([513, 64], [2, 1], 8, 2, 128, 16, kind, seed=8)
    c.q.mul_(6.0)
    check(q, c, scale=0.5)
    check(q, c, scale=-0.25)
    check(q, c, scale=0.0)


def test_scores_near_the_lowest(q):
    """Every visible score near binary32's lowest value (-1.96 * 2^127 in base 2, the same for
    all keys): the weights are still equal.  Equal scores leave only the rounding of a 16-bit
    output and of binary32 sums."""
    c = Cache([300, 37], [1, 2], 8, 2, 64, 16, "bf16", seed=8)
    c.q.fill_(2.0 ** 60)
    for b, n in enumerate(c.lens_list):
        for j in range(n):
            pid, off = c.row(b, j)
            c.k[pid, :, off] = -2.0 ** 61
            c.k64[pid, :, off] = -2.0 ** 61
    ref = c.reference(scale=1.36)
    out, lse = q.attn_paged(c.q, *c.args(), max_new=2, scale=1.36, lse=torch.empty(c.T, 8, device=DEV), **c.kw)
    assert q.device_error() == 0
    tol = 2.0 ** -9 * ref[0].abs() * (1 + 2.0 ** -6) + 400 * 2.0 ** -24 * ref[3]
    assert bool(((out.double() - ref[0]).abs() <= 2 * tol).all())
    assert bool(((lse.double() / ref[1] - 1).abs() <= 2.0 ** -20).all())


@pytest.mark.parametrize("kind", ["fp16", "int8", "bf16"])
@pytest.mark.parametrize("new", [1, 5])
@pytest.mark.parametrize("gap", [17.5, 18.0, 19.0])
def test_weights_far_below_the_largest_count(q, kind, new, gap):
    """Every 64th key scores `gap` above the others and has a value of 0: the row is what the
    others' weights, e^-gap (2^-25.2 to 2^-27.4), leave of their values.  Per element: scores are
    exact (one product); a weight's rounding u where the type is normal, and where it is not the
    2^-25 of a weight whose largest is at least 2^7, 2^-32 n |v| in all; exponents 2^-22 + 64 steps of
    binary32; one rounding of the output."""
    d, n = 64, 4000
    c = Cache([n], [new], 6, 1, d, 16, kind, seed=1)
    v = torch.randint(1, 101, (n, d), generator=torch.Generator().manual_seed(9)).double().to(DEV)
    v[::64] = 0.0
    key = torch.arange(n, device=DEV)
    pid, off = c.table[0].long()[key // 16], key % 16
    if kind == "int8":
        k8 = torch.zeros(n, d, dtype=torch.int8, device=DEV)
        k8[::64, 0] = 64
        c.k[pid, 0, off], c.v[pid, 0, off] = k8, v.to(torch.int8)
        c.kw["k_scale"][pid, 0, off] = 2.0 ** -6
        c.kw["v_scale"][pid, 0, off] = 1.0
    else:
        c.k[pid, 0, off] = 0.0
        c.k[pid[::64], 0, off[::64], 0] = 1.0
        c.v[pid, 0, off] = v.to(c.act)
    c.q.zero_()
    c.q[:, :, 0] = gap
    out = q.attn_paged(c.q, *c.args(), max_new=new, scale=1.0, **c.kw).double()
    assert q.device_error() == 0
    u, e = torch.finfo(c.act).eps / 2, 2.0 ** -24
    for t in range(new):
        m = n - new + t + 1
        p = torch.where(key[:m] % 64 == 0, 1.0, math.exp(-gap)).double()
        p /= p.sum()
        want = p @ v[:m]
        tol = (2 * u + 2.0 ** -20 + 128 * e) * want + m * 2.0 ** -32 * 100 / (m // 64)
        if c.act == torch.float16:
            tol = tol + 2.0 ** -25
        assert bool(((out[t] - want).abs() <= tol).all()), (t, float(out[t, 0, 0]), float(want[0]))


@pytest.mark.parametrize("kind", ["fp16", "bf16", "int8"])
@pytest.mark.parametrize("d,G,new", [(64, 6, 1), (128, 8, 2), (256, 8, 1), (256, 6, 2), (128, 16, 2), (64, 16, 4)])
def test_weights_of_opposite_values(q, kind, d, G, new):
    """Two keys with values A and -A and scores that differ by a little (exactly, one product):
    A tanh of half the difference, 0 to 13 % of A.  What the weights lose shows beside
    that: two terms of 16 bits hold a weight to u^2 of itself, exponents, sums and the quotient
    2^-20 of A, and one rounding of the output.  With several tokens a later one's infinite
    value lies in the strip (16-bit caches), which then is summed key by key."""
    A = 1016.0
    n = new + 1
    c = Cache([n], [new], 2 * G, 2, d, 16, kind, seed=1)
    pid = int(c.table[0, 0])
    one = 64 if kind == "int8" else 1
    c.k[pid, :, :n], c.v[pid, :, :n] = 0, 0
    c.k[pid, :, 0, 0] = one
    c.v[pid, :, 0], c.v[pid, :, 1] = (127, -127) if kind == "int8" else (A, -A)
    if kind == "int8":
        c.kw["k_scale"][pid], c.kw["v_scale"][pid] = 2.0 ** -6, 8.0
    elif new > 1:
        c.v[pid, :, 2:n] = float("inf")
    c.q.zero_()
    delta = torch.arange(c.T * 2 * G, device=DEV).view(c.T, 2 * G).double() % 64 / 256
    c.q[:, :, 0] = delta.to(c.act)
    out = q.attn_paged(c.q, *c.args(), max_new=new, scale=1.0, **c.kw).double()
    assert q.device_error() == 0
    want = (A * torch.tanh(delta / 2))[:, :, None]
    u = torch.finfo(c.act).eps / 2
    tol = A * (u * u + 2.0 ** -20) + u * want * (1 + 2.0 ** -6)
    assert bool(((out[0] - want[0]).abs() <= tol[0]).all()), float(((out[0] - want[0]).abs() / tol[0]).max())
    # later tokens: further keys of value 0 and score 0 (int8), or the infinity they see
    for t in range(1, new):
        if kind == "int8":
            w = torch.exp(delta[t])
            w = (A * (w - 1) / (w + 1 + t))[:, None]
            assert bool(((out[t] - w).abs() <= A * (u * u + 2.0 ** -20) + u * w.abs() * (1 + 2.0 ** -6)).all())
        else:
            assert not bool(torch.isfinite(out[t]).any())


@pytest.mark.parametrize("v_scale", [2.0 ** -13, 2.0 ** 8])
def test_int8_values_of_any_size(q, v_scale):
    """The weight carries the value's scale: small scales must not lose its bits."""
    c = Cache([700], [1], 8, 2, 128, 16, "int8", seed=4, v_scale=v_scale)
    check(q, c)


def test_zero_scale_rows(q):
    c = Cache([50, 3], [1, 1], 4, 2, 64, 16, "int8", seed=4)
    for b, j in ((0, 7), (0, 49), (1, 0), (1, 1), (1, 2)):
        pid, off = c.row(b, j)
        for s, x in ((c.kw["k_scale"], c.k64), (c.kw["v_scale"], c.v64)):
            s[pid, :, off] = 0.0
            x[pid, :, off] = 0.0
    check(q, c)


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_hidden_values_never_reach_a_row(q, kind, value):
    """A key that one new token sees and another does not (a later token; a key that leaves
    the window between them) may hold anything: only the rows that see it are affected."""
    for window, sinks, hidden, sees in ((0, 0, 59, lambda t: t == 4), (20, 0, 36, lambda t: t == 0),
                                        (20, 2, 37, lambda t: t <= 1)):
        c = Cache([60], [5], 12, 2, 128, 16, kind, seed=2)
        pid, off = c.row(0, hidden)
        clean = c.reference(window, sinks)
        tol, _ = c.tolerances(clean)
        c.v[pid, 0, off, 10:14] = value
        c.k[pid, 1, off, 3] = value
        out = q.attn_paged(c.q, *c.args(), max_new=5, window=window, sinks=sinks)
        assert q.device_error() == 0
        for t in range(5):
            if not sees(t):
                assert bool(((out[t].double() - clean[0][t]).abs() <= tol[t]).all()), (window, t)
            else:
                assert not bool(torch.isfinite(out[t, :6, 10:14]).any())


@pytest.mark.parametrize("kind,d", [("fp16", 64), ("bf16", 128), ("fp16", 256), ("bf16", 256)])
@pytest.mark.parametrize("G,new", [(16, 2), (16, 4), (32, 2), (6, 3), (6, 6), (8, 3), (8, 5), (12, 2), (64, 3)])
def test_hidden_values_of_other_blocks(q, kind, d, G, new):
    """Columns in blocks of 16: a block that lies in one token shares its strips with blocks of
    other tokens, whose keys it does not see.  Every key that some token does not see holds an
    infinity or a NaN in turn; the rows that do not see it stay as they were."""
    n, window = 70, 37
    for win, sinks in ((0, 0), (window, 0), (window, 2)):
        c = Cache([n, 33], [new, 1], 2 * G, 2, d, 16, kind, seed=G + new)
        clean = c.reference(win, sinks)
        tol, _ = c.tolerances(clean)
        first = n - new                                      # position of the first new token
        keys = list(range(first + 1, n)) + ([j for j in range(first - win + 1, n - win)] if win else [])
        for i, j in enumerate(keys):
            pid, off = c.row(0, j)
            kept = c.v[pid, :, off].clone()
            c.v[pid, :, off, 5:9] = (float("inf"), float("nan"), float("-inf"))[i % 3]
            out = q.attn_paged(c.q, *c.args(), max_new=new, window=win, sinks=sinks)
            c.v[pid, :, off] = kept
            for t in range(new):
                at = first + t
                if j <= at and (not win or j > at - win or j < sinks):
                    assert not bool(torch.isfinite(out[t, :, 5:9]).any())
                else:
                    assert bool(((out[t].double() - clean[0][t]).abs() <= tol[t]).all()), (win, j, t)
            assert bool(((out[new:].double() - clean[0][new:]).abs() <= tol[new:]).all())
    assert q.device_error() == 0


def test_int8_hidden_scales(q):
    c = Cache([60], [5], 4, 1, 64, 16, "int8", seed=2)
    clean = c.reference()
    tol, _ = c.tolerances(clean)
    pid, off = c.row(0, 59)
    c.kw["k_scale"][pid, 0, off] = float("nan")
    c.kw["v_scale"][pid, 0, off] = float("inf")
    out = q.attn_paged(c.q, *c.args(), max_new=5, **c.kw)
    assert bool(((out[:4].double() - clean[0][:4]).abs() <= tol[:4]).all())


def test_shared_prefix_pages(q):
    c = Cache([64, 64], [1, 1], 8, 2, 64, 16, "fp16", seed=6)
    c.table[1, :3] = c.table[0, :3]
    check(q, c)


def test_bad_pages_and_lengths(q):
    """A page id out of range reads as zeros, a length past the table as the table's end."""
    c = Cache([60, 40], [1, 1], 4, 2, 64, 16, "fp16", seed=6)
    good = c.table.clone()
    c.table[0, 1], c.table[1, 2] = c.k.shape[0], -5
    out = q.attn_paged(c.q, *c.args())
    assert q.device_error() == q.QW_ERR_BAD_INDEX and q.device_error() == 0
    zero = int(c.k.shape[0] - 1)
    used = set(good.flatten().tolist())
    zero = next(p for p in range(c.k.shape[0]) if p not in used)
    c.k[zero], c.v[zero] = 0.0, 0.0
    c.k64[zero], c.v64[zero] = 0.0, 0.0
    c.table[0, 1], c.table[1, 2] = zero, zero
    ref = c.reference()
    tol, _ = c.tolerances(ref)
    assert bool(((out.double() - ref[0]).abs() <= tol).all())
    c = Cache([64], [1], 4, 2, 64, 16, "fp16", seed=6)
    want = q.attn_paged(c.q, *c.args())
    c.lens[0] = 1 << 30
    got = q.attn_paged(c.q, *c.args())
    assert q.device_error() == q.QW_ERR_BAD_INDEX and torch.equal(got, want)


def test_offsets_out_of_order(q):
    """Offsets beyond q or descending: clamped, reported, nothing read or written outside."""
    c = Cache([40, 40, 40], [1, 1, 1], 4, 2, 64, 16, "fp16", seed=6)
    c.cu.copy_(torch.tensor([0, 900, -3, 2], device=DEV))
    out = torch.full_like(c.q, 3.0).contiguous()
    q.attn_paged(c.q, *c.args(), out=out)
    assert q.device_error() == q.QW_ERR_BAD_INDEX


@pytest.mark.parametrize("cu,left", [([1, 3, 2, 4], [0, 4, 5]), ([-7, 1, 1, 2], [2, 3, 4, 5]),
                                     ([5, 900, 900, 900], [0, 1, 2, 3, 4]), ([6, -2, -2, 0], [0, 1, 2, 3, 4, 5])])
def test_offsets_stay_inside(q, cu, left):
    """Offsets that descend or leave 0 .. T write no row outside q's nor one of no sequence."""
    c = Cache([40, 40, 40], [2, 2, 2], 4, 2, 64, 16, "fp16", seed=6)
    c.cu.copy_(torch.tensor(cu, device=DEV))
    big = torch.full((c.T + 16, 4, 64), 3.0, dtype=torch.float16, device=DEV)
    lse = torch.full((c.T + 16, 4), 3.0, device=DEV)
    q.attn_paged(c.q, *c.args(), max_new=2, out=big[8:8 + c.T], lse=lse[8:8 + c.T])
    assert q.device_error() == q.QW_ERR_BAD_INDEX and q.device_error() == 0
    keep = torch.ones(c.T + 16, dtype=torch.bool, device=DEV)
    keep[8:8 + c.T] = False
    keep[[8 + t for t in left]] = True
    assert bool((big[keep] == 3.0).all()) and bool((lse[keep] == 3.0).all())
    assert bool(torch.isfinite(big.float()).all()) and not bool((big[~keep] == 3.0).any())


def test_overlapping_offsets_past_2_to_31_places(q):
    """Offsets that descend can name each token many times: 128 sequences of all 4096 tokens, 64
    heads and 4096 strips would be 17 * 2^30 places.  Nothing is computed, and the next call,
    with the same workspace, is right."""
    i32 = dict(dtype=torch.int32, device=DEV)
    T, H, B = 4096, 64, 256
    k = torch.randn(1, H, 1024, 64, device=DEV).half()
    table = torch.zeros(B, 64, **i32)
    lens = torch.full((B,), 65536, **i32)
    cu = torch.tensor([0, T] * (B // 2) + [0], **i32)
    qq = torch.randn(T, H, 64, device=DEV).half()
    ws = q.Workspace(torch.device("cuda:0"))
    out = torch.full_like(qq, 3.0)
    q.attn_paged(qq, k, k, table, lens, cu, out=out, ws=ws)
    assert q.device_error() == q.QW_ERR_BAD_INDEX and bool((out == 3.0).all())
    c = Cache([40, 3000], [1, 1], 64, 64, 64, 16, "fp16", seed=6)
    check(q, c, ws=ws)


def test_rows_of_no_sequence_are_left(q):
    c = Cache([30, 30], [1, 1], 4, 2, 64, 16, "fp16", seed=6)
    c.cu[2] = 1
    out = torch.full(c.q.shape, 3.0, dtype=torch.float16, device=DEV)
    q.attn_paged(c.q, *c.args(), out=out)
    assert q.device_error() == 0 and bool((out[1] == 3.0).all()) and not bool((out[0] == 3.0).all())


def test_graph_follows_lengths(q):
    """A captured step replays with longer contexts: lengths are read on the device."""
    c = Cache([400, 900], [1, 1], 24, 4, 256, 16, "fp16", seed=9)
    ws = q.Workspace(torch.device("cuda:0"))
    out = torch.empty(c.q.shape, dtype=torch.float16, device=DEV)
    q.attn_paged(c.q, *c.args(), out=out, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.attn_paged(c.q, *c.args(), out=out, ws=ws)
    for lens in ([1, 900], [400, 17], [333, 801]):
        c.lens_list = lens
        c.lens.copy_(torch.tensor(lens))
        g.replay()
        torch.cuda.synchronize()
        ref = c.reference()
        tol, _ = c.tolerances(ref)
        assert bool(((out.double() - ref[0]).abs() <= tol).all())
    assert q.device_error() == 0


def test_another_stream(q):
    c = Cache([500, 20], [1, 1], 24, 4, 256, 16, "fp16", seed=9)
    want = q.attn_paged(c.q, *c.args())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = q.attn_paged(c.q, *c.args())
    s.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("kind", ["fp16", "int8"])
@pytest.mark.parametrize("dim", [0, 1, 2])
def test_strides_of_extents_of_one_mean_nothing(q, kind, dim):
    """A dimension of one element may have any stride, in K another than in V."""
    shape = [(1, 2, 16), (5, 1, 16), (20, 2, 1)][dim]
    pages, Hkv, page = shape
    n = min(pages * page, 16)
    c = Cache([n], [1], 4 * Hkv, Hkv, 64, page, kind, seed=dim, spare=pages - -(-n // page))
    assert tuple(c.k.shape[:3]) == shape
    want = q.attn_paged(c.q, *c.args(), **c.kw)
    odd = [list(c.k.stride()) for _ in range(2)]
    odd[0][dim], odd[1][dim] = 7, 3

    def restride(x, st):
        return x.as_strided(x.shape, st)
    k, v = restride(c.k, odd[0]), restride(c.v, odd[1])
    qq = c.q.as_strided(c.q.shape, (5, 64, 1))                       # one token
    got = q.attn_paged(qq, k, v, *c.args()[2:], **c.kw)
    assert torch.equal(got, want)
    new = torch.randn(1, Hkv, 64, device=DEV).half()
    for x, y in ((c.k, c.v), (k, v)):
        q.kv_append(new if x is c.k else new.as_strided(new.shape, (3, 64, 1)), new, x, y, *c.args()[2:], **c.kw)
        pid, off = c.row(0, n - 1)
        if kind == "fp16":
            assert torch.equal(c.k[pid, :, off], new[0]) and torch.equal(c.v[pid, :, off], new[0])
        c.k[pid, :, off] = 0
    # copies: one layer, or one page
    pool = torch.randn(1, 4, 2, 8, 64, device=DEV).half()
    want = pool.clone()
    want[:, 2] = want[:, 1]
    pairs = torch.tensor([[1, 2]], dtype=torch.int32, device=DEV)
    q.kv_copy_pages(pairs, pool.as_strided(pool.shape, (1, *pool.stride()[1:])))
    assert torch.equal(pool, want)
    one = pool[:, :1].as_strided((1, 1, 2, 8, 64), (1, 1, *pool.stride()[2:]))
    q.kv_copy_pages(torch.zeros(1, 2, dtype=torch.int32, device=DEV), one)
    assert torch.equal(pool, want) and q.device_error() == 0


@pytest.mark.parametrize("d,new,ctas", [(64, 1, 4), (128, 1, 4), (256, 1, 2), (64, 2, 4), (128, 2, 2), (256, 2, 1)])
def test_workspace_is_what_the_launch_can_use(q, d, new, ctas):
    """Two partial sums (m, l and d channels a column) for each CTA that the widest launch has."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    cols = 8 if new == 1 else 64
    want = 12288 + 2 * ctas * sms * cols * (d + 2) * 4
    assert q.lib().attn_paged_workspace_bytes(d, 12, 2, new) == want


def test_binding_refusals(q):
    c = Cache([20], [1], 4, 2, 64, 16, "fp16")
    a = c.args()
    with pytest.raises(TypeError):
        q.attn_paged(c.q.bfloat16(), *a)
    with pytest.raises(ValueError):
        q.attn_paged(c.q[..., :32], *a)
    with pytest.raises(ValueError):
        q.attn_paged(c.q, c.k, c.v[:, :, :8], *a[2:])
    with pytest.raises(ValueError):
        q.attn_paged(c.q, c.k, c.v, a[2].long(), *a[3:])
    with pytest.raises(ValueError):
        q.attn_paged(c.q, c.k, c.v, a[2], a[3], a[4][:1])
    with pytest.raises(ValueError):
        q.attn_paged(c.q, *a, k_scale=torch.zeros(1, device=DEV))
    with pytest.raises(ValueError):
        q.attn_paged(c.q, *a, out=torch.empty(1, 4, 64, device=DEV))
    with pytest.raises(ValueError):
        q.attn_paged(c.q, *a, lse=torch.empty(1, 3, device=DEV))
    with pytest.raises(q.QgemmError):
        q.attn_paged(c.q[:, :3].contiguous(), *a)           # 2 KV heads do not divide 3
    with pytest.raises(q.QgemmError):
        q.attn_paged(c.q, *a, window=-1)
    T0 = q.attn_paged(c.q[:0], c.k, c.v, a[2], a[3], torch.zeros_like(a[4]))
    assert T0.shape == (0, 4, 64) and q.device_error() == 0
