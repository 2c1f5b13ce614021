"""attn_tree against its definition in binary64.  Every slot of the cache that holds no key of the
batch is NaN (int8: with a NaN scale)."""
import math

import numpy as np
import pytest
import torch

import int8_weight_quantized_int4_gb300 as q
from tests import _tree_ref as ref
from tests._decode_ref import DEV, Cache

pytestmark = pytest.mark.gpu


class Case(Cache):
    def __init__(self, lens, news, Hq, Hkv, d, page, kind="fp16", nhd=False, seed=0, spread=6, roots=1, **kw):
        super().__init__(lens, news, Hq, Hkv, d, page, kind, nhd, seed, **kw)
        rng = np.random.default_rng(seed)
        self.trees = [ref.tree(rng, m, spread, roots) for m in news]
        self.parents = torch.tensor([p for t in self.trees for p in t], dtype=torch.int32, device=DEV)

    def see(self, b, window, sinks):
        """[nodes, len]: what each node of sequence b sees."""
        n, m = self.lens_list[b], self.news[b]
        see, s, keys = np.zeros((m, max(n, 0)), bool), n - m, np.arange(n)
        for r in range(m):
            line = ref.ancestors(self.trees[b], r)
            pos = s + len(line) - 1
            see[r] = (keys < s) & ((keys > pos - window) | (keys < sinks) if window else True)
            for e, i in enumerate(line):
                if s + i >= 0 and (not window or s + e > pos - window or s + e < sinks):
                    see[r, s + i] = True
        return torch.from_numpy(see).to(DEV)

    def reference(self, window=0, sinks=0, scale=None):
        """(out, lse, bound of |x| terms per row, sum p |v|, largest |v|), as Cache.reference."""
        s = 1.0 / math.sqrt(self.d) if scale is None else scale
        G, T, H = self.Hq // self.Hkv, self.T, self.Hkv
        out = torch.zeros(T, self.Hq, self.d, dtype=torch.float64, device=DEV)
        mag, vmax = out.clone(), out.clone()
        lse = torch.full((T, self.Hq), -math.inf, dtype=torch.float64, device=DEV)
        dx = torch.zeros(T, self.Hq, dtype=torch.float64, device=DEV)
        t = 0
        for b, (n, m) in enumerate(zip(self.lens_list, self.news)):
            if n == 0 or m == 0:
                t += m
                continue
            see = self.see(b, window, sinks)
            j = torch.arange(n, device=DEV)
            pid, off = self.table[b].long()[j // self.page], j % self.page
            k, v = self.k64[pid, :, off], self.v64[pid, :, off]
            hidden = ~see.any(0)
            k, v = k.clone(), v.clone()
            k[hidden], v[hidden] = 0, 0
            qq = self.q[t:t + m].double().view(m, H, G, self.d)
            x = torch.einsum("rhgd,khd->rhgk", qq, k) * s
            x = x.masked_fill(~see[:, None, None], -math.inf)
            none = ~see.any(1)
            p = torch.softmax(x, -1)
            p[none] = 0
            clean = v.nan_to_num(0, 0, 0)
            out[t:t + m] = torch.einsum("rhgk,khd->rhgd", p, clean).reshape(m, self.Hq, self.d)
            mag[t:t + m] = torch.einsum("rhgk,khd->rhgd", p, clean.abs()).reshape(m, self.Hq, self.d)
            vmax[t:t + m] = clean.abs().amax(0)[None, :, None].expand(m, H, G, self.d).reshape(m, self.Hq, self.d)
            lse[t:t + m] = torch.logsumexp(x, -1).flatten(1)
            bound = torch.einsum("rhgd,khd->rhgk", qq.abs(), k.abs()).masked_fill(~see[:, None, None], 0)
            dx[t:t + m] = (bound.amax(-1) * abs(s)).flatten(1)
            t += m
        return out, lse, dx, mag, vmax

    def tolerances(self, r):
        """Elementwise bounds of out's and lse's error; e = 2^-24, u half a step of the output.
          score: d products summed in binary32 (up to 2 e a step, the tensor core may truncate),
            times the scale (int8: scales): (2 d + 8) e sum |q k| scale
          weight: that, ex2's 2^-22, and what its two 16-bit terms leave: 2^-22 (bf16 2^-16); fp16
            also 2^-32 of the largest, absolutely
          sums: up to 2 e a step over n keys in steps of 16, parts joined: (n / 8 + 64) e
          out: the weights' relative error times p |v| and again in the denominator; one rounding."""
        out, lse, dx, mag, vmax = r
        u = torch.finfo(self.act).eps / 2
        e, n = 2.0 ** -24, max(self.lens_list + [1])
        w = (2 * self.d + 8) * e * dx + 2.0 ** -22 + (n / 8 + 64) * e
        term = 2.0 ** -16 if self.act == torch.bfloat16 else 2.0 ** -22
        tol = (term + 2 * w)[..., None] * mag + u * out.abs() * (1 + 2.0 ** -6)
        if self.act == torch.float16:
            tol = tol + n * 2.0 ** -32 * vmax + 2.0 ** -25
        return tol, w + 8 * e * torch.where(lse.isinf(), 0.0, lse.abs())


def run(c, window=0, sinks=0, scale=None, **kw):
    lse = torch.full((c.T, c.Hq), 7.0, device=DEV)
    kw.setdefault("max_nodes", max(c.news + [1]))
    return q.attn_tree(c.q, *c.args(), c.parents, window=window, sinks=sinks, scale=scale, lse=lse, **c.kw, **kw)


def check(c, window=0, sinks=0, scale=None, **kw):
    r = c.reference(window, sinks, scale)
    tol, lse_tol = c.tolerances(r)
    out, lse = run(c, window, sinks, scale, **kw)
    assert q.device_error() == 0
    err = (out.double() - r[0]).abs()
    assert bool((err <= tol).all()), (float((err / tol).nan_to_num(1e9).max()), float(err.max()))
    empty = torch.isinf(r[1])
    assert torch.equal(torch.isneginf(lse), empty)
    assert bool((out[empty] == 0).all())
    d = (lse.double() - r[1])[~empty].abs()
    assert bool((d <= lse_tol[~empty]).all()), float((d / lse_tol[~empty]).max())
    return out, lse


def same(a, b):
    return torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


SHAPES = [("fp16", 128, 16, 4, 16, False), ("fp16", 256, 24, 4, 16, False), ("bf16", 128, 32, 8, 64, True),
          ("int8", 256, 24, 4, 16, False), ("fp16", 64, 64, 8, 1, False), ("bf16", 256, 8, 8, 48, False),
          ("int8", 128, 16, 1, 7, False), ("int8", 64, 6, 2, 32, True), ("fp16", 128, 40, 10, 33, True), ("bf16", 128, 160, 1, 16, False), ("fp16", 64, 100, 2, 8, True),
          ("bf16", 64, 16, 1, 128, False)]


@pytest.mark.parametrize("kind,d,Hq,Hkv,page,nhd", SHAPES)
@pytest.mark.parametrize("lens,news", [([1], [1]), ([64], [1]), ([65], [7]), ([129, 1], [30, 1]), ([1003], [12]),
                                       ([0, 1, 2, 63, 64, 65, 300, 20], [0, 1, 2, 3, 64, 1, 33, 20]), ([500], [256])])
def test_trees(kind, d, Hq, Hkv, page, nhd, lens, news):
    check(Case(lens, news, Hq, Hkv, d, page, kind, nhd, seed=len(lens) + d + sum(news)))


@pytest.mark.parametrize("kind,d,Hq,Hkv,page,nhd", SHAPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (3, 70), (16, 4), (100, 0), (130, 64), (64, 300), (5000, 4)])
def test_window_and_sinks(kind, d, Hq, Hkv, page, nhd, window, sinks):
    c = Case([1, 100, 101, 260, 777, 30], [1, 13, 40, 2, 64, 30], Hq, Hkv, d, page, kind, nhd, seed=window, spread=2)
    check(c, window, sinks)


@pytest.mark.parametrize("kind,d,Hq,Hkv,page", [("fp16", 256, 24, 4, 16), ("bf16", 128, 8, 2, 64), ("int8", 256, 6, 1, 16),
                                                ("int8", 64, 4, 4, 16), ("fp16", 64, 2, 1, 80), ("int8", 128, 24, 4, 16)])
def test_long_contexts_are_split_and_joined(kind, d, Hq, Hkv, page):
    c = Case([20011, 3, 70, 1, 6000], [33, 1, 20, 1, 64], Hq, Hkv, d, page, kind, seed=3)
    a = check(c)
    for _ in range(5):                                   # joined in a fixed order: the same bits
        assert same(a, run(c))
    check(c, window=9000, sinks=500)


def test_many_sequences():
    """More segments a CTA than are listed at a time."""
    rng = np.random.default_rng(1)
    lens = [int(rng.integers(1, 90)) for _ in range(700)]
    news = [int(rng.integers(0, min(n, 5) + 1)) for n in lens]
    check(Case(lens, news, 32, 32, 64, 16, "bf16", seed=2))
    check(Case(lens, news, 16, 16, 128, 16, "int8", seed=2))
    check(Case(lens, news, 8, 8, 256, 16, "fp16", seed=2))


@pytest.mark.parametrize("kind,d", [("fp16", 256), ("bf16", 128), ("int8", 64)])
def test_a_chain_is_attn_paged(kind, d):
    c = Case([300, 77, 900], [9, 1, 30], 16, 4, d, 16, kind, seed=5, spread=1)
    a, la = check(c)
    b, lb = q.attn_paged(c.q, *c.args(), max_new=30, lse=torch.empty_like(la), **c.kw)
    tol, lse_tol = c.tolerances(c.reference())
    assert bool(((a.double() - b.double()).abs() <= 2 * tol).all()) and bool(((la - lb).abs() <= 2 * lse_tol).all())


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_hidden_values_that_are_not_finite(kind, d):
    """A node's value is infinite or NaN: only the rows that see it are not finite."""
    for lens, news in (([200, 90], [40, 30]), ([30], [30]), ([64 + 17], [17])):
        c = Case(lens, news, 8, 2, d, 16, kind, seed=7)
        clean = c.reference()
        tol, _ = c.tolerances(clean)
        t = 0
        hurt = torch.zeros(c.T, dtype=torch.bool, device=DEV)
        for b, (n, m) in enumerate(zip(lens, news)):
            for i, v in ((3, float("nan")), (m - 2, float("inf")), (m - 1, float("-inf"))):
                p, r = c.row(b, n - m + i)
                c.v[p, :, r] = v
                hurt[t:t + m] |= c.see(b, 0, 0)[:, n - m + i]
            t += m
        out, lse = run(c)
        assert q.device_error() == 0
        assert bool(hurt.any()) and bool((~hurt).any())
        err = (out.double() - clean[0]).abs()
        assert bool((err <= tol)[~hurt].all())
        assert not bool(torch.isfinite(out[hurt]).any())
        assert bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("kind", ["fp16", "bf16", "int8"])
def test_hidden_keys_that_are_not_finite(kind):
    c = Case([200, 90], [40, 30], 8, 2, 128, 16, kind, seed=8)
    clean = c.reference()
    tol, _ = c.tolerances(clean)
    hurt, t = torch.zeros(c.T, dtype=torch.bool, device=DEV), 0
    for b, (n, m) in enumerate(zip(c.lens_list, c.news)):
        p, r = c.row(b, n - 1)
        if kind == "int8":
            c.kw["k_scale"][p, :, r] = float("nan")
            c.kw["v_scale"][p, :, r] = float("nan")
        else:
            c.k[p, :, r] = float("nan")
        hurt[t:t + m] |= c.see(b, 0, 0)[:, n - 1]
        t += m
    out, _ = run(c)
    assert bool(((out.double() - clean[0]).abs() <= tol)[~hurt].all()) and bool(out[hurt].isnan().all())


def test_windowed_values_that_are_not_finite():
    """Keys that some nodes' windows have left are infinite."""
    c = Case([400], [20], 8, 2, 128, 16, "fp16", seed=9, spread=1)       # a chain: positions differ by the node
    clean = c.reference(50, 4)
    tol, _ = c.tolerances(clean)
    j = 400 - 20 - 50 + 6                                                 # seen by nodes 0 .. 5
    p, r = c.row(0, j)
    c.v[p, :, r] = float("inf")
    see = c.see(0, 50, 4)[:, j]
    out, _ = run(c, 50, 4)
    assert int(see.sum()) == 6
    assert bool(((out.double() - clean[0]).abs() <= tol)[~see].all()) and not bool(torch.isfinite(out[see]).any())


@pytest.mark.parametrize("kind", ["fp16", "bf16", "int8"])
def test_opposite_values_and_extreme_scores(kind):
    c = Case([900, 40], [20, 40], 8, 2, 128, 16, kind, seed=10, v_scale=1e-2 if kind == "int8" else 1.0)
    for scale in (0.0, -0.05, 3.0, 1e-6):
        check(c, scale=scale)
    if kind == "int8":                                                    # rows of zeros have scale 0
        c.kw["v_scale"][c.table[1, 0].long()] = 0.0
        c.vs[int(c.table[1, 0])] = 0.0
        c.v64[int(c.table[1, 0])] = 0.0
        check(c)
        c.kw["v_scale"].mul_(2.0 ** -20)
        c.v64.mul_(2.0 ** -20)
        r = c.reference()
        out, _ = run(c)
        tol, _ = c.tolerances(r)
        assert bool(((out.double() - r[0]).abs() <= tol).all())


def test_rows_of_no_sequence_and_hints():
    c = Case([100, 50], [10, 5], 8, 2, 128, 16, "fp16", seed=11)
    a = run(c)
    assert same(a, run(c, max_nodes=256))
    pad = torch.zeros(20, *c.qkv.shape[1:], dtype=c.act, device=DEV)
    pad[2:17] = c.qkv
    cu = c.cu + 2
    out = torch.full((20, 8, 128), 5.0, dtype=c.act, device=DEV)
    lse = torch.full((20, 8), 5.0, device=DEV)
    parents = torch.full((20,), 99, dtype=torch.int32, device=DEV)
    parents[2:17] = c.parents
    q.attn_tree(pad[:, :8], c.k, c.v, c.table, c.lens, cu, parents, out=out, lse=lse)
    assert q.device_error() == 0
    assert torch.equal(out[2:17], a[0]) and torch.equal(lse[2:17], a[1])
    assert bool((out[:2] == 5).all()) and bool((out[17:] == 5).all()) and bool((lse[:2] == 5).all())


def test_bad_parents_pages_and_lengths():
    c = Case([100, 50], [10, 5], 8, 2, 128, 16, "fp16", seed=12)
    good = run(c)
    c.parents[12] = 7                                                     # node 2 of the second: not an earlier one
    c.trees[1][2] = -1
    out, _ = run(c)
    assert q.device_error() == q.QW_ERR_BAD_INDEX
    r = c.reference()
    assert bool(((out.double() - r[0]).abs() <= c.tolerances(r)[0]).all())
    assert torch.equal(out[:10], good[0][:10])
    c = Case([100, 50], [10, 5], 8, 2, 128, 16, "fp16", seed=12)
    run(c, max_nodes=9)                                                   # the first has 10
    assert q.device_error() == q.QW_ERR_BAD_INDEX
    out, lse = run(c, max_nodes=9)
    assert bool((out[:10] == 0).all()) and bool(torch.isneginf(lse[:10]).all()) and torch.equal(out[10:], good[0][10:])
    q.device_error()
    c.table[0, 2] = 1 << 20                                               # a page outside the pool: rows of zeros
    out, lse = run(c)
    assert q.device_error() == q.QW_ERR_BAD_INDEX and bool(torch.isfinite(out).all()) and torch.equal(out[10:], good[0][10:])
    c.table[0, 2] = -1
    run(c)
    assert q.device_error() == q.QW_ERR_BAD_INDEX
    c = Case([100, 50], [10, 5], 8, 2, 128, 16, "fp16", seed=12)
    c.lens[1] = 4000
    run(c)
    assert q.device_error() == q.QW_ERR_BAD_INDEX


def test_pages_outside_the_window_are_not_read():
    c = Case([900], [10], 8, 2, 128, 16, "fp16", seed=13)
    a = check(c, 100, 4)
    c.table[0, 2:49] = -1                                                 # slots 32 .. 783; the window starts at 791
    b = run(c, 100, 4)
    assert q.device_error() == 0 and same(a, b)


def test_fewer_positions_than_nodes():
    """Nodes before the first position have no slot; others see what there is."""
    check(Case([3, 100, 60], [10, 2, 90], 8, 2, 128, 16, "bf16", seed=14))


@pytest.mark.parametrize("kind", ["fp16", "int8"])
def test_padded_strides_and_no_pages(kind):
    """Rows, heads and pages any multiple of 16 bytes apart; a cache of one page, and of none."""
    c = Case([300, 40], [20, 9], 8, 2, 128, 16, kind, seed=21)
    want = run(c)
    for pad in ((0, 0, 16), (0, 3, 0), (2, 0, 48), (1, 5, 16)):
        shape = [n + p for n, p in zip(c.k.shape[1:], pad)]
        both = torch.full((2, c.k.shape[0], *shape), 7, dtype=c.k.dtype, device=DEV)
        k, v = (x[:, :2, :16, :128] for x in both)
        k.copy_(c.k)
        v.copy_(c.v)
        assert same(want, (q.attn_tree(c.q, k, v, *c.args()[2:], c.parents, lse=torch.empty_like(want[1]), **c.kw)))
    one = Case([16], [5], 8, 2, 64, 16, kind, seed=22, spare=0)
    assert one.k.shape[0] == 1
    check(one)
    e = {n: v[:0] for n, v in c.kw.items()}
    out, lse = q.attn_tree(c.q, c.k[:0], c.v[:0], *c.args()[2:], c.parents, lse=torch.empty_like(want[1]), **e)
    assert q.device_error() == q.QW_ERR_BAD_INDEX and bool((out == 0).all())


def test_streams_graphs_and_workspaces():
    c = Case([5000, 700], [30, 64], 24, 4, 256, 16, "fp16", seed=15)
    want = run(c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = run(c)
    side.synchronize()
    assert same(want, other)
    ws = q.Workspace()
    assert same(want, run(c, ws=ws))
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.attn_tree(c.q, *c.args(), c.parents, max_nodes=64, out=out, lse=lse, ws=ws, **c.kw)
    for _ in range(3):
        out.zero_()
        g.replay()
        assert same(want, (out, lse))
    c.lens -= 60                                                          # the graph follows lengths that change
    g.replay()
    assert same((out, lse), run(c))


def test_repeated_calls_of_many_shapes_share_a_workspace():
    ws = q.Workspace()
    cases = [Case([3000, 10], [20, 5], 8, 2, d, 16, k, seed=d) for d in (64, 128, 256) for k in ("fp16", "int8")]
    want = [run(c) for c in cases]
    for _ in range(3):
        for c, w in zip(cases, want):
            assert same(w, run(c, ws=ws))


def test_binding_refusals():
    c = Case([100], [10], 8, 2, 128, 16, "fp16", seed=16)
    a = c.args()
    with pytest.raises(ValueError):
        q.attn_tree(c.q, *a, c.parents[:5])
    with pytest.raises(TypeError):
        q.attn_tree(c.q, *a, c.parents.long())
    with pytest.raises(TypeError):
        q.attn_tree(c.q, *a, c.parents.cpu())
    with pytest.raises(q.QgemmError):
        q.attn_tree(c.q, *a, c.parents, max_nodes=257)
    with pytest.raises(q.QgemmError):
        q.attn_tree(c.q, *a, c.parents, max_nodes=0)
    with pytest.raises(q.QgemmError):
        q.attn_tree(c.q, *a, c.parents, window=-1)
    with pytest.raises(ValueError):
        q.attn_tree(c.q, *a, c.parents, out=torch.empty(3, 8, 128, dtype=torch.float16, device=DEV))
    with pytest.raises(TypeError):
        q.attn_tree(c.q.bfloat16(), *a, c.parents)


@pytest.mark.parametrize("kind,d,Hq,Hkv", [("fp16", 256, 160, 1), ("int8", 256, 160, 1), ("bf16", 256, 512, 2), ("fp16", 64, 1024, 1)])
def test_more_heads_than_rows_of_a_block(kind, d, Hq, Hkv):
    check(Case([200, 5, 70], [3, 5, 1], Hq, Hkv, d, 16, kind, seed=31))


@pytest.mark.parametrize("kind", ["fp16", "int8"])
@pytest.mark.parametrize("d,page", [(128, 16), (64, 7), (256, 32)])
def test_broadcast_tensors(kind, d, page):
    """One query row for all nodes or heads, one KV head for all: strides of 0."""
    c = Case([300, 40], [20, 9], 8, 4, d, page, kind, seed=32)
    lse = torch.empty(c.T, 8, device=DEV)
    call = lambda qq, k=c.k, v=c.v, kw=c.kw: q.attn_tree(qq, k, v, *c.args()[2:], c.parents, lse=lse.clone(), **kw)
    for qq in (c.q[:1].expand_as(c.q), c.q[:, :1].expand_as(c.q), c.q[:1, :1].expand_as(c.q)):
        assert same(call(qq), call(qq.contiguous()))
    k, v = (x[:, :1].expand_as(x) for x in (c.k, c.v))
    kw = {n: x[:, :1].expand_as(x).contiguous() for n, x in c.kw.items()}
    assert same(call(c.q, k, v, kw), call(c.q, k.contiguous(), v.contiguous(), kw))
    assert q.device_error() == 0


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [8, 64, 48])
def test_scales_at_any_address(d, page):
    c = Case([300, 40, 1000], [20, 9, 64], 8, 2, d, page, "int8", seed=33)
    want = check(c)
    for off in (1, 2, 3):
        both = torch.full((2, c.kw["k_scale"].numel() + 4), math.nan, device=DEV)
        kw = {}
        for x, (n, s) in zip(both, c.kw.items()):
            kw[n] = x[off:off + s.numel()].view(s.shape)
            kw[n].copy_(s)
        assert same(want, q.attn_tree(c.q, *c.args(), c.parents, lse=torch.empty_like(want[1]), **kw))


@pytest.mark.parametrize("Hq", [8, 64])
def test_a_sequence_of_more_nodes_than_said(Hq):
    """It gets rows of zeros and the flag, whatever blocks it would take; the others their own."""
    c = Case([500, 1000, 64, 900, 30], [9, 256, 5, 70, 3], Hq, 2, 128, 16, "fp16", seed=34)
    want = run(c)
    assert q.device_error() == 0
    out, lse = run(c, max_nodes=9)
    assert q.device_error() == q.QW_ERR_BAD_INDEX
    t = 0
    for m in c.news:
        rows = slice(t, t + m)
        if m > 9:
            assert bool((out[rows] == 0).all()) and bool(torch.isneginf(lse[rows]).all())
        else:
            r = c.reference()
            assert bool(((out.double() - r[0]).abs() <= c.tolerances(r)[0])[rows].all())
        t += m


def test_two_calls_at_once():
    """Calls of two streams with workspaces of their own, none waiting for another; and two captured graphs."""
    c = [Case([9000, 700], [30, 64], 24, 4, 256, 16, "fp16", seed=35), Case([5000, 3, 800], [64, 3, 20], 16, 4, 128, 16, "int8", seed=36)]
    want = [run(x) for x in c]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(c[i]))
    torch.cuda.synchronize()
    assert all(same(w, x) for w, g in zip(want, got) for x in g)
    graphs, outs = [], []
    for x in c:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append([run(x) for _ in range(4)])
        graphs.append(g)
    for _ in range(5):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(same(w, x) for w, g in zip(want, outs) for x in g) and q.device_error() == 0


@pytest.mark.parametrize("kind,d,page", [("fp16", 64, 16), ("bf16", 128, 8), ("fp16", 256, 64), ("int8", 64, 16), ("int8", 128, 7),
                                         ("int8", 256, 16), ("fp16", 128, 5)])
def test_wait_limit_ends_the_kernel(kind, d, page):
    """At a limit of 0 every wait that is not over when first looked at gives up, in unmodified kernels;
    afterwards the same workspace serves as before."""
    c = Case([3000, 40, 700], [40, 9, 64], 8, 2, d, page, kind, seed=37)
    ws = q.Workspace()
    want = run(c, ws=ws)
    assert q.device_error() == 0
    q.set_wait_limit_us(0)
    errs = []
    try:
        for _ in range(3):
            run(c, ws=ws)
            errs.append(q.device_error())
    finally:
        q.set_wait_limit_us(None)
    assert errs == [q.QW_ERR_TIMEOUT] * 3
    assert same(want, run(c, ws=ws)) and q.device_error() == 0


@pytest.mark.parametrize("kind,page", [("fp16", 16), ("fp16", 12), ("int8", 16), ("int8", 7)])
def test_pages_far_into_a_large_cache(kind, page):
    """Pools of over 2^32 bytes: the pages at their end, as those of a small cache."""
    c = Case([400, 60], [20, 9], 8, 4, 256, page, kind, seed=38)
    want = run(c)
    n = c.k.shape[0]
    total = (5 << 30) // (4 * page * 256 * c.k.element_size()) + n
    k, v = (torch.empty((total, *c.k.shape[1:]), dtype=c.k.dtype, device=DEV) for _ in range(2))
    k[-n:], v[-n:] = c.k, c.v
    kw = {}
    for name, s in c.kw.items():
        kw[name] = torch.zeros((total, *s.shape[1:]), device=DEV)
        kw[name][-n:] = s
    table = c.table + (total - n)
    assert same(want, q.attn_tree(c.q, k, v, table, c.lens, c.cu, c.parents, lse=torch.empty_like(want[1]), **kw))
    assert q.device_error() == 0
    # and its rows moved
    path, count = torch.tensor([[0, 4, 9], [2, 8, -1]], dtype=torch.int32, device=DEV), torch.tensor([3, 2], dtype=torch.int32, device=DEV)
    small = q.kv_keep_path(path, count, c.table, c.lens, c.cu, c.k, c.v, *c.kw.values())
    large = q.kv_keep_path(path, count, table, c.lens, c.cu, k, v, *kw.values())
    assert torch.equal(small, large) and q.device_error() == 0
    used = c.table.long().unique()
    for x, y in zip((c.k, c.v, *c.kw.values()), (k, v, *kw.values())):
        assert torch.equal(x[used].nan_to_num(7), y[-n:][used].nan_to_num(7))


def test_nothing_to_do():
    """No new tokens, and no sequences."""
    c = Case([100, 50], [10, 5], 8, 2, 128, 16, "fp16", seed=39)
    zero = torch.zeros(3, dtype=torch.int32, device=DEV)
    out, lse = q.attn_tree(c.q[:0], c.k, c.v, c.table, c.lens, zero, c.parents[:0], lse=torch.empty(0, 8, device=DEV))
    assert out.shape == (0, 8, 128) and lse.shape == (0, 8)
    out = torch.full_like(c.q.contiguous(), 3.0)
    q.attn_tree(c.q, c.k, c.v, c.table[:0], c.lens[:0], zero[:1], c.parents, out=out)
    assert bool((out == 3).all())
    path = torch.zeros(0, 4, dtype=torch.int32, device=DEV)
    assert q.kv_keep_path(path, zero[:0], c.table[:0], c.lens[:0], zero[:1], c.k, c.v).shape == (0,)
    assert q.device_error() == 0


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [1, 7, 16])
def test_int8_tiles_that_wait_for_values(d, page):
    """Large trees over pages that are gathered: the loads bound the call, so a slot of codes is filled
    again as soon as it is given back.  Every run the same."""
    c = Case([2653, 4761, 3900, 1135, 3167], [1, 130, 224, 1, 250], 24, 4, d, page, "int8", seed=40)
    want = check(c)
    for _ in range(10):
        assert same(want, run(c))


@pytest.mark.parametrize("cu,left", [([1, 3, 2, 4], [0, 4, 5]), ([-7, 1, 1, 2], [2, 3, 4, 5]),
                                     ([5, 900, 900, 900], [0, 1, 2, 3, 4]), ([6, -2, -2, 0], [0, 1, 2, 3, 4, 5])])
def test_offsets_stay_inside(cu, left):
    """Offsets that descend or leave 0 .. T write no row outside q's nor one of no sequence."""
    c = Case([40, 40, 40], [2, 2, 2], 4, 2, 64, 16, "fp16", seed=44)
    c.cu.copy_(torch.tensor(cu, device=DEV))
    c.parents.fill_(-1)
    big = torch.full((c.T + 16, 4, 64), 3.0, dtype=torch.float16, device=DEV)
    lse = torch.full((c.T + 16, 4), 3.0, device=DEV)
    q.attn_tree(c.q, *c.args(), c.parents, max_nodes=2, out=big[8:8 + c.T], lse=lse[8:8 + c.T])
    assert q.device_error() == q.QW_ERR_BAD_INDEX and q.device_error() == 0
    keep = torch.ones(c.T + 16, dtype=torch.bool, device=DEV)
    keep[8:8 + c.T] = False
    keep[[8 + t for t in left]] = True
    assert bool((big[keep] == 3.0).all()) and bool((lse[keep] == 3.0).all())
    assert bool(torch.isfinite(big.float()).all()) and not bool((big[~keep] == 3.0).any())


@pytest.mark.parametrize("d", [64, 128, 256])
def test_overlapping_offsets_past_2_to_32_places(d):
    """Offsets that descend can name each node many times: 8200 sequences of all 256 nodes, 64 KV heads of 1024 tiles,
    would be more than 2^32 places.  Nothing is computed, and the next call, with the same workspace, is right.
    Fewer of them are computed."""
    i32 = dict(dtype=torch.int32, device=DEV)
    T, H, B = 256, 64, 16400
    k = torch.randn(1, H, 1024, d, device=DEV).half()
    table, lens = torch.zeros(B, 64, **i32), torch.full((B,), 65536, **i32)
    cu = torch.tensor([0, T] * (B // 2) + [0], **i32)
    qq, parents = torch.randn(T, 16 * H, d, device=DEV).half(), torch.full((T,), -1, **i32)
    ws = q.Workspace(torch.device("cuda:0"))
    out = torch.full_like(qq, 3.0)
    q.attn_tree(qq, k, k, table, lens, cu, parents, max_nodes=256, out=out, ws=ws)
    assert q.device_error() == q.QW_ERR_BAD_INDEX and bool((out == 3.0).all())
    check(Case([40, 3000], [1, 20], 64, 64, d, 16, "fp16", seed=45), ws=ws)
    few = torch.tensor([0, 2, 0, 2, 2], **i32)            # the first and third sequence alike
    got = q.attn_tree(qq[:2, :H], k, k, table[:4, :1].contiguous(), torch.full((4,), 500, **i32), few, parents[:2], ws=ws)
    assert q.device_error() == q.QW_ERR_BAD_INDEX
    want = q.attn_tree(qq[:2, :H], k, k, table[:1, :1].contiguous(), torch.full((1,), 500, **i32), few[:2], parents[:2], ws=ws)
    assert q.device_error() == 0 and float((got - want).abs().max()) <= 2 ** -9 * float(want.abs().max())


@pytest.mark.parametrize("kind,d,page", [("fp16", 64, 16), ("bf16", 128, 7), ("fp16", 256, 48), ("int8", 64, 16), ("int8", 128, 16),
                                         ("int8", 256, 64), ("int8", 128, 7), ("int8", 64, 1)])
@pytest.mark.parametrize("bad", [-1, 1 << 20])
def test_pages_outside_the_pool_are_rows_of_zeros(kind, d, page, bad):
    """Compared with the definition, whose cache has a page of zeros there."""
    c = Case([700, 90], [20, 9], 8, 2, d, page, kind, seed=41)
    for x in ("k64", "v64"):
        setattr(c, x, torch.cat([getattr(c, x), torch.zeros_like(getattr(c, x)[:1])]))
    places = [(0, 3), (0, 5), (0, (700 - 1) // page), (1, 0)]
    for b, i in places:
        c.table[b, i] = c.k64.shape[0] - 1
    r = c.reference()
    for b, i in places:
        c.table[b, i] = bad
    out, lse = run(c)
    assert q.device_error() == q.QW_ERR_BAD_INDEX
    tol, lse_tol = c.tolerances(r)
    assert bool(((out.double() - r[0]).abs() <= tol).all()) and bool(((lse.double() - r[1]).abs() <= lse_tol).all())


@pytest.mark.parametrize("d,ctas", [(64, 2), (128, 2), (256, 1)])
def test_a_page_outside_the_pool_has_no_scales(d, ctas):
    """Twenty tiles a CTA, every third of a page that is none: its scores are 0, whatever scales the tiles before had (large ones,
    with codes of 0)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = 64 * 20 * ctas * sms
    k, v = torch.zeros(1, 1, 64, d, dtype=torch.int8, device=DEV), torch.ones(1, 1, 64, d, dtype=torch.int8, device=DEV)
    ks, vs = torch.full((1, 1, 64), 5e37, device=DEV), torch.ones(1, 1, 64, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    table = torch.where(torch.arange(n // 64, device=DEV) % 3 == 2, -1, 0).int()[None]
    qq = torch.randn(1, 1, d, device=DEV).half()
    lse = torch.empty(1, 1, device=DEV)
    out, lse = q.attn_tree(qq, k, v, table, torch.tensor([n], **i32), torch.tensor([0, 1], **i32), torch.tensor([-1], **i32), scale=4.0,
                           k_scale=ks, v_scale=vs, lse=lse)
    assert q.device_error() == q.QW_ERR_BAD_INDEX
    share = float((table == 0).sum()) / table.numel()
    assert bool(((out.double() - share).abs() <= 2.0 ** -10).all())      # (fp16's rounding: 2^-12)
    assert abs(float(lse) - math.log(n)) <= 2.0 ** -20 * math.log(n)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_the_largest_scales(d):
    """Value scales up to 2^127: the outputs pass fp16, the sum of exponentials does not care."""
    c = Case([300, 70], [20, 9], 8, 2, d, 16, "int8", seed=42)
    want = run(c)
    for s in (2.0 ** 125, 2.0 ** 126, 2.0 ** 127):
        c.kw["v_scale"].fill_(s)
        c.v.fill_(3)
        out, lse = run(c)
        tol = c.tolerances(c.reference())[1]
        assert q.device_error() == 0 and bool(torch.isposinf(out).all()) and bool(((lse - want[1]).abs() <= 2 * tol).all())


def test_sequences_of_more_nodes_than_any():
    """Between others, in CTAs whose shared memory holds NaN from the call before: rows of zeros, the others their own."""
    lens, news = [60, 400, 33] * 150, [5, 300, 7] * 150
    for kind, d in (("fp16", 128), ("bf16", 64), ("fp16", 256)):
        c = Case(lens, news, 8, 8, d, 16, kind, seed=43)
        small = [b for b, m in enumerate(news) if m < 100]
        rows = torch.cat([torch.arange(int(c.cu[b]), int(c.cu[b + 1]), device=DEV) for b in small])
        nan = torch.full_like(c.k, math.nan)
        want = None
        for _ in range(3):
            q.attn_paged(c.q[:450], nan, nan, c.table, c.lens, torch.arange(451, dtype=torch.int32, device=DEV))
            out, lse = run(c, max_nodes=8)
            assert q.device_error() == q.QW_ERR_BAD_INDEX
            alone = torch.ones(c.T, dtype=torch.bool, device=DEV)
            alone[rows] = False
            assert bool((out[alone] == 0).all()) and bool(torch.isneginf(lse[alone]).all())
            want = want or (out, lse)
            assert same(want, (out, lse))
        s = Case([lens[b] for b in small[:6]], [news[b] for b in small[:6]], 8, 8, d, 16, kind, seed=43)
        s.k, s.v, s.k64, s.v64 = c.k, c.v, c.k64, c.v64
        s.table, s.q = c.table[small[:6]], c.q[rows[:s.T]]
        s.trees = [c.trees[b] for b in small[:6]]
        r = s.reference()
        tol, lse_tol = s.tolerances(r)
        assert bool(((out[rows[:s.T]].double() - r[0]).abs() <= tol).all()) and bool(((lse[rows[:s.T]].double() - r[1]).abs() <= lse_tol).all())
