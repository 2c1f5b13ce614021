"""Argument checks of attn_tree, sample_tokens, tree_accept and kv_keep_path, made on the host
before any device access (no GPU needed: the pointers are never read)."""
import ctypes

import pytest

import int8_weight_quantized_int4_gb300 as q
from tests import _tree_ref as ref
from tests.test_decode_step_abi import B, BAD_CACHES, N0, P, batch, cache

ODD = ctypes.c_void_p(B + 2)


@pytest.fixture(scope="module", autouse=True)
def built():
    from int8_weight_quantized_int4_gb300 import build
    build.build()


def tree(c, b, parents=P, qp=P, T=3, Hq=8, st=(1024, 128), max_nodes=8, window=0, sinks=0, scale=1.0, out=P, lse=N0, ws=P,
         n=1 << 40):
    return q.lib().attn_tree(c, b, parents, qp, T, Hq, *st, max_nodes, window, sinks, scale, out, lse, ws, n, N0)


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_cache_refusals(kw, code):
    assert tree(cache(**kw), batch()) == code and q.lib().qw_last_error_string()


def test_attn_tree_refusals():
    c, b = cache(), batch()
    assert tree(c, b, Hq=6) == tree(c, b, Hq=2048) == tree(c, b, max_nodes=257) == q.QW_ERR_UNSUPPORTED_SHAPE
    assert tree(c, b, Hq=0) == tree(c, b, max_nodes=0) == tree(c, b, T=-2) == q.QW_ERR_INVALID_ARG
    assert tree(c, b, window=-1) == tree(c, b, sinks=-1) == q.QW_ERR_INVALID_ARG
    assert tree(c, b, scale=float("nan")) == tree(c, b, scale=float("inf")) == q.QW_ERR_INVALID_ARG
    assert tree(c, b, qp=N0) == tree(c, b, out=N0) == tree(c, b, parents=N0) == q.QW_ERR_INVALID_ARG
    assert tree(c, batch(page_table=0)) == tree(c, batch(B=-1)) == q.QW_ERR_INVALID_ARG
    assert tree(c, b, st=(1028, 128)) == tree(c, b, out=ctypes.c_void_p(B + 8)) == q.QW_ERR_ALIGNMENT
    assert tree(c, b, lse=ODD) == tree(c, b, parents=ODD) == tree(c, b, ws=ctypes.c_void_p(B + 64)) == q.QW_ERR_ALIGNMENT
    assert tree(c, b, T=(1 << 31) - 1) == tree(c, batch(max_pages=1 << 27)) == q.QW_ERR_UNSUPPORTED_SHAPE
    assert tree(c, b, T=0, qp=N0, out=N0, ws=N0, parents=N0) == q.QW_OK
    assert tree(c, batch(B=0, page_table=0, seq_lens=0, cu_tokens=0)) == q.QW_OK
    assert tree(None, b) == tree(c, None) == q.QW_ERR_INVALID_ARG
    assert q.lib().attn_tree_workspace_bytes(96, 8, 4) == 0 and q.lib().attn_tree_workspace_bytes(128, 6, 4) == 0


def sample(x=P, dtype=q.QW_F16, M=2, N=100, row=100, u=P, token=P, lp=P, **kw):
    s = q.SamplingDesc(**{**dict(temperature=1.0, top_p=1.0), **kw})
    return q.lib().sample_tokens(x, dtype, M, N, row, u, s, token, lp, N0)


def test_sample_refusals():
    assert sample(dtype=3) == sample(M=-1) == sample(row=-1) == q.QW_ERR_INVALID_ARG
    assert sample(N=0) == sample(N=(1 << 20) + 1) == q.QW_ERR_UNSUPPORTED_SHAPE
    assert sample(x=N0) == sample(u=N0) == sample(token=N0) == q.QW_ERR_INVALID_ARG
    assert sample(x=ctypes.c_void_p(B + 1)) == sample(x=ODD, dtype=q.QW_F32) == sample(u=ODD) == q.QW_ERR_ALIGNMENT
    assert sample(token=ODD) == sample(lp=ODD) == sample(temperatures=B + 2) == sample(top_ks=B + 2) == q.QW_ERR_ALIGNMENT
    assert sample(top_ps=B + 1) == sample(min_ps=B + 1) == q.QW_ERR_ALIGNMENT
    assert sample(M=0, x=N0, u=N0, token=N0) == q.QW_OK
    assert q.lib().sample_tokens(P, 0, 2, 100, 100, P, None, P, P, N0) == q.QW_ERR_INVALID_ARG


def test_accept_refusals():
    def call(t=P, d=P, p=P, cu=P, B_=2, T=5, w=3, path=P, count=P, nxt=P):
        return q.lib().tree_accept(t, d, p, cu, B_, T, w, path, count, nxt, N0)
    assert call(B_=-1) == call(T=-1) == call(w=0) == q.QW_ERR_INVALID_ARG
    assert call(t=N0) == call(d=N0) == call(p=N0) == call(cu=N0) == q.QW_ERR_INVALID_ARG
    assert call(path=N0) == call(count=N0) == call(nxt=N0) == q.QW_ERR_INVALID_ARG
    assert call(t=ODD) == call(d=ODD) == call(p=ODD) == call(cu=ODD) == call(path=ODD) == q.QW_ERR_ALIGNMENT
    assert call(count=ODD) == call(nxt=ODD) == q.QW_ERR_ALIGNMENT
    assert call(B_=0, t=N0, d=N0, p=N0, cu=N0, path=N0, count=N0, nxt=N0) == q.QW_OK


def test_keep_refusals():
    def call(b=None, n_pools=1, T=5, page=16, path=P, count=P, w=3, lens=P, **kw):
        d = dict(base=B, layers=2, num_pages=4, heads=2, row_bytes=256, layer_stride=1 << 16, page_stride=8192,
                 head_stride=4096, token_stride=256)
        d.update(kw)
        pool = q.RowPoolDesc(*[d[k] for k, _ in q.RowPoolDesc._fields_])
        return q.lib().kv_keep_path(pool, n_pools, batch() if b is None else b, T, page, path, count, w, lens, N0)
    for kw in (dict(n_pools=-1), dict(n_pools=5), dict(T=-1), dict(page=0), dict(w=-1), dict(layers=-1), dict(heads=-1),
               dict(num_pages=-1), dict(row_bytes=-4), dict(page_stride=-1), dict(base=0), dict(path=N0), dict(count=N0),
               dict(token_stride=128), dict(b=batch(B=-1)), dict(b=batch(seq_lens=0))):
        assert call(**kw) == q.QW_ERR_INVALID_ARG, kw
    for kw in (dict(row_bytes=254), dict(page=1 << 21), dict(b=batch(max_pages=1 << 27)), dict(row_bytes=1 << 21),
               dict(layers=1 << 24, heads=1 << 10)):
        assert call(**kw) == q.QW_ERR_UNSUPPORTED_SHAPE, kw
    for kw in (dict(base=B + 2), dict(head_stride=4098), dict(path=ODD), dict(count=ODD), dict(lens=ODD),
               dict(b=batch(page_table=B + 2))):
        assert call(**kw) == q.QW_ERR_ALIGNMENT, kw
    assert call(b=batch(B=0, page_table=0, seq_lens=0, cu_tokens=0)) == q.QW_OK
    assert call(lens=N0, layers=0) == call(lens=N0, n_pools=0) == q.QW_OK
    assert q.lib().kv_keep_path(None, 1, batch(), 5, 16, P, P, 3, P, N0) == q.QW_ERR_INVALID_ARG
    assert q.lib().kv_keep_path(None, 0, None, 5, 16, P, P, 3, P, N0) == q.QW_ERR_INVALID_ARG


def test_strides_that_make_no_sense_are_refused():
    c, b = cache(), batch()
    assert tree(c, b, st=(-1024, 128)) == tree(c, b, st=(1024, -128)) == q.QW_ERR_INVALID_ARG
    sizes = dict(base=B, layers=2, num_pages=4, heads=2, row_bytes=256, layer_stride=1 << 16, page_stride=8192, head_stride=4096,
                 token_stride=256)
    names = [k for k, _ in q.RowPoolDesc._fields_]

    def keep(n=1, lens=ctypes.c_void_p(B + 64), **kw):
        pools = (q.RowPoolDesc * n)(*[q.RowPoolDesc(*[{**sizes, **kw}[k] for k in names]) for _ in range(n)])
        return q.lib().kv_keep_path(pools, n, batch(), 5, 16, P, P, 3, lens, N0)
    for name in ("layer_stride", "page_stride", "head_stride", "token_stride"):      # rows that overlap would be moved twice
        assert keep(**{name: 0}) == keep(**{name: 128}) == q.QW_ERR_INVALID_ARG, name
    assert keep(n=2) == q.QW_ERR_INVALID_ARG                                         # as would a pool given twice
    assert keep(lens=ctypes.c_void_p(batch().seq_lens)) == q.QW_ERR_INVALID_ARG      # lengths that other warps still read


def test_definitions():
    """The plain forms that the GPU tests compare with, on cases that can be seen."""
    import math

    import numpy as np
    x = np.log(np.array([0.1, 0.4, 0.4, 0.1]))
    assert ref.draw(x, 0.0)[0] == 0 and ref.draw(x, 0.05)[0] == 0 and ref.draw(x, 0.3)[0] == 1
    assert ref.draw(x, 0.7)[0] == 2 and ref.draw(x, 0.95)[0] == 3
    t, lp = ref.draw(x, 0.6, top_k=2)
    assert t == 2 and abs(lp - math.log(0.5)) < 1e-12
    assert ref.draw(x, 0.99, top_p=0.3)[0] == 1                    # the first reaches 0.3 by itself
    assert ref.draw(x, 0.99, top_p=0.85)[0] == 2                   # 0.1 more: the lower index first
    assert ref.draw(x, 0.0, top_p=0.85)[0] == 0
    assert ref.draw(x, 0.99, min_p=0.5)[0] == 2 and ref.draw(x, 0.9, temperature=0)[0] == 1
    assert ref.draw(np.array([-math.inf, math.nan]), 0.5) == (-1, -math.inf)
    assert ref.accept([9, 5, 5, 7], [5, 7, 7, 1], [-1, 0, 0, 1], 9) == ([0, 1, 3], 1)
    assert ref.accept([9, 5, 5, 7], [5, 7, 7, 1], [-1, 0, 0, 1], 2) == ([0, 1], 7)
    assert ref.accept([], [], [], 2) == ([], -1)
    assert ref.ancestors([-1, 0, 0, 2], 3) == [0, 2, 3]


def row_pool(base, shape, strides, row):
    return q.RowPoolDesc(base, shape[0], shape[1], shape[2], row, strides[0], strides[1], strides[2], strides[3])


def keep_pools(*pools, page=16):
    """What kv_keep_path says of the pools: no offsets are given, so what passes ends with an aligned pointer's refusal."""
    a = (q.RowPoolDesc * len(pools))(*pools)
    return q.lib().kv_keep_path(a, len(pools), batch(), 5, page, ODD, P, 3, P, N0)


def test_rows_that_overlap_are_refused():
    """Strides that are fine one by one."""
    page, heads, row = 16, 4, 256
    good, bad = q.QW_ERR_ALIGNMENT, q.QW_ERR_INVALID_ARG
    hnd, nhd = (4 * 16384, 16384, 4096, 256), (4 * 16384, 16384, 256, 1024)
    for st in (hnd, nhd, (1 << 40, 16384 + 64, 4096 + 16, 256), (16384, 2 * 16384, 256, 1024), (256, 512, 2048, 8192 * 4)):
        assert keep_pools(row_pool(B, (2, 4, heads), st, row)) == good, st
    for st in ((4 * 16384, 16384, 256, 256), (4 * 16384, 16384, 256, 1020), (4 * 16384, 16380, 4096, 256), (16384, 16384, 4096, 256),
               (3 * 16384, 16384, 4096, 256), (4 * 16384, 16384, 4092, 256), (1 << 62, 1 << 62, 1 << 62, 1 << 62)):
        assert keep_pools(row_pool(B, (2, 4, heads), st, row)) == bad, st
    # dimensions of one entry mean nothing
    assert keep_pools(row_pool(B, (1, 4, 1), (0, 4096, 0, 256), row)) == good
    assert keep_pools(row_pool(B, (2, 4, heads), (1024, 2048, 256, 0), row), page=1) == good


def test_pools_that_share_rows_are_refused():
    good, bad = q.QW_ERR_ALIGNMENT, q.QW_ERR_INVALID_ARG
    hnd, shape = (4 * 16384, 16384, 4096, 256), (2, 4, 4)
    size = 2 * 4 * 16384
    k = row_pool(B, shape, hnd, 256)
    assert keep_pools(k, row_pool(B + size, shape, hnd, 256)) == good                       # one after the other
    assert keep_pools(k, row_pool(B + size - 256, shape, hnd, 256)) == bad                  # by its last row
    assert keep_pools(k, row_pool(B + 4, shape, hnd, 256)) == bad
    assert keep_pools(k, row_pool(B + 4 * 16384, (1, 4, 4), hnd, 256)) == bad               # pools[0] and pools[0][1:]
    assert keep_pools(row_pool(B, (1, 4, 4), hnd, 256), row_pool(B + 4 * 16384, (1, 4, 4), hnd, 256)) == good      # its layers
    # K and V laced by layer, page, head or token
    for st, gap in (((8 * 16384, 16384, 4096, 256), 4 * 16384), ((8 * 16384, 32768, 4096, 256), 16384), ((8 * 16384, 32768, 8192, 256), 4096),
                    ((8 * 16384, 32768, 8192, 512), 256)):
        assert keep_pools(row_pool(B, shape, st, 256), row_pool(B + gap, shape, st, 256)) == good, st
        assert keep_pools(row_pool(B + gap, shape, st, 256), row_pool(B, shape, st, 256)) == good, st
        assert keep_pools(row_pool(B, shape, st, 256), row_pool(B + gap - 16, shape, st, 256)) == bad, st
    # codes and scales in one page: 16 rows of 256 bytes, then 16 numbers
    st = (4 * 4 * 4160, 4 * 4160, 4160)
    codes, scales = row_pool(B, shape, (*st, 256), 256), row_pool(B + 4096, shape, (*st, 4), 4)
    assert keep_pools(codes, scales) == keep_pools(scales, codes) == good
    assert keep_pools(codes, row_pool(B + 4092, shape, (*st, 4), 4)) == bad
    # a row's scale behind its codes
    st = (16 * 4 * 4 * 260, 16 * 4 * 260, 16 * 260, 260)
    assert keep_pools(row_pool(B, shape, st, 256), row_pool(B + 256, shape, st, 4)) == good
    assert keep_pools(row_pool(B, shape, st, 260), row_pool(B + 256, shape, st, 4)) == bad
    # four pools, and one without rows
    four = [row_pool(B + i * size, shape, hnd, 256) for i in range(4)]
    assert keep_pools(*four) == good and keep_pools(*four[:3], four[1]) == bad
    assert keep_pools(k, row_pool(B, (0, 4, 4), hnd, 256)) == good


def test_pools_that_meet_by_chance():
    """Random strides, compared with all rows laid out."""
    import random
    rng = random.Random(3)
    seen = [0, 0]
    for _ in range(400):
        pools, rows = [], []
        for _ in range(2):
            n = [rng.randint(1, 3) for _ in range(3)] + [2]
            row, order, st, span = 4 * rng.randint(1, 3), rng.sample(range(4), 4), [0] * 4, 0
            span = row
            for i in order:
                st[i] = span + 4 * rng.choice([0, 0, 0, 1, 2, 8])
                span += (n[i] - 1) * st[i]
            base = 4 * rng.randint(0, 60)
            pools.append(row_pool(B + base, n[:3], st, row))
            rows.append({base + a * st[0] + b * st[1] + c * st[2] + d * st[3] + e for a in range(n[0]) for b in range(n[1])
                         for c in range(n[2]) for d in range(n[3]) for e in range(row)})
        meet = bool(rows[0] & rows[1])
        seen[meet] += 1
        assert keep_pools(*pools, page=2) == (q.QW_ERR_INVALID_ARG if meet else q.QW_ERR_ALIGNMENT)
    assert min(seen) > 60
