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
