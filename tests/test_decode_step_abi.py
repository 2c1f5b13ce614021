"""Argument checks of the paged cache's and the token log probabilities' entry points, made
on the host before any device access (no GPU needed: the pointers are never read)."""
import ctypes

import pytest
import torch

import int8_weight_quantized_int4_gb300 as q

B = 1 << 20
P = ctypes.c_void_p(B)
N0 = ctypes.c_void_p(0)
OK = (q.QW_OK, q.QW_ERR_ARCH)                       # past the checks: no device here, or done


@pytest.fixture(scope="module", autouse=True)
def built():
    from int8_weight_quantized_int4_gb300 import build
    build.build()


def cache(**kw):
    d = dict(k=B, v=B, k_scale=B, v_scale=B, dtype=q.QW_KV_F16, num_pages=4, page=16, Hkv=4, d=128,
             page_stride=16 * 4 * 128, head_stride=16 * 128, token_stride=128)
    d.update(kw)
    return q.KvCacheDesc(*[d[n] for n, _ in q.KvCacheDesc._fields_])


def batch(**kw):
    d = dict(page_table=B, seq_lens=B, cu_tokens=B, B=2, max_pages=4)
    d.update(kw)
    return q.KvBatchDesc(*[d[n] for n, _ in q.KvBatchDesc._fields_])


def append(c, b, k=P, v=P, T=3, s=(512, 128, 512, 128)):
    return q.lib().kv_append(c, b, k, v, T, *s, N0)


BAD_CACHES = [
    (dict(dtype=5), q.QW_ERR_INVALID_ARG), (dict(page=0), q.QW_ERR_INVALID_ARG),
    (dict(num_pages=-1), q.QW_ERR_INVALID_ARG), (dict(Hkv=0), q.QW_ERR_INVALID_ARG),
    (dict(d=96), q.QW_ERR_UNSUPPORTED_SHAPE), (dict(d=512), q.QW_ERR_UNSUPPORTED_SHAPE),
    (dict(k=0), q.QW_ERR_INVALID_ARG), (dict(dtype=q.QW_KV_INT8, v_scale=0), q.QW_ERR_INVALID_ARG),
    (dict(k=B + 8), q.QW_ERR_ALIGNMENT), (dict(v=B + 2), q.QW_ERR_ALIGNMENT),
    (dict(token_stride=132), q.QW_ERR_ALIGNMENT), (dict(page_stride=8196), q.QW_ERR_ALIGNMENT),
    (dict(dtype=q.QW_KV_INT8, head_stride=8), q.QW_ERR_ALIGNMENT),
    (dict(dtype=q.QW_KV_INT8, k_scale=B + 2), q.QW_ERR_ALIGNMENT),
    (dict(page_stride=-8192), q.QW_ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_cache_refusals(kw, code):
    assert append(cache(**kw), batch()) == code
    L = q.lib()
    assert L.attn_paged(cache(**kw), batch(), P, 3, 8, 1024, 128, 1, 0, 0, 1.0, P, N0, P, B, N0) == code
    assert L.qw_last_error_string()


def test_append_refusals():
    c, b = cache(), batch()
    assert append(c, b, T=-1) == q.QW_ERR_INVALID_ARG
    assert append(c, b, k=N0) == append(c, b, v=N0) == q.QW_ERR_INVALID_ARG
    assert append(c, b, k=ctypes.c_void_p(B + 8)) == q.QW_ERR_ALIGNMENT
    assert append(c, b, s=(516, 128, 512, 128)) == q.QW_ERR_ALIGNMENT
    assert append(c, batch(B=-1)) == q.QW_ERR_INVALID_ARG
    assert append(c, batch(page_table=0)) == q.QW_ERR_INVALID_ARG
    assert append(c, batch(seq_lens=B + 2)) == q.QW_ERR_ALIGNMENT
    assert append(c, batch(max_pages=1 << 27)) == q.QW_ERR_UNSUPPORTED_SHAPE      # 2^31 keys
    assert append(c, b, T=0, k=N0, v=N0) == q.QW_OK
    assert append(c, batch(B=0, page_table=0, seq_lens=0, cu_tokens=0)) == q.QW_OK
    assert q.lib().kv_append(None, b, P, P, 3, 512, 128, 512, 128, N0) == q.QW_ERR_INVALID_ARG
    assert q.lib().kv_append(c, None, P, P, 3, 512, 128, 512, 128, N0) == q.QW_ERR_INVALID_ARG


def test_attn_refusals():
    L, c, b = q.lib(), cache(), batch()

    def call(qp=P, T=3, Hq=8, st=(1024, 128), max_new=1, window=0, sinks=0, scale=1.0, out=P, lse=N0, ws=P, n=1 << 30):
        return L.attn_paged(c, b, qp, T, Hq, *st, max_new, window, sinks, scale, out, lse, ws, n, N0)
    assert call(Hq=6) == q.QW_ERR_UNSUPPORTED_SHAPE            # 4 KV heads do not divide 6
    assert call(Hq=2048) == q.QW_ERR_UNSUPPORTED_SHAPE
    assert call(Hq=0) == call(max_new=0) == call(T=-2) == q.QW_ERR_INVALID_ARG
    assert call(window=-1) == call(sinks=-1) == q.QW_ERR_INVALID_ARG
    assert call(scale=float("nan")) == call(scale=float("inf")) == q.QW_ERR_INVALID_ARG
    assert call(qp=N0) == call(out=N0) == q.QW_ERR_INVALID_ARG
    assert call(st=(1028, 128)) == call(out=ctypes.c_void_p(B + 4)) == q.QW_ERR_ALIGNMENT
    assert call(lse=ctypes.c_void_p(B + 2)) == call(ws=ctypes.c_void_p(B + 64)) == q.QW_ERR_ALIGNMENT
    assert call(T=(1 << 31) - 1) == q.QW_ERR_UNSUPPORTED_SHAPE
    assert call(T=0, qp=N0, out=N0, ws=N0) == q.QW_OK
    assert L.attn_paged_workspace_bytes(96, 8, 4, 1) == 0 and L.attn_paged_workspace_bytes(128, 6, 4, 1) == 0
    assert L.attn_paged_workspace_zero_bytes(128, 8, 4, 1) == 12288


def test_copy_refusals():
    L = q.lib()

    def call(n=2, pairs=P, n_pools=1, **kw):
        d = dict(base=B, layers=2, num_pages=4, layer_stride=1 << 16, page_stride=4096, page_bytes=4096)
        d.update(kw)
        pool = q.PagePoolDesc(*[d[k] for k, _ in q.PagePoolDesc._fields_])
        return L.kv_copy_pages(pool, n_pools, pairs, n, N0)
    assert call(n=-1) == call(n_pools=5) == call(n_pools=-1) == q.QW_ERR_INVALID_ARG
    assert call(layers=-1) == call(num_pages=-1) == call(page_bytes=-4) == q.QW_ERR_INVALID_ARG
    assert call(page_bytes=4098) == q.QW_ERR_UNSUPPORTED_SHAPE
    assert call(page_stride=2048) == q.QW_ERR_INVALID_ARG                 # pages would overlap
    assert call(base=0) == call(pairs=N0) == q.QW_ERR_INVALID_ARG
    assert call(base=B + 2) == call(page_stride=4098) == call(pairs=ctypes.c_void_p(B + 4)) == q.QW_ERR_ALIGNMENT
    assert call(n=0, pairs=N0) == call(layers=0) == call(page_bytes=0) == q.QW_OK
    assert L.kv_copy_pages(None, 0, N0, 0, N0) == q.QW_OK
    assert L.kv_copy_pages(None, 1, P, 1, N0) == q.QW_ERR_INVALID_ARG


def test_logprobs_refusals():
    L = q.lib()

    def call(x=P, dtype=q.QW_F16, M=2, N=100, tok=P, tb=4, C=1, k=5, lp=P, e=P, lse=P, tl=P, ti=P, ws=P):
        return L.token_logprobs(x, dtype, M, N, N, tok, tb, C, k, lp, e, lse, tl, ti, ws, 1 << 30, N0)
    assert call(dtype=3) == call(M=-1) == call(C=-1) == call(k=-1) == call(tb=2) == q.QW_ERR_INVALID_ARG
    assert call(N=0, k=0) == call(k=65) == call(N=4, k=5) == call(N=(1 << 30) + 1) == q.QW_ERR_UNSUPPORTED_SHAPE
    for name in ("x", "tok", "lp", "e", "lse", "tl", "ti"):
        assert call(**{name: N0}) == q.QW_ERR_INVALID_ARG
    assert call(x=ctypes.c_void_p(B + 1)) == call(ti=ctypes.c_void_p(B + 2)) == q.QW_ERR_ALIGNMENT
    assert call(tb=8, tok=ctypes.c_void_p(B + 4)) == call(ws=ctypes.c_void_p(B + 16)) == q.QW_ERR_ALIGNMENT
    assert call(M=0, x=N0) == q.QW_OK
    assert call(C=0, k=0, tok=N0, lp=N0, tl=N0, ti=N0) in OK
    assert L.token_logprobs_workspace_bytes(2, 0, 0, 0) == L.token_logprobs_workspace_bytes(2, 10, 11, 0) == 0


def test_binding_refuses_cpu_tensors():
    k = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    i = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(TypeError):
        q.kv_append(k[0], k[0], k, k, i, i[0], i[0])
    with pytest.raises(TypeError):
        q.attn_paged(k[0], k, k, i, i[0], i[0])
    with pytest.raises(TypeError):
        q.kv_copy_pages(i, k)
    with pytest.raises(TypeError):
        q.token_logprobs(k[0, 0], i[0])
