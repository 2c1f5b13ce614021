"""kv_append and kv_copy_pages on the GPU: bytes moved exactly, nothing else touched; int8
rows bit-exact against the quantizer's definition (IEEE divisions, round half to even)."""
import numpy as np
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


def bits(t):
    return t.contiguous().view({1: torch.int8, 2: torch.int16, 4: torch.int32}[t.element_size()])


BATCHES = [
    ([1], [1]), ([17], [17]), ([16, 33, 5], [1, 1, 1]), ([40, 0, 7, 100, 3], [0, 0, 7, 31, 2]),
    (list(range(1, 71)), [1] * 70), ([300] * 3 + [9] * 40, [37, 0, 300] + [2] * 40),
]


@pytest.mark.parametrize("kind,d,Hq,Hkv,page,nhd", [
    ("fp16", 256, 24, 4, 16, False), ("bf16", 128, 32, 8, 64, True), ("fp16", 64, 6, 2, 1, False),
    ("bf16", 64, 8, 8, 48, False), ("int8", 256, 24, 4, 16, False), ("int8", 128, 5, 5, 7, False),
    ("int8", 64, 3, 1, 32, False)])
@pytest.mark.parametrize("lens,news", BATCHES)
def test_append(q, kind, d, Hq, Hkv, page, nhd, lens, news):
    c = Cache(lens, news, Hq, Hkv, d, page, kind, nhd, seed=d + len(lens), stale=0.5)
    k, v = c.qkv[:, Hq:Hq + Hkv], c.qkv[:, Hq + Hkv:]
    if kind == "int8" and c.T > 2:
        k[1, 0] = 0.0                                      # a zero row: scale 0, codes 0
        v[2, -1, 3] = 200.0                                # one large value
    want_k, want_v = c.k.clone(), c.v.clone()
    want_ks, want_vs = c.ks.clone(), c.vs.clone()
    t = 0
    for b, (n, m) in enumerate(zip(lens, news)):
        for j in range(n - m, n):
            pid, off = c.row(b, j)
            for want, ws, src in ((want_k, want_ks, k), (want_v, want_vs, v)):
                if kind == "int8":
                    x = src[t].float().cpu().numpy()
                    s = (np.abs(x).max(-1) / np.float32(127)).astype(np.float32)
                    safe = np.where(s == 0, np.float32(1), s)
                    code = np.where(s[:, None] == 0, 0, np.rint((x / safe[:, None]).astype(np.float32)))
                    want[pid, :, off] = torch.from_numpy(code.astype(np.int8)).to(DEV)
                    ws[pid, :, off] = torch.from_numpy(s)
                else:
                    want[pid, :, off] = src[t]
            t += 1
    q.kv_append(k, v, *c.args(), **c.kw)
    assert q.device_error() == 0
    assert torch.equal(bits(c.k), bits(want_k)) and torch.equal(bits(c.v), bits(want_v))
    if kind == "int8":
        assert torch.equal(bits(c.kw["k_scale"].cpu()), bits(want_ks))
        assert torch.equal(bits(c.kw["v_scale"].cpu()), bits(want_vs))


def test_append_bad_pages_are_skipped(q):
    c = Cache([20, 20, 20], [2, 2, 2], 4, 2, 64, 16, stale=0.25)
    k, v = c.qkv[:, 4:6], c.qkv[:, 6:]
    c.table[1, 1] = c.k.shape[0]                           # one past the last page
    c.table[2, 1] = -1
    before = c.k.clone()
    pid = int(c.table[0, 1])
    q.kv_append(k, v, *c.args())
    assert q.device_error() == q.QW_ERR_BAD_INDEX and q.device_error() == 0
    before[pid, :, 2:4] = k[0:2].transpose(0, 1)
    assert torch.equal(bits(c.k), bits(before))
    # a length beyond the page table, and one shorter than the new tokens
    c = Cache([20, 20], [1, 3], 4, 2, 64, 16, stale=0.25)
    c.lens[0], c.lens[1] = 33, 2
    before = c.v.clone()
    q.kv_append(c.qkv[:, 4:6], c.qkv[:, 6:], *c.args())
    assert q.device_error() == q.QW_ERR_BAD_INDEX
    before[int(c.table[1, 0]), :, 0:2] = c.qkv[2:4, 6:].transpose(0, 1)
    assert torch.equal(bits(c.v), bits(before))


@pytest.mark.parametrize("kind", ["fp16", "int8"])
@pytest.mark.parametrize("cu", [[0, 2, 1, 6], [0, 900, 6, 6], [-1, 2, 4, 6], [0, 2, 4, 7], [5, 3, 1, 0], [0, 6, 6, 6, 6, 6, 6, 6, 5]])
def test_append_offsets_out_of_order(q, kind, cu):
    """Offsets that descend or leave 0 .. T are recorded; what is written stays in the named
    sequences' pages, and those alone."""
    B = len(cu) - 1
    c = Cache([20] * B, [6] + [0] * (B - 1), 4, 2, 64, 16, kind, stale=0.25, spare=5)
    c.cu.copy_(torch.tensor(cu, device=DEV))
    before = c.k.clone(), c.v.clone()
    q.kv_append(c.qkv[:, 4:6], c.qkv[:, 6:], *c.args(), **c.kw)
    assert q.device_error() == q.QW_ERR_BAD_INDEX and q.device_error() == 0
    spare = torch.ones(c.k.shape[0], dtype=torch.bool, device=DEV)
    spare[c.table.flatten().long()] = False
    assert int(spare.sum()) == 5
    for x, w in zip((c.k, c.v), before):
        assert torch.equal(bits(x[spare]), bits(w[spare]))


def test_append_tokens_of_no_sequence(q):
    """Rows past cu_tokens[B] belong to nobody and are left out."""
    c = Cache([20], [3], 4, 2, 64, 16, stale=0.25)
    c.cu[1] = 2
    c.lens[0] = 19
    before = c.k.clone()
    q.kv_append(c.qkv[:, 4:6], c.qkv[:, 6:], *c.args())
    before[int(c.table[0, 1]), :, 1:3] = c.qkv[:2, 4:6].transpose(0, 1)
    assert q.device_error() == 0 and torch.equal(bits(c.k), bits(before))


@pytest.mark.parametrize("dtype,L,pages,Hkv,page,d,n", [
    (torch.float16, 3, 40, 4, 16, 256, 1), (torch.int8, 2, 50, 3, 1, 64, 20), (torch.bfloat16, 1, 30, 1, 7, 128, 15),
    (torch.int8, 4, 64, 5, 33, 128, 32), (torch.float16, 16, 20, 8, 64, 128, 10)])
@pytest.mark.parametrize("nhd", [False, True])
def test_copy_pages(q, dtype, L, pages, Hkv, page, d, n, nhd):
    g = torch.Generator(device=DEV).manual_seed(n)
    shape = (L, pages, page, Hkv, d) if nhd else (L, pages, Hkv, page, d)

    def pool():
        x = torch.randint(-128, 128, shape, generator=g, device=DEV, dtype=torch.int8).to(dtype)
        return x.transpose(2, 3) if nhd else x
    pools = [pool(), pool()]
    if dtype == torch.int8:
        pools += [torch.rand(L, pages, Hkv, page, generator=g, device=DEV) for _ in range(2)]
    pairs = torch.randperm(pages, generator=g, device=DEV)[:2 * n].int().view(n, 2).contiguous()
    want = [x.clone() for x in pools]
    for s, e in pairs.tolist():
        for x in want:
            x[:, e] = x[:, s]
    q.kv_copy_pages(pairs, *pools)
    assert q.device_error() == 0
    for x, w in zip(pools, want):
        assert torch.equal(bits(x), bits(w))


def test_copy_one_layer_and_bad_pairs(q):
    x = torch.randn(10, 2, 16, 64, device=DEV, dtype=torch.float16)
    want = x.clone()
    want[7] = x[2]
    pairs = torch.tensor([[2, 7], [3, 10], [-1, 4], [5, 5]], dtype=torch.int32, device=DEV)
    q.kv_copy_pages(pairs, x)
    assert q.device_error() == q.QW_ERR_BAD_INDEX
    assert torch.equal(bits(x), bits(want))
    q.kv_copy_pages(pairs[:0], x)                          # nothing to copy
    # pages that are not dense blocks are refused
    with pytest.raises(ValueError):
        q.kv_copy_pages(pairs, torch.zeros(10, 2, 16, 128, device=DEV, dtype=torch.float16)[..., :64])
    with pytest.raises(ValueError):
        q.kv_copy_pages(pairs, x[0, 0])


def test_copy_offsets_past_4_gib(q):
    """Pages beyond 2^32 bytes of a pool, and a row offset beyond 2^31 elements in append."""
    pages = 2100
    k = torch.zeros(pages, 8, 512, 256, device=DEV, dtype=torch.float16)       # 2 MiB a page, 4.4 GB
    v = torch.zeros_like(k)
    k[1] = 1.5
    pairs = torch.tensor([[1, pages - 1]], dtype=torch.int32, device=DEV)
    q.kv_copy_pages(pairs, k)
    new = torch.randn(1, 8, 256, device=DEV, dtype=torch.float16)
    i32 = dict(dtype=torch.int32, device=DEV)
    table = torch.tensor([[pages - 1]], **i32)
    lens, cu = torch.tensor([512], **i32), torch.tensor([0, 1], **i32)
    q.kv_append(new, new, k, v, table, lens, cu)
    assert q.device_error() == 0
    assert bool((k[pages - 1, :, :511] == 1.5).all()) and torch.equal(k[pages - 1, :, 511], new[0])
    assert torch.equal(v[pages - 1, :, 511], new[0]) and float(k[2:pages - 1].abs().max()) == 0.0
    # and the attention reads them there: one key's weight is spread over 512 equal ones
    k[pages - 1], v[pages - 1] = 0.25, 0.5
    out = q.attn_paged(new.expand(1, 8, 256).contiguous(), k, v, table, lens, cu)
    assert q.device_error() == 0 and bool((out == 0.5).all())
