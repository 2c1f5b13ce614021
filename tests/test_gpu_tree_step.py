"""tree_accept and kv_keep_path against plain Python (tests/_tree_ref.py): exact."""
import numpy as np
import pytest
import torch

import int8_weight_quantized_int4_gb300 as q
from tests import _tree_ref as ref

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def forest(seed, news, vocab=4):
    """Trees of `news` nodes: few token ids, so paths are long and siblings equal."""
    rng = np.random.default_rng(seed)
    par, tok, drw = [], [], []
    for n in news:
        par.append(ref.tree(rng, n, spread=int(rng.integers(1, 9)), roots=int(rng.integers(1, 3))))
        tok.append(rng.integers(0, vocab, n).tolist())
        drw.append(rng.integers(0, vocab, n).tolist())
    return par, tok, drw


def flat(x):
    return i32([v for row in x for v in row])


@pytest.mark.parametrize("news", [[1], [7], [0], [2, 0, 5, 1], [64] * 9, [31, 32, 33, 63, 65, 128, 129, 200, 0, 1], [1000, 3], list(range(70))])
@pytest.mark.parametrize("vocab", [1, 2, 4, 30])
def test_accept(news, vocab):
    par, tok, drw = forest(len(news) + vocab, news, vocab)
    cu = np.cumsum([0] + news).tolist()
    for width in (1, 2, 5, 32, 33, 70):
        r = q.tree_accept(flat(tok), flat(drw), flat(par), i32(cu), max_path=width)
        want = [ref.accept(t, d, p, width) for t, d, p in zip(tok, drw, par)]
        assert r.count.tolist() == [len(p) for p, _ in want]
        assert r.next_token.tolist() == [n for _, n in want]
        assert r.path.tolist() == [p + [-1] * (width - len(p)) for p, _ in want]
    assert q.device_error() == 0


def test_accept_a_long_chain():
    n = 300
    tok = list(range(n))
    r = q.tree_accept(i32(tok), i32([t + 1 for t in tok]), i32([i - 1 for i in range(n)]), i32([0, n]), max_path=n)
    assert r.path[0].tolist() == tok and r.count.tolist() == [n] and r.next_token.tolist() == [n]


def test_accept_bad_parents_and_offsets():
    r = q.tree_accept(i32([5, 6, 7]), i32([6, 7, 7]), i32([-1, 0, 2]), i32([0, 3]), max_path=4)    # node 2 under itself
    assert r.path.tolist() == [[0, 1, -1, -1]] and r.next_token.tolist() == [7]
    assert q.device_error() == q.QW_ERR_BAD_INDEX
    q.tree_accept(i32([5, 6]), i32([6, 7]), i32([-1, -2]), i32([0, 2]), max_path=4)
    assert q.device_error() == q.QW_ERR_BAD_INDEX
    r = q.tree_accept(i32([5, 6]), i32([6, 9]), i32([-1, 0]), i32([0, 5]), max_path=4)             # past the end
    assert r.path.tolist() == [[0, 1, -1, -1]] and r.next_token.tolist() == [9]
    assert q.device_error() == q.QW_ERR_BAD_INDEX
    r = q.tree_accept(i32([]), i32([]), i32([]), i32([0, 0]), max_path=2)
    assert r.path.tolist() == [[-1, -1]] and r.count.tolist() == [0] and r.next_token.tolist() == [-1]
    assert q.tree_accept(i32([]), i32([]), i32([]), i32([0]), max_path=2).path.shape == (0, 2)
    assert q.device_error() == 0


# ---------------------------------------------------------------- keep path --
def step(seed, B, page, most, long):
    rng = np.random.default_rng(seed)
    news = [int(rng.integers(0, most + 1)) for _ in range(B)]
    lens = [n + int(rng.integers(0, long)) for n in news]
    need = [-(-n // page) for n in lens]
    order = rng.permutation(sum(need) + 3).tolist()
    table, at = np.zeros((B, max(need + [1])), dtype=np.int64), 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    paths = []
    for n in news:
        c = int(rng.integers(0, n + 1))
        paths.append(sorted(rng.choice(n, c, replace=False).tolist()))
    return news, lens, table, len(order), paths


@pytest.mark.parametrize("kind", ["fp16", "int8", "bf16"])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
@pytest.mark.parametrize("page,B,most,long,L,heads,d", [(16, 5, 20, 40, 3, 2, 64), (1, 3, 9, 5, 1, 1, 128), (48, 1, 70, 3, 5, 3, 256),
                                                         (8, 40, 7, 100, 2, 4, 128), (128, 4, 100, 300, 2, 1, 64)])
def test_keep(kind, layout, page, B, most, long, L, heads, d):
    news, lens, table, pages, paths = step(B + page, B, page, most, long)
    g = torch.Generator().manual_seed(page)

    def pool(dtype):
        shape = [L, pages, heads, page, d] if layout == "hnd" else [L, pages, page, heads, d]
        x = torch.randint(-100, 100, shape, generator=g).to(dtype).cuda()
        return x if layout == "hnd" else x.transpose(2, 3)
    dtype = dict(fp16=torch.float16, int8=torch.int8, bf16=torch.bfloat16)[kind]
    pools = [pool(dtype), pool(dtype)]
    if kind == "int8":
        pools += [torch.rand(L, pages, heads, page, generator=g).cuda() for _ in range(2)]
    want = [x.cpu().clone() for x in pools]
    old = [x.cpu().clone() for x in pools]
    for b in range(B):
        s = lens[b] - news[b]
        for i, a in enumerate(paths[b]):
            for x, y in zip(old, want):
                y[:, table[b][(s + i) // page], :, (s + i) % page] = x[:, table[b][(s + a) // page], :, (s + a) % page]
    width = max([len(p) for p in paths] + [1])
    path = i32([p + [-1] * (width - len(p)) for p in paths])
    args = path, i32([len(p) for p in paths]), i32(table.tolist()), i32(lens), i32(np.cumsum([0] + news).tolist())
    one_layer = [x[L // 2].clone() if kind == "int8" else x[L // 2] for x in pools]
    held = [x.clone() for x in pools]
    new = q.kv_keep_path(*args, *pools)
    assert new.tolist() == [n - m + len(p) for n, m, p in zip(lens, news, paths)]
    for x, y in zip(pools, want):
        assert torch.equal(x.cpu(), y)
    # one layer's pools without the leading dimension
    for x, h in zip(pools, held):
        x.copy_(h)
    single = [x[L // 2] for x in pools]
    q.kv_keep_path(*args, *single)
    for x, y, o in zip(pools, want, old):
        assert torch.equal(x[L // 2].cpu(), y[L // 2])
        for l in set(range(L)) - {L // 2}:
            assert torch.equal(x[l].cpu(), o[l])
    assert q.device_error() == 0 and one_layer is not None


def test_keep_bad_entries_move_nothing():
    x = torch.arange(4 * 1 * 4 * 64, dtype=torch.float16, device="cuda").view(4, 1, 4, 64)
    y = x.clone()
    table, lens, cu = i32([[0, 1, 2]]), i32([9]), i32([0, 6])             # slots 3 .. 8
    new = q.kv_keep_path(i32([[0, 2, 2, 9]]), i32([4]), table, lens, cu, x)  # 2 again, 9 is no node
    assert q.device_error() == q.QW_ERR_BAD_INDEX and new.tolist() == [7]
    y[1, 0, 0] = y[1, 0, 1]                                               # slot 4 takes slot 5
    assert torch.equal(x, y)
    assert q.kv_keep_path(i32([[0, 2]]), i32([7]), table, lens, cu, x).tolist() == [5]     # a count past the width
    assert q.device_error() == q.QW_ERR_BAD_INDEX
    y[1, 0, 0] = y[1, 0, 1]
    assert torch.equal(x, y)
    z = x.clone()
    q.kv_keep_path(i32([[0, 2]]), i32([2]), i32([[0, 7, 2]]), lens, cu, x)   # a page outside the pool
    assert q.device_error() == q.QW_ERR_BAD_INDEX and torch.equal(x, z)
    q.kv_keep_path(i32([[0, 2]]), i32([-1]), table, lens, cu, x)
    assert q.device_error() == q.QW_ERR_BAD_INDEX and torch.equal(x, z)
    assert q.kv_keep_path(i32([[0, 2]]), i32([2]), table, lens, cu).tolist() == [5]        # no pools: the lengths alone
    assert q.device_error() == 0


def test_keep_binding_refusals():
    x = torch.zeros(4, 1, 4, 64, dtype=torch.float16, device="cuda")
    ok = i32([[0, 2]]), i32([2]), i32([[0, 1, 2]]), i32([9]), i32([0, 6])
    with pytest.raises(ValueError):
        q.kv_keep_path(*ok, x.transpose(2, 3))                            # d not contiguous
    with pytest.raises(ValueError):
        q.kv_keep_path(*ok, x, torch.zeros(4, 1, 8, 64, device="cuda", dtype=torch.float16))
    with pytest.raises(ValueError):
        q.kv_keep_path(*ok, x.cpu())
    with pytest.raises(ValueError):
        q.kv_keep_path(*ok, x, x, x, x, x)
    with pytest.raises(TypeError):
        q.kv_keep_path(ok[0].long(), *ok[1:], x)
    with pytest.raises(ValueError):
        q.kv_keep_path(ok[0], i32([2, 2]), *ok[2:], x)
    with pytest.raises(TypeError):
        q.tree_accept(torch.zeros(3, device="cuda"), i32([1, 2, 3]), i32([-1, 0, 0]), i32([0, 3]), max_path=2)
    with pytest.raises(ValueError):
        q.tree_accept(i32([1, 2, 3]), i32([1, 2]), i32([-1, 0, 0]), i32([0, 3]), max_path=2)
    with pytest.raises(ValueError):
        q.tree_accept(i32([1]), i32([1]), i32([-1]), i32([0, 1]), max_path=0)


def test_keep_entries_in_their_place_that_do_not_ascend():
    """Entry 1 names slot 1, where it is, after an entry that did so already."""
    x = torch.arange(4 * 1 * 4 * 64, dtype=torch.float16, device="cuda").view(4, 1, 4, 64)
    table, lens, cu = i32([[0, 1, 2]]), i32([9]), i32([0, 6])             # slots 3 .. 8
    y = x.clone()
    y[0, 0, 3] = y[1, 0, 0]                                               # slot 3 takes slot 4
    new = q.kv_keep_path(i32([[1, 1]]), i32([2]), table, lens, cu, x)
    assert new.tolist() == [5] and torch.equal(x, y) and q.device_error() == q.QW_ERR_BAD_INDEX
    q.kv_keep_path(i32([[0, 1, 2]]), i32([3]), table, lens, cu, x)        # all in their place
    assert torch.equal(x, y) and q.device_error() == 0
