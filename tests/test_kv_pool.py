"""kv_pool on the host: page hand-out, references, forks with copy on write, truncation,
compaction, and refusals that leave everything as it was.  A pool is checked against a model
of the cache's contents: every page holds the tokens that were written to it, copies move
them, and each sequence must read back its own tokens."""
import random

import pytest

import int8_weight_quantized_int4_gb300 as q


@pytest.fixture(scope="module", autouse=True)
def built():
    from int8_weight_quantized_int4_gb300 import build
    build.build()


class Model:
    """Pages as lists of tokens beside a KvPool."""

    def __init__(self, n, page):
        self.pool, self.page = q.KvPool(n, page), page
        self.mem = [[None] * page for _ in range(n)]
        self.seqs = {}

    def copy(self, pairs):
        src, dst = [p[0] for p in pairs], [p[1] for p in pairs]
        assert len(set(dst)) == len(dst) and not set(src) & set(dst)
        for s, d in pairs:
            self.mem[d] = list(self.mem[s])

    def rows(self, s):
        table, lens = self.pool.table([s])
        assert int(lens[0]) == len(self.seqs[s]) == self.pool.length(s)
        return table[0].tolist()

    def extend(self, s, tokens):
        self.copy(self.pool.extend(s, len(tokens)))
        at = len(self.seqs[s])
        self.seqs[s] = self.seqs[s] + tokens
        pages = self.rows(s)
        for i, t in enumerate(tokens, at):
            self.mem[pages[i // self.page]][i % self.page] = t

    def check(self):
        for s, tokens in self.seqs.items():
            pages = self.rows(s)
            assert len(pages) == -(-len(tokens) // self.page) == self.pool.pages(s)
            assert [self.mem[pages[i // self.page]][i % self.page] for i in range(len(tokens))] == tokens
        live = {p for s in self.seqs for p in self.rows(s)}
        assert self.pool.free_pages() == len(self.mem) - len(live)


@pytest.mark.parametrize("page,seed", [(1, 0), (4, 1), (16, 2), (5, 3)])
def test_random_walk_keeps_every_sequence(page, seed):
    rng = random.Random(seed)
    m, tick = Model(60, page), 0
    for _ in range(600):
        ids = list(m.seqs)
        op = rng.random()
        if op < 0.15 or not ids:
            s = m.pool.add()
            assert s not in m.seqs
            m.seqs[s] = []
        elif op < 0.55:
            s = rng.choice(ids)
            new = [tick + i for i in range(rng.randint(0, 2 * page))]
            tick += len(new)
            free, before = m.pool.free_pages(), m.rows(s)
            try:
                m.extend(s, new)
            except q.QgemmError as e:
                assert e.code == q.QW_ERR_NO_PAGES
                assert m.pool.free_pages() == free and m.rows(s) == before
        elif op < 0.7:
            s = rng.choice(ids)
            c = m.pool.fork(s)
            assert c not in m.seqs
            m.seqs[c] = list(m.seqs[s])
        elif op < 0.8:
            s = rng.choice(ids)
            keep = rng.randint(0, len(m.seqs[s]))
            m.pool.truncate(s, keep)
            m.seqs[s] = m.seqs[s][:keep]
        elif op < 0.92:
            s = rng.choice(ids)
            m.pool.free(s)
            del m.seqs[s]
        else:
            most = rng.choice([None, 0, 1, 3])
            m.copy(m.pool.compact(most))
            if most is None:
                live = {p for s in m.seqs for p in m.rows(s)}
                assert live == set(range(len(live)))
        m.check()


def test_pages_are_handed_out_lowest_first_and_again_after_free():
    p = q.KvPool(8, 4)
    a, b = p.add(), p.add()
    assert p.extend(a, 9) == [] and p.extend(b, 4) == []
    assert p.table([a, b])[0].tolist() == [[0, 1, 2], [3, 0, 0]]
    p.free(a)
    assert p.extend(b, 4) == [] and p.table([b])[0].tolist() == [[3, 0]]
    assert p.free_pages() == 6


def test_fork_copies_only_a_partly_filled_last_page():
    p = q.KvPool(8, 4)
    a = p.add()
    p.extend(a, 6)                                  # pages 0, 1 (half full)
    c, e = p.fork(a), p.fork(a)
    assert p.free_pages() == 6
    assert p.extend(c, 1) == [[1, 2]]               # c writes to a copy
    assert p.extend(e, 1) == [[1, 3]]
    assert p.extend(a, 1) == []                     # the page is a's alone now
    p.extend(a, 1)                                  # page 1 full
    f = p.fork(a)
    assert p.extend(f, 1) == []                     # a full last page is not copied
    assert p.table([f])[0].tolist() == [[0, 1, 4]]


def test_refusals():
    for n, page in ((-1, 4), (4, 0), (4, -3), (4, (1 << 20) + 1)):
        with pytest.raises(q.QgemmError) as e:
            q.KvPool(n, page)
        assert e.value.code == q.QW_ERR_INVALID_ARG
    p = q.KvPool(3, 4)
    a = p.add()
    for call in (lambda: p.extend(7, 1), lambda: p.extend(a, -1), lambda: p.fork(-1), lambda: p.free(5),
                 lambda: p.truncate(a, 1), lambda: p.truncate(a, -1), lambda: p.table([a, 9]), lambda: p.length(3),
                 lambda: p.compact(-1)):
        with pytest.raises(q.QgemmError) as e:
            call()
        assert e.value.code == q.QW_ERR_INVALID_ARG
    with pytest.raises(q.QgemmError) as e:
        p.extend(a, 13)                             # four pages of three
    assert e.value.code == q.QW_ERR_NO_PAGES and p.free_pages() == 3 and p.length(a) == 0
    with pytest.raises(q.QgemmError) as e:
        p.extend(a, (1 << 31) - 1)
    assert e.value.code in (q.QW_ERR_UNSUPPORTED_SHAPE, q.QW_ERR_NO_PAGES)
    p.extend(a, 12)
    with pytest.raises(q.QgemmError) as e:
        p.table([a], max_pages=2)
    assert e.value.code == q.QW_ERR_UNSUPPORTED_SHAPE
    c = p.fork(a)
    p.truncate(c, 11)
    with pytest.raises(q.QgemmError) as e:
        p.extend(c, 1)                              # needs a page for the copy
    assert e.value.code == q.QW_ERR_NO_PAGES
    p.free(a)
    with pytest.raises(q.QgemmError):
        p.extend(a, 1)                              # freed
    assert p.extend(c, 1) == []                     # the page is c's alone again
    empty = q.KvPool(0, 16)
    s = empty.add()
    assert empty.extend(s, 0) == [] and empty.free_pages() == 0 and empty.compact() == []
    assert empty.table([s])[0].shape == (1, 0) and empty.table([])[1].shape == (0,)


def test_sizes_past_32_bits_are_refused():
    """ctypes takes an int modulo 2^32: 2^32 + 3 tokens would be 3."""
    pool = q.KvPool(10, 4)
    s = pool.add()
    assert pool.extend(s, 10) == []
    for call in (lambda: q.KvPool(2 ** 32 + 5, 4), lambda: q.KvPool(5, 2 ** 32 + 4), lambda: pool.extend(s, 2 ** 32 + 3),
                 lambda: pool.truncate(s, 2 ** 32 + 3), lambda: pool.length(2 ** 32 + s), lambda: pool.pages(2 ** 32 + s),
                 lambda: pool.fork(2 ** 32 + s), lambda: pool.free(2 ** 32 + s), lambda: pool.table([2 ** 32 + s])):
        with pytest.raises(ValueError):
            call()
    assert pool.length(s) == 10 and pool.pages(s) == 3 and pool.compact(2 ** 40) == []
