"""The operators of a verify step over trees of drafted tokens, run together over several steps as a
server runs them: kv_append, attn_tree, sample_tokens, tree_accept and kv_keep_path.

The model: keys, values and queries of a layer depend on a token and its position alone, so what
the cache holds after each step is known to the bit; logits are a product with the attention's
outputs."""
import math

import numpy as np
import pytest
import torch

import int8_weight_quantized_int4_gb300 as q
from tests import _tree_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
VOCAB, PLACES, LAYERS, HKV, GROUP, WIDTH = 9, 96, 2, 2, 3, 8
FILTERS = dict(temperature=0.8, top_k=5, top_p=0.97, min_p=0.01)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Model:
    def __init__(self, kind, d, page, B, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.act = torch.bfloat16 if kind == "bf16" else torch.float16
        self.d, self.page, self.int8 = d, page, kind == "int8"
        random = lambda *s: torch.randn(*s, generator=g, device=DEV)
        self.k, self.v = (random(LAYERS, VOCAB, PLACES, HKV, d).to(self.act) for _ in range(2))
        self.q = random(LAYERS, VOCAB, PLACES, HKV * GROUP, d).to(self.act)
        self.w = random(LAYERS * HKV * GROUP * d, VOCAB) * 0.3
        need = -(-PLACES // page)
        self.table = i32(rng.permutation(B * need).reshape(B, need))
        self.pools = self.cache(B * need)
        # what the cache makes of every row: all of them as one sequence
        n = VOCAB * PLACES
        rows = self.cache(-(-n // page))
        table = torch.arange(rows[0].shape[1], dtype=torch.int32, device=DEV)[None]
        for l in range(LAYERS):
            self.append(rows, l, self.k[l].flatten(0, 1), self.v[l].flatten(0, 1), table, i32([n]), i32([0, n]))
        order = torch.arange(n, device=DEV)
        self.rows = [x[:, order // page, :, order % page].transpose(0, 1).unflatten(1, (VOCAB, PLACES)) for x in rows]

    def cache(self, pages):
        dtype = torch.int8 if self.int8 else self.act
        x = [torch.full((LAYERS, pages, HKV, self.page, self.d), 77 if self.int8 else math.nan, dtype=dtype, device=DEV) for _ in range(2)]
        if self.int8:
            x += [torch.full((LAYERS, pages, HKV, self.page), math.nan, device=DEV) for _ in range(2)]
        return x

    def scales(self, pools, l):
        return dict(k_scale=pools[2][l], v_scale=pools[3][l]) if self.int8 else {}

    def append(self, pools, l, k, v, table, lens, cu):
        q.kv_append(k, v, pools[0][l], pools[1][l], table, lens, cu, **self.scales(pools, l))

    def step(self, pools, tokens, places, parents, u, lens, cu):
        outs = []
        for l in range(LAYERS):
            at = (l, tokens.long(), places.long())
            self.append(pools, l, self.k[at], self.v[at], self.table, lens, cu)
            outs.append(q.attn_tree(self.q[at], pools[0][l], pools[1][l], self.table, lens, cu, parents, max_nodes=16,
                                    **self.scales(pools, l)))
        logits = torch.cat(outs, 1).flatten(1).float() @ self.w
        drawn = q.sample_tokens(logits, u, **FILTERS)
        path = q.tree_accept(tokens, drawn.token, parents, cu, max_path=WIDTH)
        return outs, logits, drawn, path, q.kv_keep_path(path.path, path.count, self.table, lens, cu, *pools)

    def row64(self, i, l, token, place):
        """K (i = 0) or V (1) of tokens at places, as the cache holds them: [n, Hkv, d]."""
        x = self.rows[i][l, token, place].double()
        return x * self.rows[i + 2][l, token, place].double()[..., None] if self.int8 else x

    def check_attention(self, out, l, line, place):
        """out [Hq, d] of a node, line: the tokens up to it.  The error in units of e = 2^-24, as a node's
        scores (d products and a scale: (2 d + 8) e sum |q k|), weights (2^-22, their two 16-bit
        terms 2^-22, bf16 2^-16) and sums ((n / 8 + 64) e) allow, twice for the denominator, and one rounding."""
        n = len(line)
        tok, at = torch.tensor(line, device=DEV), torch.arange(n, device=DEV)
        k, v = self.row64(0, l, tok, at), self.row64(1, l, tok, at)
        x = self.q[l, line[-1], place].double().view(HKV, GROUP, self.d)
        s = torch.einsum("hgd,nhd->hgn", x, k) / math.sqrt(self.d)
        p = torch.softmax(s, -1)
        want = torch.einsum("hgn,nhd->hgd", p, v).flatten(0, 1)
        mag = torch.einsum("hgn,nhd->hgd", p, v.abs()).flatten(0, 1)
        dx = (torch.einsum("hgd,nhd->hgn", x.abs(), k.abs()).amax(-1) / math.sqrt(self.d)).flatten()[:, None]
        e = 2.0 ** -24
        w = (2 * self.d + 8) * e * dx + 2.0 ** -22 + (n / 8 + 64) * e
        term = 2.0 ** -16 if self.act == torch.bfloat16 else 2.0 ** -22
        tol = (term + 2 * w) * mag + torch.finfo(self.act).eps / 2 * want.abs() * (1 + 2.0 ** -6)
        tol = tol + n * 2.0 ** -32 * v.abs().amax() + 2.0 ** -25
        assert bool(((out.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("kind,d,page", [("fp16", 64, 16), ("bf16", 128, 8), ("int8", 128, 16), ("int8", 64, 7), ("fp16", 256, 5)])
@pytest.mark.parametrize("good", [False, True])
def test_steps_eager_and_replayed(kind, d, page, good):
    news, lens = [12, 1, 7, 16, 3, 0], [0, 1, 15, 16, 33, 20]
    B, T = len(news), sum(news)
    rng = np.random.default_rng(d + page)
    m = Model(kind, d, page, B, d + page)
    hist = [rng.integers(0, VOCAB, n).tolist() for n in lens]
    tok = torch.tensor(sum(hist, []), device=DEV)
    place = torch.tensor([i for n in lens for i in range(n)], device=DEV)
    for l in range(LAYERS):                        # the prompts
        m.append(m.pools, l, m.k[l, tok, place], m.v[l, tok, place], m.table, i32(lens), i32(np.cumsum([0] + lens)))
    cu = i32(np.cumsum([0] + news))
    other = [x.clone() for x in m.pools]           # stepped by a captured graph
    current = rng.integers(0, VOCAB, B).tolist()
    numbers = rng.random((B, PLACES)).astype(np.float32)
    static = [torch.zeros(T, dtype=torch.int32, device=DEV), torch.zeros(T, dtype=torch.int32, device=DEV),
              torch.full((T,), -1, dtype=torch.int32, device=DEV), torch.zeros(T, device=DEV), i32(lens)]
    graph, longest, moved = None, 0, 0
    for _ in range(9):
        trees = [ref.tree(rng, n, spread=3) for n in news]
        lines = [[ref.ancestors(t, i) for i in range(n)] for t, n in zip(trees, news)]
        tokens = [rng.integers(0, VOCAB, n).tolist() for n in news]
        for b in range(B):
            tokens[b][:1] = current[b:b + 1] if news[b] else []
        places = [[len(hist[b]) + len(line) - 1 for line in lines[b]] for b in range(B)]
        u = [numbers[b, p] for b in range(B) for p in places[b]]
        full = [len(hist[b]) + news[b] for b in range(B)]
        args = [i32(sum(tokens, [])), i32(sum(places, [])), i32(sum(trees, [])), torch.tensor(np.array(u), device=DEV), i32(full)]
        for _ in range(5 if good else 0):          # drafts that hit: the last child has the token drawn at its parent
            drawn_list, t = m.step([x.clone() for x in m.pools], *args, cu)[2].token.tolist(), 0
            for b in range(B):
                for i, parent in enumerate(trees[b]):
                    if parent >= 0 and parent not in trees[b][i + 1:]:
                        tokens[b][i] = drawn_list[t + parent]
                t += news[b]
            args[0] = i32(sum(tokens, []))
        outs, logits, drawn, path, left = m.step(m.pools, *args, cu)
        # the captured step, its inputs written over
        for x, y in zip(static, args):
            x.copy_(y)
        if graph is None:
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                replayed = m.step(other, *static, cu)
        graph.replay()
        torch.cuda.synchronize()
        assert q.device_error() == 0
        assert all(torch.equal(a, b) for a, b in zip(outs, replayed[0]))
        assert torch.equal(drawn.token, replayed[2].token) and torch.equal(drawn.logprob, replayed[2].logprob)
        assert all(torch.equal(a, b) for a, b in zip(path, replayed[3])) and torch.equal(left, replayed[4])
        # each stage from what the stage before it gave
        t = 0
        drawn_list, logits64 = drawn.token.tolist(), logits.double().cpu().numpy()
        for b in range(B):
            for i, line in enumerate(lines[b]):
                seen = hist[b] + [tokens[b][j] for j in line]
                for l in range(LAYERS):
                    m.check_attention(outs[l][t + i], l, seen, places[b][i])
                assert drawn_list[t + i] in ref.draws(logits64[t + i], float(u[t + i]), **FILTERS)
            want, following = ref.accept(tokens[b], drawn_list[t:t + news[b]], trees[b], WIDTH)
            assert path.path[b].tolist() == want + [-1] * (WIDTH - len(want)) and path.next_token[b] == following
            t += news[b]
            longest = max(longest, len(want))
            moved += sum(i != j for i, j in enumerate(want))
            hist[b] += [tokens[b][j] for j in want]
            current[b] = following
            assert left[b] == len(hist[b])
            # the cache: the accepted tokens' rows, one after another
            n = len(hist[b])
            at = torch.arange(n, device=DEV)
            line = torch.tensor(hist[b], device=DEV, dtype=torch.long)
            pid = m.table[b].long()[at // page]
            for pools in (m.pools, other):
                for x, y in zip(pools, m.rows):
                    assert torch.equal(x[:, pid, :, at % page], y[:, line, at].transpose(0, 1))
    assert not good or longest >= 4 and moved      # (else too little was accepted to show anything)
