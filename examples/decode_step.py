"""A decode loop on the paged cache, from token ids to log probabilities: a small decoder of
random int4 weights whose layers attend over their caches, with a shared prompt, forked
continuations, a speculative verify step, and compaction of the pool.

    python examples/decode_step.py

One step of `Decoder.step` is what a serving loop runs: embedding gather, then per layer the
fused q/k/v projection, kv_append, attn_paged and the output projection, then the lm_head and
token_logprobs.  The weights are random (and there are no rotary angles or feed-forward
blocks), so the text means nothing; the cache's bookkeeping is the real one.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int8_weight_quantized_int4_gb300 as q  # noqa: E402

DEV = torch.device("cuda:0")


def _weights(n, k, gen, bits):
    lim = 7 if bits == 4 else 127
    codes = torch.randint(-lim, lim + 1, (n, k), generator=gen, dtype=torch.int8)
    size = (0.35 if bits == 4 else 0.06) / k ** 0.5
    scales = ((torch.rand(n, k // 128, generator=gen) + 0.5) * size)
    scales *= (torch.rand(n, k // 128, generator=gen) < 0.5).float() * 2 - 1
    pack = q.qpack_w4 if bits == 4 else q.qpack_w8
    return pack(codes.to(DEV), scales.half().to(DEV))


def _norm(x):
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).half()


class Decoder:
    """L attention layers over one pool of pages (16-bit or int8 cache)."""

    def __init__(self, vocab=1024, dim=512, layers=2, Hq=8, Hkv=2, d=64, pages=64, page=16, cache="fp16", seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.vocab, self.dim, self.L, self.Hq, self.Hkv, self.d = vocab, dim, layers, Hq, Hkv, d
        self.wqkv = [_weights((Hq + 2 * Hkv) * d, dim, gen, 4) for _ in range(layers)]
        self.wo = [_weights(dim, Hq * d, gen, 4) for _ in range(layers)]
        self.table_w8 = _weights(vocab, dim, gen, 8)               # embedding and lm_head
        self.pool = q.KvPool(pages, page)
        shape = (layers, pages, Hkv, page, d)
        dtype = torch.int8 if cache == "int8" else torch.float16
        self.k, self.v = (torch.zeros(shape, dtype=dtype, device=DEV) for _ in range(2))
        self.ks = self.vs = None
        if cache == "int8":
            self.ks, self.vs = (torch.zeros(shape[:-1], device=DEV) for _ in range(2))
        self.ws = q.Workspace(DEV)

    def _copy(self, pairs):
        if pairs:
            pools = [x for x in (self.k, self.v, self.ks, self.vs) if x is not None]
            q.kv_copy_pages(torch.tensor(pairs, dtype=torch.int32, device=DEV), *pools)

    def step(self, seqs, tokens, window=0, sinks=0):
        """Appends tokens[i] (a list) to sequence seqs[i]; returns the logits [T, vocab] after
        each of them, in order."""
        self._copy([p for s, t in zip(seqs, tokens) for p in self.pool.extend(s, len(t))])
        table, lens = self.pool.table(seqs)
        cu = [0]
        for t in tokens:
            cu.append(cu[-1] + len(t))
        batch = (table.to(DEV), lens.to(DEV), torch.tensor(cu, dtype=torch.int32, device=DEV))
        ids = torch.tensor([t for ts in tokens for t in ts], dtype=torch.int32, device=DEV)
        T, heads = ids.numel(), self.Hq + 2 * self.Hkv
        x = q.embed_gather_w8(ids, self.table_w8, self.vocab, self.dim)
        for i in range(self.L):
            qkv = q.qgemm_w4a16(_norm(x), self.wqkv[i], heads * self.d, self.dim, ws=self.ws).view(T, heads, self.d)
            qq, k, v = qkv[:, :self.Hq], qkv[:, self.Hq:self.Hq + self.Hkv], qkv[:, self.Hq + self.Hkv:]
            scales = {} if self.ks is None else dict(k_scale=self.ks[i], v_scale=self.vs[i])
            q.kv_append(k, v, self.k[i], self.v[i], *batch, **scales)
            o = q.attn_paged(qq, self.k[i], self.v[i], *batch, max_new=max(map(len, tokens)), window=window,
                             sinks=sinks, **scales)
            x = x + q.qgemm_w4a16(o.view(T, -1), self.wo[i], self.dim, self.Hq * self.d, ws=self.ws)
        return q.qgemm_w8a16(_norm(x), self.table_w8, self.vocab, self.dim, ws=self.ws)

    def score(self, logits, tokens, k=4):
        return q.token_logprobs(logits, torch.tensor(tokens, dtype=torch.int32, device=DEV), k=k)

    def compact(self):
        self._copy(self.pool.compact())


def generate(model, prompt, branches, length):
    """Continues the prompt in `branches` sequences: the i-th starts with the prompt's i-th most
    likely next token and goes on greedily.  Returns (sequences, their tokens, log probabilities)."""
    root = model.pool.add()
    logits = model.step([root], [prompt])
    best = model.score(logits[-1:], [0], k=branches)
    seqs = [root] + [model.pool.fork(root) for _ in range(branches - 1)]
    last = best.top_idx[0].tolist()
    total = best.top_logprob[0].clone()
    out = [[t] for t in last]
    for _ in range(length - 1):
        logits = model.step(seqs, [[t] for t in last])
        r = model.score(logits, [0] * branches, k=1)
        last = r.top_idx[:, 0].tolist()
        total += r.top_logprob[:, 0]
        for o, t in zip(out, last):
            o.append(t)
    return seqs, out, total


def main(cache="fp16"):
    model = Decoder(cache=cache)
    prompt = [(37 * i + 11) % model.vocab for i in range(41)]
    seqs, out, total = generate(model, prompt, branches=4, length=24)
    for o, p in zip(out, total.tolist()):
        print(f"log p {p:8.3f}  tokens {o[:8]} ...")
    # speculative verify: a draft's tokens in one step, then the rejected ones are dropped
    draft = out[1][:5]
    check = model.pool.add()
    model.step([check], [prompt + out[1][:1]])
    logits = model.step([check], [draft[1:]])
    r = model.score(logits, out[1][2:6])
    print("verify: log p of the draft's next tokens", [round(x, 3) for x in r.logprob.tolist()],
          "entropy", [round(x, 3) for x in r.entropy.tolist()])
    model.pool.truncate(check, len(prompt) + 3)
    # the others leave, the pool closes up, and the rest goes on
    for s in seqs[1:]:
        model.pool.free(s)
    model.compact()
    logits = model.step([seqs[0], check], [[out[0][-1]], [draft[3]]])
    torch.cuda.synchronize()
    assert q.device_error() == 0
    print("free pages", model.pool.free_pages(), "of", model.pool.num_pages)
    return model, out, logits


if __name__ == "__main__":
    main(*sys.argv[1:2])
