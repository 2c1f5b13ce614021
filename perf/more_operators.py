"""The operators of a verify step over trees of drafted tokens, as measured: attention of a
tree's nodes over a paged key-value cache, drawing a token a row of logits, the path of a tree
that the drawn tokens accept, and the accepted path's rows moved together in the cache.

`run(state)` is one pass through one operator.  With `own` false it computes the operator's
definition with elementary torch operations, in binary32 (drawing in binary64: a draw falls
next to a border of the distribution now and then); with `own` true it makes the calls of
int8_weight_quantized_int4_gb300 that a user makes.  `exact(case, seed)` is the definition
again in binary64, sequence by sequence.

Shared conventions (those of the package): a cache is k_pages, v_pages [pages, Hkv, page, d]
(any strides with d contiguous), page_table [B, max_pages] int32, seq_lens [B] int32 the
length of every sequence with its new tokens, cu_tokens [B + 1] int32 the offsets of each
sequence's new tokens, which are its last positions.  The new tokens are the nodes of a tree:
parents [T] int32 holds each node's parent as its place among the sequence's new tokens, always
an earlier one, -1 for a root.  Node 0 is the token that the last step drew.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"fp16": 2, "bf16": 2, "fp32": 4, "int8": 1}
VOCAB = 32000


# ------------------------------------------------------------------ the cases --
def listed():
    return [
        # one user, a short context, a small tree: latency
        {"name": "tree_one_1k_fp16", "op": "tree", "B": 1, "len": 1003, "nodes": 7, "Hq": 24, "Hkv": 4, "d": 256,
         "page": 16, "dtype": "fp16", "layout": "hnd", "window": 0, "sinks": 0, "lse": False},
        # a serving batch of ragged contexts, a tree of up to 24 nodes each
        {"name": "tree_batch_8k_bf16", "op": "tree", "B": 40, "len": 8190, "nodes": 24, "Hq": 32, "Hkv": 8, "d": 128,
         "page": 64, "dtype": "bf16", "layout": "nhd", "window": 0, "sinks": 0, "lse": False},
        # wide trees: the matrix products count as much as the reading
        {"name": "tree_wide_16k_fp16", "op": "tree", "B": 12, "len": 16384, "nodes": 64, "Hq": 24, "Hkv": 4, "d": 256,
         "page": 32, "dtype": "fp16", "layout": "hnd", "window": 0, "sinks": 0, "lse": True},
        # a few long contexts on the int8 cache
        {"name": "tree_long_64k_int8", "op": "tree", "B": 5, "len": 65535, "nodes": 13, "Hq": 24, "Hkv": 4, "d": 256,
         "page": 16, "dtype": "int8", "layout": "hnd", "window": 0, "sinks": 0, "lse": True},
        # the sampler of one user, every filter on
        {"name": "sample_one_fp16", "op": "sample", "M": 1, "N": 248320, "dtype": "fp16", "filters": "all", "masked": 0.0},
        # a token for every node of a batch's trees, nucleus sampling
        {"name": "sample_nodes_bf16", "op": "sample", "M": 768, "N": 50257, "dtype": "bf16", "filters": "topp",
         "masked": 0.0},
        # requests with settings of their own, greedy ones among them, binary32 logits after penalties, a grammar
        # hiding most of the vocabulary
        {"name": "sample_mixed_fp32", "op": "sample", "M": 64, "N": 128257, "dtype": "fp32", "filters": "mixed",
         "masked": 0.9},
        # the whole distribution
        {"name": "sample_plain_fp16", "op": "sample", "M": 200, "N": 32000, "dtype": "fp16", "filters": "none",
         "masked": 0.0},
        # the walk down one small tree: latency
        {"name": "accept_one", "op": "accept", "B": 1, "nodes": 7, "path": 7},
        # a large batch of wide trees
        {"name": "accept_batch", "op": "accept", "B": 500, "nodes": 64, "path": 24},
        # one user's accepted path in all layers
        {"name": "keep_one_fp16", "op": "keep", "B": 1, "len": 1003, "nodes": 7, "L": 16, "Hkv": 4, "d": 256, "page": 16,
         "dtype": "fp16", "layout": "hnd"},
        # a batch's accepted paths in all layers, int8 rows and their scales
        {"name": "keep_batch_int8", "op": "keep", "B": 64, "len": 400, "nodes": 64, "L": 48, "Hkv": 4, "d": 256,
         "page": 32, "dtype": "int8", "layout": "hnd"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 280)


def draw(rng):
    """One more case of the listed ranges; sizes are drawn again until the case costs no more
    than the largest listed one of its operator."""
    op = rng.choice(["tree", "tree", "tree", "sample", "sample", "sample", "accept", "keep"])
    top = max(_cost(c) for c in listed() if c["op"] == op)
    heads = [(24, 4), (32, 8), (64, 8), (8, 8), (16, 1), (40, 10), (6, 2)]
    while True:
        Hq, Hkv = rng.choice(heads)
        d = rng.choice([64, 128, 256])
        page = rng.choice([1, 8, 16, 16, 32, 48, 64, 128])
        layout = rng.choice(["hnd", "nhd"])
        nodes = _log(rng, 1, 64)
        if op == "tree":
            window = 0 if rng.random() < 0.7 else _log(rng, 16, 4096)
            c = {"op": op, "B": _log(rng, 1, 64), "len": nodes + _log(rng, 1, 65536), "nodes": nodes, "Hq": Hq,
                 "Hkv": Hkv, "d": d, "page": page, "dtype": rng.choice(["fp16", "bf16", "int8"]), "layout": layout,
                 "window": window, "sinks": rng.choice([0, 1, 4, 16]) if window else 0, "lse": rng.random() < 0.5}
            cells = c["B"] * (c["len"] + page) * max(Hkv * d, Hq * nodes)
        elif op == "sample":
            c = {"op": op, "M": _log(rng, 1, 1024), "N": _log(rng, 100, 262144),
                 "dtype": rng.choice(["fp16", "bf16", "fp32"]),
                 "filters": rng.choice(["none", "topk", "topp", "minp", "all", "mixed"]),
                 "masked": rng.choice([0.0, 0.0, 0.5, 0.98])}
            cells = 10 * c["M"] * c["N"]
        elif op == "accept":
            c = {"op": op, "B": _log(rng, 1, 500), "nodes": nodes, "path": rng.randint(1, nodes)}
            cells = c["B"] * nodes * nodes
        else:
            c = {"op": op, "B": _log(rng, 1, 64), "len": nodes + _log(rng, 1, 600), "nodes": nodes, "L": _log(rng, 1, 48),
                 "Hkv": Hkv, "d": d, "page": page, "dtype": rng.choice(["fp16", "bf16", "int8"]), "layout": layout}
            cells = c["L"] * c["B"] * (c["len"] + page) * Hkv * d
        if _cost(c) <= top and cells <= 1.3e9:
            return c


def _lens(case):
    """(context lengths with the nodes, nodes) of each sequence: given by the case alone.  A
    lone sequence has the full length and tree; a batch is ragged."""
    B, top, most = case["B"], case.get("len", case["nodes"]), case["nodes"]
    rng = random.Random(B * 1000003 + top * 101 + most)
    news = [most if B == 1 or i == 0 else rng.randint(max(1, most // 2), most) for i in range(B)]
    lens = [top if B == 1 or i == 0 else rng.randint(min(top, 6), top) for i in range(B)]
    return [max(n, m) for n, m in zip(lens, news)], news


def _seen(case):
    """Of each sequence, the cached keys before its tree that the tree's nodes can see together."""
    W, out = case["window"], []
    for n, m in zip(*_lens(case)):
        lo = max(0, n - m - W + 1) if W else 0
        out.append(n - m - lo + min(case["sinks"], lo))
    return out


def work(case):
    op = case["op"]
    if op == "tree":
        _, news = _lens(case)
        T, seen = sum(news), _seen(case)
        row = case["Hkv"] * (case["d"] * BYTES[case["dtype"]] + (4 if case["dtype"] == "int8" else 0))
        return {"bytes": 2 * (sum(seen) + T) * row + sum(-(-(s + m) // case["page"]) for s, m in zip(seen, news)) * 4
                + 2 * T * case["Hq"] * case["d"] * 2 + (4 * T * case["Hq"] if case["lse"] else 0) + 4 * T,
                "flops": 4 * case["Hq"] * case["d"] * sum((s + 1) * m for s, m in zip(seen, news))}
    if op == "sample":
        return {"bytes": case["M"] * case["N"] * BYTES[case["dtype"]] + 12 * case["M"], "flops": 4 * case["M"] * case["N"]}
    B, T = case["B"], sum(_lens(case)[1])
    if op == "accept":
        return {"bytes": 12 * T + 4 * B + 4 * B * (case["path"] + 2), "flops": 0}
    counts = _counts(case)
    row = case["d"] * BYTES[case["dtype"]] + (4 if case["dtype"] == "int8" else 0)
    return {"bytes": 2 * 2 * case["L"] * case["Hkv"] * (sum(counts) - B) * row + 4 * (2 * sum(counts) + 4 * B), "flops": 0}


def _counts(case):
    """Nodes of each sequence's accepted path: given by the case alone."""
    rng = random.Random(case["B"] * 7919 + case["nodes"])
    return [1 + min(max(m - 2, 0), rng.randint(1, 9)) for m in _lens(case)[1]]


# ------------------------------------------------------------------ the inputs --
def _randn(gen, *shape, dtype=torch.float16, scale=1.0):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32 if scale != 1.0 else dtype)
    return (x * scale).to(dtype) if scale != 1.0 else x


def _pool(gen, case, lead, pages):
    """One pool of pages (K or V): values, and for int8 the scale of every row."""
    shape = [*lead, pages, case["Hkv"], case["page"], case["d"]]
    if case["dtype"] == "int8":
        codes = torch.randint(-127, 128, shape, generator=gen, device="cuda", dtype=torch.int8)
        scale = torch.rand(shape[:-1], generator=gen, device="cuda") * 0.015 + 0.005
        return codes, scale
    if case["layout"] == "nhd":
        shape[-3], shape[-2] = shape[-2], shape[-3]
        return _randn(gen, *shape, dtype=DTYPES[case["dtype"]]).transpose(-3, -2), None
    return _randn(gen, *shape, dtype=DTYPES[case["dtype"]]), None


def _batch(gen, case):
    """Lengths, offsets and a page table over pages handed out in random order."""
    lens, news = _lens(case)
    need = [-(-n // case["page"]) for n in lens]
    total = sum(need) + 8
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    at = torch.tensor([0] + need, device="cuda").cumsum(0)
    col = torch.arange(max(need), device="cuda")[None]
    used = col < (at[1:] - at[:-1])[:, None]
    table = torch.where(used, order[(at[:-1, None] + col).clamp_max(total - 1)], torch.zeros_like(order[:1]))
    i32 = dict(device="cuda", dtype=torch.int32)
    return total, table.contiguous(), torch.tensor(lens, **i32), torch.tensor(np.cumsum([0] + news), **i32)


def _trees(case, seed):
    """Parents of all nodes, drafted tokens and the tokens drawn at the nodes, as a drafter and
    a model that agree about half of the time make them; host arrays.  A node hangs under one of
    the eight nodes before it."""
    rng = np.random.default_rng(seed)
    news = np.array(_lens(case)[1])
    start = np.repeat(np.cumsum(news) - news, news)
    T = int(news.sum())
    at = np.arange(T) - start
    parents = np.where(at == 0, -1, at - 1 - (rng.random(T) * np.minimum(at, 8)).astype(np.int64))
    tokens = rng.integers(0, VOCAB, T)
    tokens = np.where((rng.random(T) < 0.05) & (at > 1), np.roll(tokens, 1), tokens)    # equal siblings happen
    drawn = rng.integers(0, VOCAB, T)
    hit = np.flatnonzero((parents >= 0) & (rng.random(T) < 0.7))[::-1]
    drawn[(start + parents)[hit]] = tokens[hit]
    return [torch.from_numpy(x.astype(np.int32)) for x in (parents, tokens, drawn)]


def _settings(gen, case):
    """The sampler's settings: numbers for all rows, or tensors of one a row."""
    M, kind = case["M"], case["filters"]
    if kind != "mixed":
        return {"none": {}, "topk": {"temperature": 0.8, "top_k": 50}, "topp": {"temperature": 0.8, "top_p": 0.95},
                "minp": {"temperature": 1.1, "min_p": 0.02},
                "all": {"temperature": 0.7, "top_k": 200, "top_p": 0.95, "min_p": 0.01}}[kind]

    def pick(values, dtype=torch.float32):
        at = torch.randint(0, len(values), (M,), generator=gen, device="cuda")
        return torch.tensor(values, device="cuda", dtype=dtype)[at]

    return {"temperature": pick([0.0, 0.6, 0.8, 1.0, 1.2]), "top_k": pick([0, 0, 1, 20, 50, 1000], torch.int32),
            "top_p": pick([1.0, 1.0, 0.9, 0.95, 0.5]), "min_p": pick([0.0, 0.0, 0.05, 0.1])}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    if op == "sample":
        M, N = case["M"], case["N"]
        x = _randn(gen, M, N, dtype=torch.float32, scale=2.5)
        # a few dozen tokens stand out, as after any context
        at = torch.randint(0, N, (M, 64), generator=gen, device="cuda")
        x.scatter_reduce_(1, at, torch.rand((M, 64), generator=gen, device="cuda") * 12 + 4, "amax")
        if case["masked"]:
            hide = torch.rand((M, N), generator=gen, device="cuda") < case["masked"]
            hide[:, :1] = False
            x.masked_fill_(hide, float("-inf"))
        s["logits"] = x.to(DTYPES[case["dtype"]])
        s["u"] = torch.rand((M,), generator=gen, device="cuda")
        s["settings"] = _settings(gen, case)
        return s
    if op in ("tree", "keep"):
        pages, s["table"], s["lens"], s["cu"] = _batch(gen, case)
        lead = (case["L"],) if op == "keep" else ()
        s["k_pages"], s["k_scale"] = _pool(gen, case, lead, pages)
        s["v_pages"], s["v_scale"] = _pool(gen, case, lead, pages)
    else:
        s["cu"] = torch.tensor(np.cumsum([0] + _lens(case)[1]), device="cuda", dtype=torch.int32)
    if op != "keep":
        s["parents"], s["tokens"], s["drawn"] = (x.cuda() for x in _trees(case, seed))
    if op == "tree":
        # q is a slice of one projection's output, as a model has it
        act = DTYPES["fp16" if case["dtype"] == "int8" else case["dtype"]]
        T, Hq, d = s["parents"].shape[0], case["Hq"], case["d"]
        s["q"] = _randn(gen, T, Hq + 2 * case["Hkv"], d, dtype=act, scale=2.0)[:, :Hq]
        s["out"] = torch.empty((T, Hq, d), device="cuda", dtype=act)
        s["lse"] = torch.empty((T, Hq), device="cuda") if case["lse"] else None
    elif op == "keep":
        # accepted paths as tree_accept gives them: the root and some later nodes, none in its place yet
        rng, counts = random.Random(seed), _counts(case)
        path = [[0] + sorted(rng.sample(range(2, m), c - 1)) + [-1] * (case["nodes"] - c)
                for c, m in zip(counts, _lens(case)[1])]
        s["path"], s["count"] = (torch.tensor(x, device="cuda", dtype=torch.int32) for x in (path, counts))
    return s


# --------------------------------------------------------------- the plain forms --
def _nodes(s):
    """Of every node: its sequence, and its place in the tree."""
    cu = s["cu"].long()
    t = torch.arange(s["parents"].shape[0], device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    return b, t - cu[b]


def _padded(s, b, i, x, fill):
    out = torch.full((s["cu"].shape[0] - 1, s["case"]["nodes"]), fill, device="cuda", dtype=torch.long)
    out[b, i] = x.long()
    return out


def _above(parents):
    """[B, m, m]: whether node j is node i or one of its ancestors; parents [B, m], -1 for none.
    Steps up the tree double with each product."""
    m = parents.shape[1]
    j = torch.arange(m, device="cuda")
    up = ((parents[..., None] == j) | (j[:, None] == j)).float()
    for _ in range(max(1, (m - 1).bit_length())):
        up = (torch.matmul(up, up) > 0).float()
    return up > 0


def _plain_tree(s):
    c = s["case"]
    Hq, Hkv, d, page = c["Hq"], c["Hkv"], c["d"], c["page"]
    B, G, W, m = c["B"], c["Hq"] // c["Hkv"], c["window"], c["nodes"]
    b, i = _nodes(s)
    above = _above(_padded(s, b, i, s["parents"], -1))                       # [B, m, m]
    depth = above.sum(-1) - 1                                                # [B, m]
    lens, width = s["lens"].long(), s["table"].shape[1] * page
    n = s["cu"].long()[1:] - s["cu"].long()[:-1]
    pos0 = lens - n
    # the slots that are read: the whole table, or the sinks and those from the window's start
    j = torch.arange(width, device="cuda").expand(B, width)
    far = torch.zeros_like(j, dtype=torch.bool)
    if W:
        first = (pos0 - W + 1).clamp_min(0)
        near = first[:, None] + torch.arange(W + m, device="cuda")
        sink = torch.arange(c["sinks"], device="cuda").expand(B, c["sinks"])
        j = torch.cat([sink, near], 1)
        far = torch.cat([sink >= first[:, None], torch.zeros_like(near, dtype=torch.bool)], 1)   # listed twice
        at_page, off = s["table"].long().gather(1, (j // page).clamp_max(s["table"].shape[1] - 1)), j % page
    S = j.shape[1]

    def context(pages, scale):
        if not W:                                                  # whole pages
            x = pages[s["table"].long()].float()                   # [B, max_pages, Hkv, page, d]
            if scale is not None:
                x = x * scale[s["table"].long()][..., None]
            return x.transpose(1, 2).reshape(B, Hkv, S, d)
        x = pages.transpose(1, 2)[at_page, off].float()            # [B, S, Hkv, d]
        if scale is not None:
            x = x * scale.transpose(1, 2)[at_page, off][..., None]
        return x.transpose(1, 2)

    q = torch.zeros((B, m, Hq, d), device="cuda")
    q[b, i] = s["q"].float()
    # slot j holds position j before the tree, and node j - pos0 in it
    node = (j - pos0[:, None]).clamp(0, m - 1)
    tree = (j >= pos0[:, None]) & (j < lens[:, None])
    pos = torch.where(tree, pos0[:, None] + depth.gather(1, node), j)[:, None]           # [B, 1, S]
    seen = torch.where(tree[:, None], above.gather(2, node[:, None].expand(B, m, S)), (j < pos0[:, None])[:, None])
    if W:
        at = (pos0[:, None] + depth)[..., None]
        seen = seen & ~far[:, None] & ((pos > at - W) | (pos < c["sinks"]))
    seen = seen[:, None, :, None]                                  # [B, 1, m, 1, S]
    x = q.view(B, m, Hkv, G, d).transpose(1, 2).reshape(B, Hkv, m * G, d)
    x = torch.matmul(x, context(s["k_pages"], s["k_scale"]).transpose(-1, -2)).view(B, Hkv, m, G, S) / math.sqrt(d)
    x = x.masked_fill(~seen, float("-inf"))
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p = torch.exp(x - top)
    total = p.sum(-1)
    o = torch.matmul(p.view(B, Hkv, m * G, S), context(s["v_pages"], s["v_scale"])).view(B, Hkv, m, G, d)
    o = o / torch.where(total == 0, torch.ones_like(total), total)[..., None]
    out = o.permute(0, 2, 1, 3, 4).reshape(B, m, Hq, d)[b, i].to(s["out"].dtype)
    lse = (top[..., 0] + torch.log(total)).permute(0, 2, 1, 3).reshape(B, m, Hq)[b, i]
    return (out, lse) if c["lse"] else out


def _plain_sample(s):
    x, N = s["logits"].double(), s["logits"].shape[1]

    def setting(name, off):
        return torch.as_tensor(s["settings"].get(name, off), device="cuda", dtype=torch.float32).double().view(-1, 1)

    tau, k, top_p, min_p = (setting(*v) for v in (("temperature", 1.0), ("top_k", 0), ("top_p", 1.0), ("min_p", 0.0)))
    greedy = tau <= 0
    best = x.amax(1, keepdim=True)
    z = (x - best) / torch.where(greedy, torch.ones_like(tau), tau)
    z, order = torch.sort(z, dim=1, descending=True, stable=True)            # equal logits by their index
    w = torch.exp(z)
    rank = torch.arange(N, device="cuda")
    w = torch.where((k <= 0) | (rank < k), w, torch.zeros_like(w))
    before = w.cumsum(1) - w
    w = torch.where((top_p >= 1) | (before < top_p * w.sum(1, keepdim=True)) | (rank == 0), w, torch.zeros_like(w))
    w = torch.where((w >= min_p) | (rank == 0), w, torch.zeros_like(w))
    w = torch.where(greedy, (rank == 0).double().expand_as(w), w)
    w = torch.zeros_like(w).scatter_(1, order, w)                            # back in the order of the vocabulary
    sums = w.cumsum(1)
    total = sums[:, -1:]
    # the first token at which the sum passes u times the total, the last of all if rounding leaves none
    token = torch.searchsorted(sums, s["u"].double()[:, None] * total, right=True)
    token = torch.minimum(token, torch.where(w > 0, rank, torch.zeros_like(rank)).amax(1, keepdim=True))
    return {"token": token[:, 0].int(), "logprob": torch.log(w.gather(1, token) / total)[:, 0].float()}


def _plain_accept(s):
    width, m = s["case"]["path"], s["case"]["nodes"]
    b, i = _nodes(s)
    parents, tokens, drawn = (_padded(s, b, i, s[n], f) for n, f in (("parents", -1), ("tokens", -1), ("drawn", -2)))
    j = torch.arange(m, device="cuda")
    # accepted under its parent: drawn there, and no earlier child is the same token
    alike = (parents[:, :, None] == parents[:, None]) & (tokens[:, :, None] == tokens[:, None]) & (j < j[:, None])
    good = (parents >= 0) & (drawn.gather(1, parents.clamp_min(0)) == tokens) & ~alike.any(-1) | (j == 0)
    taken = ~(_above(parents) & ~good[:, None]).any(-1)
    n = s["cu"].long()[1:] - s["cu"].long()[:-1]
    taken &= j < n[:, None]
    count = taken.sum(1).clamp_max(width)
    path = torch.sort(torch.where(taken, j, m), 1).values[:, :width]
    path = torch.where(torch.arange(width, device="cuda") < count[:, None], path, -1)
    last = path.gather(1, (count - 1).clamp_min(0)[:, None]).clamp_min(0)
    return {"path": path.int(), "count": count.int(),
            "next_token": torch.where(count > 0, drawn.gather(1, last)[:, 0], -1).int()}


def _pools(s):
    return [s[n] for n in ("k_pages", "v_pages", "k_scale", "v_scale") if s[n] is not None]


def _plain_keep(s):
    page, path, count = s["case"]["page"], s["path"].long(), s["count"].long()
    pos0 = s["lens"].long() - (s["cu"].long()[1:] - s["cu"].long()[:-1])
    b, i = torch.nonzero(torch.arange(path.shape[1], device="cuda") < count[:, None], as_tuple=True)
    src, dst = pos0[b] + path[b, i], pos0[b] + i
    ps, pd = s["table"].long()[b, src // page], s["table"].long()[b, dst // page]
    for x in _pools(s):
        x[:, pd, :, dst % page] = x[:, ps, :, src % page]
    return _pools(s), (pos0 + count).int()


# ----------------------------------------------------------- the package's operators --
def _own_tree(s):
    import int8_weight_quantized_int4_gb300 as q
    c = s["case"]
    return q.attn_tree(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["cu"], s["parents"],
                       max_nodes=c["nodes"], window=c["window"], sinks=c["sinks"], k_scale=s["k_scale"],
                       v_scale=s["v_scale"], out=s["out"], lse=s["lse"])


def _own_sample(s):
    import int8_weight_quantized_int4_gb300 as q
    r = q.sample_tokens(s["logits"], s["u"], **s["settings"])
    return {"token": r.token, "logprob": r.logprob}


def _own_accept(s):
    import int8_weight_quantized_int4_gb300 as q
    r = q.tree_accept(s["tokens"], s["drawn"], s["parents"], s["cu"], max_path=s["case"]["path"])
    return {"path": r.path, "count": r.count, "next_token": r.next_token}


def _own_keep(s):
    import int8_weight_quantized_int4_gb300 as q
    new_lens = q.kv_keep_path(s["path"], s["count"], s["table"], s["lens"], s["cu"], *_pools(s))
    return _pools(s), new_lens


_PLAIN = {"tree": _plain_tree, "sample": _plain_sample, "accept": _plain_accept, "keep": _plain_keep}
_OWN = {"tree": _own_tree, "sample": _own_sample, "accept": _own_accept, "keep": _own_keep}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# -------------------------------------------------------------- the definition, binary64 --
def _walk(parents, i):
    """Node i and its ancestors, from the root down."""
    line = [i]
    while parents[line[-1]] >= 0:
        line.append(parents[line[-1]])
    return line[::-1]


def _exact_tree(case, s):
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["out"].shape[:2], float("-inf"), dtype=torch.float64, device="cuda")
    parents, t, W = s["parents"].tolist(), 0, case["window"]
    for b, (n, m) in enumerate(zip(*_lens(case))):
        pos0 = n - m
        lo = max(0, pos0 - W + 1) if W else 0
        keys = torch.cat([torch.arange(min(case["sinks"], lo)), torch.arange(lo, n)]).cuda()
        pid, off = s["table"][b].long()[keys // case["page"]], keys % case["page"]
        k, v = (s[p][pid, :, off].double() for p in ("k_pages", "v_pages"))              # [keys, Hkv, d]
        if case["dtype"] == "int8":
            k = k * s["k_scale"][pid, :, off].double()[..., None]
            v = v * s["v_scale"][pid, :, off].double()[..., None]
        see = np.zeros((m, len(keys)), dtype=bool)
        at = keys.cpu().numpy()
        for r in range(m):
            line = _walk(parents[t:t + m], r)
            pos = pos0 + len(line) - 1
            near = (lambda x: x > pos - W or x < case["sinks"]) if W else (lambda x: True)
            see[r] = (at < pos0) & ((at > pos - W) | (at < case["sinks"]) if W else True)
            see[r][[len(at) - m + a for e, a in enumerate(line) if near(pos0 + e)]] = True
        q = s["q"][t:t + m].double().view(m, case["Hkv"], -1, case["d"])
        z = torch.einsum("rhgd,khd->rhgk", q, k) / math.sqrt(case["d"])
        z = z.masked_fill(~torch.from_numpy(see).cuda()[:, None, None], float("-inf"))
        out[t:t + m] = torch.einsum("rhgk,khd->rhgd", torch.softmax(z, -1), v).reshape(m, case["Hq"], case["d"])
        lse[t:t + m] = torch.logsumexp(z, -1).reshape(m, case["Hq"])
        t += m
    return (out, lse) if case["lse"] else out


def _exact_sample(case, s):
    token, logprob = [], []
    rows = {n: (v.tolist() if torch.is_tensor(v) else [float(torch.tensor(v, dtype=torch.float32))] * case["M"])
            for n, v in s["settings"].items()}
    u = s["u"].tolist()
    for r in range(case["M"]):
        f = {n: v[r] for n, v in rows.items()}
        x = s["logits"][r].double().cpu().numpy()
        tau, k, p, mp = f.get("temperature", 1.0), int(f.get("top_k", 0)), f.get("top_p", 1.0), f.get("min_p", 0.0)
        if tau <= 0:
            token.append(int(x.argmax()))
            logprob.append(0.0)
            continue
        order = np.argsort(-x, kind="stable")
        w = np.exp((x[order] - x[order[0]]) / tau)
        keep = np.ones(len(w), dtype=bool)
        if k > 0:
            keep[k:] = False
        if p < 1:
            share = np.where(keep, w, 0.0)
            keep &= np.concatenate([[0.0], np.cumsum(share)[:-1]]) < p * share.sum()
        keep &= w >= mp
        keep[0] = True
        chosen = np.sort(order[keep])
        w = np.exp((x[chosen] - x.max()) / tau)
        sums = np.cumsum(w)
        j = min(int(np.searchsorted(sums, u[r] * sums[-1], side="right")), len(w) - 1)
        token.append(int(chosen[j]))
        logprob.append(math.log(w[j] / sums[-1]))
    return {"token": torch.tensor(token, dtype=torch.int32), "logprob": torch.tensor(logprob, dtype=torch.float64)}


def _exact_accept(case, s):
    parents, tokens, drawn = (s[n].tolist() for n in ("parents", "tokens", "drawn"))
    paths, counts, following, t = [], [], [], 0
    for m in _lens(case)[1]:
        path = [0]
        while len(path) < case["path"]:
            nxt = [i for i in range(m) if parents[t + i] == path[-1] and tokens[t + i] == drawn[t + path[-1]]]
            if not nxt:
                break
            path.append(nxt[0])
        paths.append(path + [-1] * (case["path"] - len(path)))
        counts.append(len(path))
        following.append(drawn[t + path[-1]])
        t += m
    return {n: torch.tensor(v, dtype=torch.int32) for n, v in
            (("path", paths), ("count", counts), ("next_token", following))}


def _exact_keep(case, s):
    out = [x.clone() for x in _pools(s)]
    table, path, count = (s[n].tolist() for n in ("table", "path", "count"))
    page, new = case["page"], []
    for b, (n, m) in enumerate(zip(*_lens(case))):
        pos0 = n - m
        for i in range(count[b]):
            j, k = pos0 + path[b][i], pos0 + i
            for x, y in zip(_pools(s), out):
                y[:, table[b][k // page], :, k % page] = x[:, table[b][j // page], :, j % page]
        new.append(pos0 + count[b])
    return [y if y.dtype == torch.int8 else y.double() for y in out], torch.tensor(new, dtype=torch.int32)


def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_tree, "sample": _exact_sample, "accept": _exact_accept, "keep": _exact_keep}[case["op"]](case, s)
