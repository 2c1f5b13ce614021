"""The operators around a decode or verify step, as measured: writing new tokens into a
paged key-value cache, copying its pages, attention over it, and the log probabilities of
given tokens.

`run(state)` is one pass through one operator.  With `own` false it computes the operator's
definition with elementary torch operations in binary32; with `own` true it makes the calls
of int8_weight_quantized_int4_gb300 that a user makes.  `exact(case, seed)` is the
definition again in binary64, sequence by sequence.

Shared conventions (those of the package): a cache is k_pages, v_pages [pages, Hkv, page, d]
(any strides with d contiguous), page_table [B, max_pages] int32, seq_lens [B] int32 the
length of every sequence with its new tokens, cu_tokens [B + 1] int32 the offsets of each
sequence's new tokens in q, k and v, which are its last positions.
"""
import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"fp16": 2, "bf16": 2, "fp32": 4, "int8": 1}


# ------------------------------------------------------------------ the cases --
def listed():
    return [
        # one decode step of a batch writes one token a sequence: a few hundred KB, latency counts
        {"name": "append_step_fp16", "op": "append", "B": 64, "len": 500, "new": 1, "Hq": 24, "Hkv": 4, "d": 256,
         "page": 16, "dtype": "fp16", "layout": "hnd"},
        # a chunk of prompts of several requests enters the cache
        {"name": "append_prompts_bf16", "op": "append", "B": 12, "len": 2500, "new": 1400, "Hq": 32, "Hkv": 8,
         "d": 128, "page": 64, "dtype": "bf16", "layout": "nhd"},
        # a fork writes to a shared last page: one page of every layer is copied
        {"name": "copy_fork_fp16", "op": "copy", "L": 16, "n": 1, "pages": 96, "Hkv": 4, "d": 256, "page": 16,
         "dtype": "fp16"},
        # compaction of a pool after many requests left
        {"name": "copy_compact_int8", "op": "copy", "L": 16, "n": 1000, "pages": 2500, "Hkv": 4, "d": 256,
         "page": 32, "dtype": "int8"},
        # one user, a short context: latency
        {"name": "attn_one_1k_fp16", "op": "attn", "B": 1, "len": 1003, "new": 1, "Hq": 24, "Hkv": 4, "d": 256,
         "page": 16, "dtype": "fp16", "layout": "hnd", "window": 0, "sinks": 0, "lse": False},
        # a serving batch of ragged contexts
        {"name": "attn_batch_8k_bf16", "op": "attn", "B": 64, "len": 8190, "new": 1, "Hq": 32, "Hkv": 8, "d": 128,
         "page": 64, "dtype": "bf16", "layout": "nhd", "window": 0, "sinks": 0, "lse": False},
        # few very long contexts on the int8 cache
        {"name": "attn_long_128k_int8", "op": "attn", "B": 4, "len": 131071, "new": 1, "Hq": 24, "Hkv": 4, "d": 256,
         "page": 16, "dtype": "int8", "layout": "hnd", "window": 0, "sinks": 0, "lse": True},
        # speculative verify: up to six tokens a sequence, a mixed batch
        {"name": "attn_verify_16k_fp16", "op": "attn", "B": 16, "len": 16384, "new": 6, "Hq": 24, "Hkv": 4, "d": 256,
         "page": 32, "dtype": "fp16", "layout": "hnd", "window": 0, "sinks": 0, "lse": True},
        # a sliding-window layer with sinks: only the window's pages and the first are read
        {"name": "attn_window_32k_fp16", "op": "attn", "B": 48, "len": 32768, "new": 1, "Hq": 64, "Hkv": 8, "d": 64,
         "page": 16, "dtype": "fp16", "layout": "hnd", "window": 1024, "sinks": 4, "lse": False},
        # the sampler of one user: the chosen token, entropy and 20 alternatives
        {"name": "logprobs_one_fp16", "op": "logprobs", "M": 1, "N": 248320, "C": 1, "k": 20, "dtype": "fp16",
         "masked": 0.0},
        # a batch after penalties in binary32, a grammar hiding most of the vocabulary
        {"name": "logprobs_batch_fp32", "op": "logprobs", "M": 64, "N": 128257, "C": 6, "k": 20, "dtype": "fp32",
         "masked": 0.9},
        # scoring a prompt: every position's next token, no alternatives
        {"name": "logprobs_prompt_bf16", "op": "logprobs", "M": 2048, "N": 50257, "C": 1, "k": 0, "dtype": "bf16",
         "masked": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ranges; sizes are drawn again until the case costs no more
    than the largest listed one of its operator."""
    op = rng.choice(["append", "copy", "attn", "attn", "attn", "logprobs", "logprobs"])
    top = max(work(c)["bytes"] for c in listed() if c["op"] == op)
    heads = [(24, 4), (32, 8), (64, 8), (8, 8), (16, 1), (40, 10), (6, 2)]
    while True:
        Hq, Hkv = rng.choice(heads)
        d = rng.choice([64, 128, 256])
        page = rng.choice([1, 8, 16, 16, 32, 48, 64, 128])
        layout = rng.choice(["hnd", "nhd"])
        if op == "append":
            new = 1 if rng.random() < 0.5 else _log(rng, 2, 1400)
            c = {"op": op, "B": _log(rng, 1, 64), "len": new + _log(rng, 1, 2000), "new": new, "Hq": Hq, "Hkv": Hkv,
                 "d": d, "page": page, "dtype": rng.choice(["fp16", "bf16"]), "layout": layout}
            cells = c["B"] * (c["len"] + page) * Hkv * d
        elif op == "copy":
            n = _log(rng, 1, 1000)
            c = {"op": op, "L": _log(rng, 1, 48), "n": n, "pages": 2 * n + _log(rng, 1, 500), "Hkv": Hkv, "d": d,
                 "page": page, "dtype": rng.choice(["fp16", "bf16", "int8"])}
            cells = c["L"] * c["pages"] * page * Hkv * d
        elif op == "attn":
            window = 0 if rng.random() < 0.6 else _log(rng, 16, 4096)
            c = {"op": op, "B": _log(rng, 1, 64), "len": _log(rng, 1, 131071),
                 "new": rng.choice([1, 1, 1, 2, 4, 6, 9]), "Hq": Hq, "Hkv": Hkv, "d": d, "page": page,
                 "dtype": rng.choice(["fp16", "bf16", "int8"]), "layout": layout, "window": window,
                 "sinks": rng.choice([0, 1, 4, 16]) if window else 0, "lse": rng.random() < 0.5}
            cells = c["B"] * (c["len"] + page) * max(Hkv * d, Hq * c["new"])
        else:
            c = {"op": op, "M": _log(rng, 1, 2048), "N": _log(rng, 100, 262144), "C": rng.choice([1, 1, 2, 6]),
                 "k": rng.choice([0, 1, 5, 20, 64]), "dtype": rng.choice(["fp16", "bf16", "fp32"]),
                 "masked": rng.choice([0.0, 0.0, 0.5, 0.98])}
            cells = c["M"] * c["N"]
        if work(c)["bytes"] <= top and cells <= 1.1e9:
            return c


def _lens(case):
    """(context lengths with the new tokens, new tokens) of each sequence: given by the case
    alone.  A lone sequence has the full length; a batch is ragged, from half a dozen tokens up."""
    B, top, new = case["B"], case["len"], case["new"]
    rng = random.Random(B * 1000003 + top * 101 + new)
    news = [new if B == 1 else rng.randint(1 if new < 8 else max(1, new // 8), new) for _ in range(B)]
    lens = [top if B == 1 or i == 0 else rng.randint(min(top, 6), top) for i in range(B)]
    return [max(n, m) for n, m in zip(lens, news)], news


def _visible(case):
    """Keys each sequence's new tokens can see together."""
    total = []
    for n, m in zip(*_lens(case)):
        if case["window"]:
            lo = max(0, n - m - case["window"] + 1)
            total.append(n - lo + min(case["sinks"], lo))
        else:
            total.append(n)
    return total


def work(case):
    op = case["op"]
    if op == "append":
        T = sum(_lens(case)[1])
        return {"bytes": 2 * 2 * T * case["Hkv"] * case["d"] * BYTES[case["dtype"]] + 4 * T + 8 * case["B"], "flops": 0}
    if op == "copy":
        return {"bytes": 2 * 2 * case["L"] * case["n"] * _page_bytes(case) + 8 * case["n"], "flops": 0}
    if op == "attn":
        lens, news = _lens(case)
        T, seen = sum(news), _visible(case)
        row = case["Hkv"] * (case["d"] * BYTES[case["dtype"]] + (4 if case["dtype"] == "int8" else 0))
        return {"bytes": 2 * sum(seen) * row + sum(-(-s // case["page"]) for s in seen) * 4
                + 2 * T * case["Hq"] * case["d"] * 2 + (4 * T * case["Hq"] if case["lse"] else 0),
                "flops": 4 * case["Hq"] * case["d"] * sum(s * m for s, m in zip(seen, news))}
    out = case["M"] * (8 + 4 * case["C"] + 8 * case["k"]) + 8 * case["M"] * case["C"]
    return {"bytes": case["M"] * case["N"] * BYTES[case["dtype"]] + out, "flops": 4 * case["M"] * case["N"]}


def _page_bytes(case):
    rows = case["Hkv"] * case["page"]
    return rows * (case["d"] * BYTES[case["dtype"]] + (4 if case["dtype"] == "int8" else 0))


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
    if case.get("layout") == "nhd":
        shape[-3], shape[-2] = shape[-2], shape[-3]
        return _randn(gen, *shape, dtype=DTYPES[case["dtype"]]).transpose(-3, -2), None
    return _randn(gen, *shape, dtype=DTYPES[case["dtype"]]), None


def _batch(gen, case):
    """Lengths, offsets and a page table over pages handed out in random order."""
    lens, news = _lens(case)
    need = [-(-n // case["page"]) for n in lens]
    total = sum(need) + 8
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    width = max(need)
    at = torch.tensor([0] + need, device="cuda").cumsum(0)
    col = torch.arange(width, device="cuda")[None]
    used = col < (at[1:] - at[:-1])[:, None]
    table = torch.where(used, order[(at[:-1, None] + col).clamp_max(total - 1)], torch.zeros_like(order[:1]))
    cu = [0]
    for m in news:
        cu.append(cu[-1] + m)
    i32 = dict(device="cuda", dtype=torch.int32)
    return total, table.contiguous(), torch.tensor(lens, **i32), torch.tensor(cu, **i32), cu[-1]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    if op in ("append", "attn"):
        pages, s["table"], s["lens"], s["cu"], T = _batch(gen, case)
        s["k_pages"], s["k_scale"] = _pool(gen, case, (), pages)
        s["v_pages"], s["v_scale"] = _pool(gen, case, (), pages)
        # q, k and v are the slices of one projection's output, as a model has them
        act = DTYPES["fp16" if case["dtype"] == "int8" else case["dtype"]]
        Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
        qkv = _randn(gen, T, Hq + 2 * Hkv, d, dtype=act, scale=2.0)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        if op == "attn":
            s["out"] = torch.empty((T, Hq, d), device="cuda", dtype=act)
            s["lse"] = torch.empty((T, Hq), device="cuda") if case["lse"] else None
    elif op == "copy":
        s["k_pages"], s["k_scale"] = _pool(gen, case, (case["L"],), case["pages"])
        s["v_pages"], s["v_scale"] = _pool(gen, case, (case["L"],), case["pages"])
        order = torch.randperm(case["pages"], generator=gen, device="cuda").to(torch.int32)
        s["pairs"] = order[:2 * case["n"]].view(case["n"], 2).contiguous()
    else:
        M, N = case["M"], case["N"]
        s["logits"] = _randn(gen, M, N, dtype=DTYPES[case["dtype"]], scale=3.0)
        if case["masked"]:
            hide = torch.rand((M, N), generator=gen, device="cuda") < case["masked"]
            hide[:, :1] = False
            s["logits"].masked_fill_(hide, float("-inf"))
        s["tokens"] = torch.randint(0, N, (M, case["C"]), generator=gen, device="cuda")
    return s


# --------------------------------------------------------------- the plain forms --
def _new_tokens(s):
    """Of every new token: its sequence, its place among that sequence's new tokens, its position."""
    cu, lens = s["cu"].long(), s["lens"].long()
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    return b, t - cu[b], lens[b] - (cu[b + 1] - cu[b]) + t - cu[b]


def _plain_append(s):
    page = s["case"]["page"]
    b, _, pos = _new_tokens(s)
    pid, off = s["table"].long()[b, pos // page], pos % page
    s["k_pages"][pid, :, off] = s["k"]
    s["v_pages"][pid, :, off] = s["v"]
    return s["k_pages"], s["v_pages"]


def _plain_copy(s):
    src, dst = s["pairs"].long().unbind(1)
    pools = [s[n] for n in ("k_pages", "v_pages", "k_scale", "v_scale") if s[n] is not None]
    for x in pools:
        x[:, dst] = x[:, src]
    return pools


def _plain_attn(s):
    c = s["case"]
    Hq, Hkv, d, page = c["Hq"], c["Hkv"], c["d"], c["page"]
    B, G, W, m = c["B"], c["Hq"] // c["Hkv"], c["window"], c["new"]
    b, i, pos = _new_tokens(s)
    lens, width = s["lens"].long(), s["table"].shape[1] * page
    # the positions that are read: the whole table, or the sinks and the window
    j = torch.arange(width, device="cuda").expand(B, width)
    sink = torch.zeros_like(j, dtype=torch.bool)
    if W:
        first = (lens - (s["cu"][1:] - s["cu"][:-1]) - W + 1).clamp_min(0)
        near = first[:, None] + torch.arange(W + m - 1, device="cuda")
        far = torch.arange(c["sinks"], device="cuda").expand(B, c["sinks"])
        j = torch.cat([far, near], 1)
        sink = torch.cat([torch.ones_like(far, dtype=torch.bool), torch.zeros_like(near, dtype=torch.bool)], 1)
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
    at = torch.full((B, m), -1, device="cuda")
    at[b, i] = pos
    j, sink = j[:, None], sink[:, None]
    seen = j <= at[..., None]
    if W:
        seen &= sink | ((j > at[..., None] - W) & (j >= c["sinks"]))
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


def _plain_logprobs(s):
    x, k = s["logits"].float(), s["case"]["k"]
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    lse = top + torch.log(total)
    below = torch.where(e == 0, torch.zeros_like(x), x - top)
    entropy = torch.log(total) - (e * below).sum(-1, keepdim=True) / total
    out = {"logprob": x.gather(1, s["tokens"]) - lse, "entropy": entropy[:, 0], "lse": lse[:, 0]}
    if k:
        val, idx = torch.sort(x, dim=-1, descending=True, stable=True)
        out["top_logprob"], out["top_idx"] = val[:, :k] - lse, idx[:, :k].int()
    return out


# ----------------------------------------------------------- the package's operators --
def _own_append(s):
    import int8_weight_quantized_int4_gb300 as q
    q.kv_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["cu"])
    return s["k_pages"], s["v_pages"]


def _own_copy(s):
    import int8_weight_quantized_int4_gb300 as q
    pools = [s[n] for n in ("k_pages", "v_pages", "k_scale", "v_scale") if s[n] is not None]
    q.kv_copy_pages(s["pairs"], *pools)
    return pools


def _own_attn(s):
    import int8_weight_quantized_int4_gb300 as q
    c = s["case"]
    return q.attn_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["cu"], max_new=c["new"],
                        window=c["window"], sinks=c["sinks"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                        out=s["out"], lse=s["lse"])


def _own_logprobs(s):
    import int8_weight_quantized_int4_gb300 as q
    r = q.token_logprobs(s["logits"], s["tokens"], k=s["case"]["k"])
    out = {"logprob": r.logprob, "entropy": r.entropy, "lse": r.lse}
    if s["case"]["k"]:
        out["top_logprob"], out["top_idx"] = r.top_logprob, r.top_idx
    return out


_PLAIN = {"append": _plain_append, "copy": _plain_copy, "attn": _plain_attn, "logprobs": _plain_logprobs}
_OWN = {"append": _own_append, "copy": _own_copy, "attn": _own_attn, "logprobs": _own_logprobs}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# -------------------------------------------------------------- the definition, binary64 --
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "append":
        out, page, t = [s["k_pages"].double(), s["v_pages"].double()], case["page"], 0
        for b, (n, m) in enumerate(zip(*_lens(case))):
            keys = torch.arange(n - m, n, device="cuda")
            pid = s["table"][b].long()[keys // page]
            for x, new in zip(out, (s["k"], s["v"])):
                x[pid, :, keys % page] = new[t:t + m].double()
            t += m
        return tuple(out)
    if op == "copy":
        pools = [s[n] for n in ("k_pages", "v_pages", "k_scale", "v_scale") if s[n] is not None]
        out = [x.clone() for x in pools]
        src, dst = s["pairs"].cpu().T.tolist()
        for x, y in zip(pools, out):
            for u, w in zip(src, dst):
                y[:, w].copy_(x[:, u])
        return [y if y.dtype == torch.int8 else y.double() for y in out]
    if op == "attn":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(s["out"].shape[:2], float("-inf"), dtype=torch.float64, device="cuda")
        G, page, t = case["Hq"] // case["Hkv"], case["page"], 0
        for b, (n, m) in enumerate(zip(*_lens(case))):
            first = max(0, n - m - case["window"] + 1) if case["window"] else 0
            keys = torch.cat([torch.arange(min(case["sinks"], first)), torch.arange(first, n)]).cuda()
            pid, off = s["table"][b].long()[keys // page], keys % page
            k, v = (s[p][pid, :, off].double() for p in ("k_pages", "v_pages"))      # [keys, Hkv, d]
            if case["dtype"] == "int8":
                k = k * s["k_scale"][pid, :, off].double()[..., None]
                v = v * s["v_scale"][pid, :, off].double()[..., None]
            for r in range(m):
                at = n - m + r
                see = keys <= at
                if case["window"]:
                    see &= (keys > at - case["window"]) | (keys < case["sinks"])
                q = s["q"][t].double().view(case["Hkv"], G, -1)
                z = torch.einsum("hgd,khd->hgk", q, k) / math.sqrt(case["d"])
                z = z.masked_fill(~see, float("-inf"))
                out[t] = torch.einsum("hgk,khd->hgd", torch.softmax(z, -1), v).reshape(out[t].shape)
                lse[t] = torch.logsumexp(z, -1).flatten()
                t += 1
        return (out, lse) if case["lse"] else out
    x = s["logits"].double()
    z = torch.log_softmax(x, -1)
    p = torch.exp(z)
    out = {"logprob": z.gather(1, s["tokens"]), "lse": torch.logsumexp(x, -1),
           "entropy": -(p * torch.where(p == 0, torch.zeros_like(z), z)).sum(-1)}
    if case["k"]:
        idx = torch.sort(-x, dim=-1, stable=True).indices[:, :case["k"]]
        out["top_logprob"], out["top_idx"] = z.gather(1, idx), idx.int()
    return out
