"""Plain binary64 forms of the paged cache's attention and of token log probabilities, and
builders of small cases -- test infrastructure only."""
import math

import torch

DEV = "cuda"


class Cache:
    """A paged cache with one batch's pages handed out in random order.  Every slot that
    holds no key of a sequence is filled with `stale` (NaN by default)."""

    def __init__(self, lens, news, Hq, Hkv, d, page, kind="fp16", nhd=False, seed=0, spare=3, stale=float("nan"),
                 extra_pages=0, v_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens_list, self.news, self.Hq, self.Hkv, self.d, self.page, self.kind = lens, news, Hq, Hkv, d, page, kind
        self.act = torch.bfloat16 if kind == "bf16" else torch.float16
        need = [-(-n // page) for n in lens]
        total = sum(need) + spare
        order = torch.randperm(total, generator=g).tolist()
        width = max(need + [1]) + extra_pages
        table = torch.zeros(len(lens), width, dtype=torch.int32)
        self.k64 = torch.full((total, Hkv, page, d), stale, dtype=torch.float64)
        self.v64 = self.k64.clone()
        self.ks = torch.full((total, Hkv, page), stale)
        self.vs = self.ks.clone()
        live = torch.zeros(total, page, dtype=torch.bool)
        at = 0
        for b, n in enumerate(lens):
            for i in range(need[b]):
                table[b, i] = order[at]
                live[order[at], :min(page, n - i * page)] = True
                at += 1
        live = live[:, None].expand(total, Hkv, page)
        m = int(live.sum())
        if kind == "int8":
            kc = torch.randint(-127, 128, (total, Hkv, page, d), generator=g, dtype=torch.int8)
            vc = torch.randint(-127, 128, (total, Hkv, page, d), generator=g, dtype=torch.int8)
            self.ks[live] = torch.rand(m, generator=g) * 0.02 + 0.004
            self.vs[live] = (torch.rand(m, generator=g) * 0.02 + 0.004) * v_scale
            self.k64 = kc.double() * self.ks.double()[..., None]
            self.v64 = vc.double() * self.vs.double()[..., None]
            k, v = kc, vc
        else:
            kv = torch.randn(2, m, d, generator=g).to(self.act)
            self.k64[live], self.v64[live] = kv[0].double(), kv[1].double() * v_scale
            k, v = self.k64.to(self.act), self.v64.to(self.act)
            self.k64, self.v64 = k.double(), v.double()

        def put(x):
            return x.transpose(1, 2).contiguous().to(DEV).transpose(1, 2) if nhd else x.to(DEV)
        self.k, self.v = put(k), put(v)
        self.kw = dict(k_scale=self.ks.to(DEV), v_scale=self.vs.to(DEV)) if kind == "int8" else {}
        self.k64, self.v64 = self.k64.to(DEV), self.v64.to(DEV)
        self.table = table.to(DEV)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        cu = [0]
        for x in news:
            cu.append(cu[-1] + x)
        self.cu, self.T = torch.tensor(cu, dtype=torch.int32, device=DEV), cu[-1]
        qkv = torch.randn(self.T, Hq + 2 * Hkv, d, generator=g).mul_(2.0).to(self.act).to(DEV)
        self.qkv, self.q = qkv, qkv[:, :Hq]                        # a slice: strided rows

    def row(self, b, j):
        """(page, row) of key j of sequence b."""
        return int(self.table[b, j // self.page]), j % self.page

    def args(self):
        return self.k, self.v, self.table, self.lens, self.cu

    def reference(self, window=0, sinks=0, scale=None):
        """(out, lse, bound of |x| terms per row, sum p |v| per element, keys seen)."""
        s = 1.0 / math.sqrt(self.d) if scale is None else scale
        G, T = self.Hq // self.Hkv, self.T
        out = torch.zeros(T, self.Hq, self.d, dtype=torch.float64, device=DEV)
        mag, lse = out.clone(), torch.full((T, self.Hq), -math.inf, dtype=torch.float64, device=DEV)
        dx = torch.zeros(T, self.Hq, dtype=torch.float64, device=DEV)
        vmax = torch.zeros(T, self.Hq, self.d, dtype=torch.float64, device=DEV)
        t = 0
        for b, (n, m) in enumerate(zip(self.lens_list, self.news)):
            for r in range(m):
                at = n - m + r
                keys = [j for j in range(max(at + 1, 0)) if not window or j > at - window or j < sinks]
                if keys:
                    keys = torch.tensor(keys, device=DEV)
                    pid, off = self.table[b].long()[keys // self.page], keys % self.page
                    k, v = self.k64[pid, :, off], self.v64[pid, :, off]          # [S, Hkv, d]
                    q = self.q[t].double().view(self.Hkv, G, self.d)
                    x = torch.einsum("hgd,khd->hgk", q, k) * s
                    p = torch.softmax(x, -1)
                    out[t] = torch.einsum("hgk,khd->hgd", p, v).reshape(self.Hq, self.d)
                    mag[t] = torch.einsum("hgk,khd->hgd", p, v.abs()).reshape(self.Hq, self.d)
                    vmax[t] = v.abs().amax(0)[:, None].expand(self.Hkv, G, self.d).reshape(self.Hq, self.d)
                    lse[t] = torch.logsumexp(x, -1).flatten()
                    dx[t] = (torch.einsum("hgd,khd->hgk", q.abs(), k.abs()).amax(-1) * abs(s)).flatten()
                t += 1
        return out, lse, dx, mag, vmax

    def tolerances(self, ref):
        """Elementwise bounds of out's and lse's error.  Half steps: u of the 16-bit type,
        e = 2^-24 of binary32.
          score: d products summed in binary32 (up to 2e a step, the tensor core may
            truncate), times the scale: dx_j <= 2 d e sum|q k| scale + 4 e |x|
          weight: relative error dx + ex2's 2^-22 + the rounding to 16 bits u
          sums: n / 16 steps of 2 e, and the join
          out: each weight's relative error times p |v|, the denominator's (no u), one
            rounding; fp16 weights below 2^-14 of the largest lose absolute 2^-25 each."""
        out, lse, dx, mag, vmax = ref
        u = torch.finfo(self.act).eps / 2
        e, n = 2.0 ** -24, max(self.lens_list + [1])
        score = (2 * self.d + 8) * e * dx
        w = score + 2.0 ** -22 + (n / 8 + 64) * e
        tol = (u + 2 * w)[..., None] * mag + u * out.abs() * (1 + 2.0 ** -6)
        if self.act == torch.float16:
            tol = tol + n * 2.0 ** -25 * vmax + 2.0 ** -25
        lt = score + 2.0 ** -22 + (n / 8 + 64) * e + 8 * e * torch.where(lse.isinf(), 0.0, lse.abs())
        return tol, lt


def logprobs_reference(x, tokens, k):
    """(logprob, entropy, lse, top_logprob, top_idx) of x [M, N], tokens [M, C], in binary64."""
    x = x.double()
    lse = torch.logsumexp(x, -1)
    none = torch.isneginf(x).all(-1)
    z = torch.where(none[:, None], torch.full_like(x, -math.inf), x - torch.where(none, 0.0, lse)[:, None])
    p = torch.exp(z)
    ent = -(p * torch.where(p == 0, torch.zeros_like(z), z)).sum(-1)
    idx = torch.sort(-(x + 0.0), dim=-1, stable=True).indices[:, :k]
    return z.gather(1, tokens.long()), ent, lse, z.gather(1, idx), idx.int()
