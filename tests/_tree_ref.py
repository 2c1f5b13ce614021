"""Plain definitions, in Python and numpy, of what a verify step over trees of drafted tokens
computes beside the attention: the draw of a token, the accepted path, the rows that move."""
import math

import numpy as np


def draw(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, log probability) of one row x (float64; NaN as -inf) in binary64."""
    x = np.where(np.isnan(x), -np.inf, x)
    top = x.max()
    if top == -np.inf:
        return -1, -math.inf
    order = np.argsort(-x, kind="stable")
    if not temperature > 0:
        return int(order[0]), 0.0
    with np.errstate(invalid="ignore", over="ignore"):
        d = np.where(x == top, 0.0, x - top)
        w = np.where(x == -np.inf, 0.0, np.exp(d / temperature))[order]
    keep = np.ones(len(w), bool)
    if 0 < top_k < len(w):
        keep[top_k:] = False
    if top_p < 1:
        share = np.where(keep, w, 0.0)
        keep &= np.cumsum(share) - share < top_p * share.sum()
    if min_p > 0:
        keep &= w >= min_p
    keep[0] = True
    kept = np.zeros(len(w))
    kept[order[keep]] = w[keep]
    sums = np.cumsum(kept)
    j = int(np.searchsorted(sums, min(max(u, 0.0), 1.0) * sums[-1], side="right"))
    if j == len(w):
        j = int(np.flatnonzero(kept)[-1])
    return j, math.log(kept[j] / sums[-1])


def draws(x, u, eps=1e-7, **kw):
    """Every answer of draw() for numbers within eps of u and, relatively, of top_p: {token: log probabilities}."""
    out = {}
    p = kw.pop("top_p", 1.0)
    for dp in ((0.0,) if p >= 1 or p <= 0 else (0.0, -eps, eps)):
        for du in (0.0, -eps, eps):
            t, lp = draw(x, u + du, top_p=p * (1 + dp), **kw)
            out.setdefault(t, []).append(lp)
    return out


def accept(tokens, drawn, parents, max_path):
    """(path, next token) of one sequence's tree; lists."""
    if not tokens:
        return [], -1
    path = [0]
    while len(path) < max_path:
        at = path[-1]
        kids = [i for i in range(at + 1, len(tokens)) if parents[i] == at and tokens[i] == drawn[at]]
        if not kids:
            break
        path.append(kids[0])
    return path, drawn[path[-1]]


def tree(rng, n, spread=6, roots=1):
    """Parents of a random tree: a node hangs under one of the `spread` before it."""
    return [-1 if i < roots else max(0, i - 1 - int(rng.integers(min(i, spread)))) for i in range(n)]


def ancestors(parents, i):
    """Node i and its ancestors, the root first."""
    line = [i]
    while 0 <= parents[line[-1]] < line[-1]:
        line.append(parents[line[-1]])
    return line[::-1]
