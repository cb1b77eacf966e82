"""Plain forms of windowed attention's masks, page weights, eviction by weight and draft
verification, for the tests: exact integers and fractions where the result is a choice,
64 bits elsewhere."""
import math
from fractions import Fraction

import torch

import _pages as P


def window_mask(L, T, tree, t, window, n_sink):
    """Bool [L]: the positions that query token t sees."""
    seen = P.seen_mask(L, T, tree, t)
    at = L - T + t if tree is None else L - T + bin(int(tree[t]) & ((1 << T) - 1)).count("1") - 1
    pos = torch.arange(L)
    return seen & ((pos > at - window) | (pos < n_sink))


def page_weights(q, lse, kv, seen, scale):
    """q [T][H][576], lse [T][H], kv [L][576], seen [T][L], all float64: each page's sum, and a bound
    on |scale q.k|, on |lse| and on the keys' absolute sums."""
    T, H = q.shape[:2]
    L = kv.shape[0]
    got = torch.zeros(-(-L // 64) * 64, dtype=torch.float64, device=q.device)
    for t in range(T):
        ok = torch.isfinite(lse[t])
        k = seen[t].nonzero().squeeze(1)
        x = torch.exp(q[t][ok] @ kv[k].T * scale - lse[t][ok][:, None])
        got[k] += x.sum(0)
    return got.view(-1, 64).sum(1)


def weights_tolerance(want, q, lse, kv, scale, fp8):
    """Relative: a score's 32-bit sum is off by at most 2^-16 of |q||k| (as in
    _pages.check_attention); FP8: query values are off by at most 2^-17.8 of their row's largest;
    the scales, the product with them and the difference with lse round to 2^-24 of their
    values, five roundings; the exponential is good to 2^-22; at most 140 nonnegative
    terms are added one after the other in 32 bits, then a few partial sums."""
    fin = torch.isfinite(lse)
    if not bool(fin.any()) or kv.shape[0] == 0:
        return torch.full_like(want, 1e-30)
    qf = q[fin]
    reach = abs(scale) * float(qf.norm(dim=1).max() * kv.norm(dim=1).max())
    e = reach * 2.0 ** -16 + 5 * 2.0 ** -24 * (reach + float(lse[fin].abs().max()))
    if fp8:
        e += abs(scale) * 2.0 ** -17.8 * float(qf.abs().max() * kv.abs().sum(1).max())
    return want.abs() * (math.expm1(e) + 2.0 ** -22 + 160 * 2.0 ** -24) + 1e-30


def evict(table, saved, weights, L, budget, n_first, n_last, saved_only):
    """table, saved: GPU and host blocks (-1: none); weights: floats. Returns the kept pages and the
    evicted ones, ascending."""
    n = -(-L // 64)
    there = [p for p in range(n) if table[p] >= 0]
    must = {p for p in there if p < n_first or p >= n - n_last or (saved_only and saved[p] < 0)}
    rest = [p for p in there if p not in must]
    key = {p: -math.inf if math.isnan(weights[p]) else weights[p] for p in rest}
    rest.sort(key=lambda p: (-key[p], p))
    stay = set(must) | set(rest if budget < 0 else rest[:max(0, budget - len(must))])
    return sorted(stay), [p for p in there if p not in stay]


def clean(x):
    """A probability as the verification takes it."""
    return 0.0 if math.isnan(x) or x <= 0 else min(x, 1.0)


def fixed(x):
    return math.floor(Fraction(clean(x)) * 2 ** 58)


def draw(values, u):
    """First index at which the sum of the integers passes u times the sum of all; -1: none."""
    total = min(sum(values), 2 ** 64 - 1)
    if total == 0:
        return -1
    u = Fraction(min(max(u, 0.0), 1 - 2.0 ** -24) if u == u else 0.0)
    run = 0
    for v, x in enumerate(values):
        run += x
        if run > u * total:
            return v
    raise AssertionError


def parents(T, tree):
    if tree is None:
        return [t - 1 for t in range(T)]
    out = []
    for t in range(T):
        above = int(tree[t]) & ((1 << t) - 1)
        out.append(above.bit_length() - 1)
    return out


def verify(tokens, p, q, tree, u):
    """tokens [T], p [T][V] and q [T-1][V] or None (nested lists of floats), tree [T] or None, u [T]:
    the path, and the next token."""
    T, V = len(tokens), len(p[0])
    par = parents(T, tree)
    ok = [0 <= x < V for x in tokens]
    uc = [Fraction(min(max(x, 0.0), 1 - 2.0 ** -24) if x == x else 0.0) for x in u]
    node, path = 0, [0]
    while True:
        row = p[node]
        left, gone, minus, go = Fraction(1), [], None, None
        for c in range(1, T):
            if par[c] != node or not ok[c]:
                continue
            x = tokens[c]
            pc = Fraction(0) if x in gone and q is None else Fraction(clean(row[x]))
            s = Fraction(clean(q[c - 1][x])) if q is not None else left
            if uc[c] * s < pc:
                go = c
                break
            if q is not None:
                minus = q[c - 1]
            else:
                left = max(left - pc, Fraction(0))
                gone.append(x)
        if go is None:
            break
        node = go
        path.append(go)
    whole = [fixed(x) for x in row]
    r = list(whole)
    if minus is not None:
        r = [max(a - fixed(b), 0) for a, b in zip(whole, minus)]
    for x in gone:
        r[x] = 0
    if sum(r) == 0:
        r = whole
    return path, draw(r, u[0])
