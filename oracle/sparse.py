"""CPU oracle for attention over parts of a paged e4m3 cache (listed pages, shared prefixes), the
choice of pages and the bounds it goes by.  TEST INFRASTRUCTURE ONLY; imports nothing from the
product path.

Conventions of the cache: oracle/cache.py.  Every result comes as (O, LSE, W, Z) like cache.attend.
"""
from __future__ import annotations

import math

import numpy as np

from .cache import rows
from .fp8 import e4m3_decode


def _softmax(q, k, v, scale):
    """q [g, d], k, v [keys, d] -> O, LSE, W, Z of g rows that see all keys."""
    g, d = q.shape
    if len(k) == 0:
        return np.zeros((g, d)), np.full(g, -np.inf), np.zeros((g, d)), np.zeros(g)
    s = scale * (q @ k.T)
    m = s.max(axis=1, keepdims=True)
    p = np.exp(s - m)
    total = p.sum(axis=1, keepdims=True)
    p = p / total
    z = (scale * (np.abs(q) @ np.abs(k).T)).max(axis=1)
    return p @ v, (m + np.log(total))[:, 0], p @ np.abs(v), z


def _per_query(q, Hkv, keys_of, scale):
    """keys_of(h, t) -> (k, v) rows that packed query t sees on K/V head h."""
    q = np.asarray(q, dtype=np.float64)
    Hq, T, d = q.shape
    g = Hq // Hkv
    O, W = np.zeros((Hq, T, d)), np.zeros((Hq, T, d))
    L, Z = np.full((Hq, T), -np.inf), np.zeros((Hq, T))
    for h in range(Hkv):
        sl = slice(h * g, (h + 1) * g)
        for t in range(T):
            O[sl, t], L[sl, t], W[sl, t], Z[sl, t] = _softmax(q[sl, t], *keys_of(h, t), scale)
    return O, L, W, Z


def queries(cu, lens, causal):
    """[(sequence, keys it sees)] of every packed query."""
    out = []
    for b in range(len(lens)):
        n = int(cu[b + 1] - cu[b])
        out += [(b, int(lens[b]) - n + i + 1 if causal else int(lens[b])) for i in range(n)]
    return out


def attend_pages(q, c, pages, causal, scale):
    """Attention over the listed pages of c (cache_cases.filled's dict); pages [Hkv, T, count]."""
    P, Hkv = c["k_cache"].shape[2], c["k_cache"].shape[1]
    at = queries(c["cu"], c["lens"], causal)

    def keys_of(h, t):
        b, seen = at[t]
        out = [[], []]
        for j in pages[h][t]:
            n = min(P, seen - int(j) * P)
            if j < 0 or n <= 0:
                continue
            page = int(c["table"][b][j])
            for o, name in zip(out, ("k", "v")):
                o.append(e4m3_decode(c[name + "_cache"][page, h, :n]) * float(c[name + "_scale"][page, h]))
        d = c["k_cache"].shape[3]
        return tuple(np.concatenate(o) if o else np.zeros((0, d)) for o in out)

    return _per_query(q, Hkv, keys_of, scale)


def attend_prefix(q, c, prefix_table, cu_prefix, prefix_lens, causal, scale):
    """Attention over a shared prefix and a sequence's own keys, in the same cache."""
    Hkv = c["k_cache"].shape[1]
    at = queries(c["cu"], c["lens"], causal)
    group = np.repeat(np.arange(len(prefix_lens)), np.diff(cu_prefix))
    kept = {}

    def part(name, table, i, n, h):
        key = (name, id(table), i, h)
        if key not in kept or len(kept[key]) < n:
            kept[key] = rows(c[name + "_cache"], c[name + "_scale"], table[i], n, h)
        return kept[key][:n]

    def keys_of(h, t):
        b, seen = at[t]
        j = group[t]
        full = int(c["lens"][b])
        return tuple(np.concatenate((part(name, prefix_table, j, int(prefix_lens[j]), h),
                                     part(name, c["table"], b, full, h)[:seen])) for name in ("k", "v"))

    return _per_query(q, Hkv, keys_of, scale)


# ------------------------------------------------------------------ choice of pages
def page_bounds(codes, n):
    """codes [pages, H, P, d], n rows of each page in use -> smallest and largest value per column,
    [pages, H, 2, d]; NaN where a column holds one, +-inf for a page without rows."""
    x = e4m3_decode(codes)
    out = np.empty(codes.shape[:2] + (2, codes.shape[3]))
    for p in range(len(codes)):
        r = x[p, :, :int(n[p])]
        out[p, :, 0] = r.min(axis=1, initial=np.inf)
        out[p, :, 1] = r.max(axis=1, initial=-np.inf)
        bad = np.isnan(r).any(axis=1)
        out[p][np.broadcast_to(bad[:, None], out[p].shape)] = np.nan
    return out


def select_pages(q, bounds, scale, table, cu, lens, P, count, first, last, causal):
    """bounds [pages, Hkv, 2, d] values before their scale; -> int32 [Hkv, T, count].

    score(p) = scale_p max over the group's heads of sum_c max(q_c, 0) hi_c + min(q_c, 0) lo_c; NaN ranks
    above all, equal scores by number.
    """
    q = np.asarray(q, dtype=np.float64)
    Hkv = bounds.shape[1]
    g = q.shape[0] // Hkv
    at = queries(cu, lens, causal)
    out = np.full((Hkv, q.shape[1], count), -1, np.int32)
    for t, (b, seen) in enumerate(at):
        n = -(-max(seen, 0) // P)
        for h in range(Hkv):
            if n <= count:
                out[h, t, :n] = np.arange(n)
                continue
            x = q[h * g:(h + 1) * g, t]
            pool = range(first, n - last)
            ranked = []
            for j in pool:
                lo, hi = bounds[int(table[b][j]), h]
                with np.errstate(invalid="ignore"):
                    s = [math.fsum(v) if np.isfinite(v).all() else float(np.sum(v)) for v in np.concatenate((np.maximum(x, 0) * hi, np.minimum(x, 0) * lo), 1)]
                    s = float(np.max(s)) * float(scale[int(table[b][j]), h])
                ranked.append((0 if math.isnan(s) else 1, -s if not math.isnan(s) else 0.0, j))
            best = [j for _, _, j in sorted(ranked)[:count - first - last]]
            out[h, t] = sorted([*range(first), *best, *range(n - last, n)])
    return out
