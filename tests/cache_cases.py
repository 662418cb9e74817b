"""Inputs and error bounds shared by the tests of the paged e4m3 cache."""
import numpy as np
import torch

import oracle.cache as oc


def bf16(x) -> torch.Tensor:
    return torch.as_tensor(np.asarray(x, dtype=np.float32)).to(torch.bfloat16)


def empty_cache(pages, H, P, d, seed=0):
    """Codes as earlier sequences left them: every code occurs, the NaN codes among them."""
    rng = np.random.RandomState(seed)
    codes = rng.randint(0, 256, (pages, H, P, d)).astype(np.uint8)
    scale = np.full((pages, H), np.float32(2.0) ** 40, dtype=np.float32)
    return codes, scale


def page_tables(lens, P, seed=0, spare=2, slack=1):
    """Page table [B, width] (shuffled pages, -1 past a sequence's end) and the page count."""
    rng = np.random.RandomState(seed + 1)
    need = [-(-int(n) // P) for n in lens]
    pages = sum(need) + spare
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((len(lens), max(need + [0]) + slack), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pages


def offsets(ns):
    return np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)


def filled(lens, ns, Hq, H, P, d, seed=0, gain=1.0):
    """A cache holding random rows (a gain for each page and head; stale codes elsewhere) and
    random queries: a dict of numpy arrays, q a bf16 tensor."""
    rng = np.random.RandomState(seed)
    table, pages = page_tables(lens, P, seed)
    out = {"table": table, "lens": np.asarray(lens, np.int32), "cu": offsets(ns)}
    for name in ("k", "v"):
        codes, scale = empty_cache(pages, H, P, d, seed + 7)
        for b, n in enumerate(lens):
            for blk in range(-(-int(n) // P)):
                m = min(P, int(n) - blk * P)
                for h in range(H):
                    x = rng.randn(m, d) * gain * np.exp2(rng.randn() * 0.7)
                    s = oc.pow2_scale(float(np.abs(x).max()))
                    codes[table[b, blk], h, :m] = oc.encode(x.astype(np.float32), s)
                    scale[table[b, blk], h] = s
        out[name + "_cache"], out[name + "_scale"] = codes, scale
    out["q"] = bf16(rng.randn(Hq, int(sum(ns)), d))
    return out


def bounds(O, L, W, Z, d):
    """Elementwise bounds on |O error| and |LSE error|.

    A score is a product sum of d terms in fp32 whose operands are exact (e4m3 in f16; q scaled
    by a power of two, components below 2^-14 of the row's largest rounded by at most 2^-25 of
    it, which the d 2^-24 covers), scaled and shifted by the maximum: its error is at most
    e_s = (d + 8) 2^-24 Z + 2^-22 Z.  The exponential adds 2^-21 relative, the weight's rounding
    to f16 2^-11 (and 2^-25 of the row's largest weight, as many as there are keys: 2^-38 after
    its shift by 2^14), fp32 sums over keys less than 2^-16.  So a weight is off by
    e_p = e_s + 2^-21 + 2^-11 + 2^-16, relatively, and O, with the error of the row sum, by
    2 e_p W; bf16 rounds it by 2^-8 |O| at most.  LSE = (max + log2 l) ln 2 is off by the score's
    error, the sum's and 2^-22 of itself."""
    e_s = (d + 8) * 2.0 ** -24 * Z + 2.0 ** -22 * Z
    e_p = e_s + 2.0 ** -21 + 2.0 ** -11 + 2.0 ** -16
    o = 2.0 ** -8 * np.abs(O) + 2 * e_p[..., None] * W * 1.01 + 1e-30
    l = e_s + 2.0 ** -16 + 2.0 ** -22 * np.abs(np.where(np.isfinite(L), L, 0.0))
    return o, l


def check(o, lse, ref, d):
    O, L, W, Z = ref
    bo, bl = bounds(O, L, W, Z, d)
    o = o.float().cpu().numpy().astype(np.float64)
    lse = lse.cpu().numpy().astype(np.float64)
    assert np.isfinite(o).all()
    worst = float(np.max(np.abs(o - O) / bo)) if O.size else 0.0
    assert worst <= 1.0, f"O off by {worst:.3g} of its bound at {np.unravel_index(np.argmax(np.abs(o - O) / bo), O.shape)}"
    none = np.isneginf(L)
    assert (np.isneginf(lse) == none).all()
    e = np.abs(np.where(none, 0.0, lse) - np.where(none, 0.0, L)) / bl
    assert e.size == 0 or e.max() <= 1.0, f"LSE off by {e.max():.3g} of its bound"
