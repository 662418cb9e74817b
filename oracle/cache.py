"""CPU oracle for the paged e4m3 key/value cache and the attention over it.  TEST
INFRASTRUCTURE ONLY; imports nothing from the product path.

Cache: codes [pages, H, P, d] (uint8, e4m3 as oracle/fp8.py reads them) and scales [pages, H];
row t of sequence b is row t % P of page table[b][t // P].

append   the n new rows of sequence b become its rows lens[b] - n .. lens[b] - 1.  Per page and
         head touched: A = max |finite new value|, s = 2^ceil(log2(A / 448)) (0 for A = 0);
         with earlier rows in the page s = max(s, s_old), and if s > s_old their codes
         become e4m3(decode(code) * s_old / s).  New codes are e4m3(x / s); infinities become
         +-448, NaN the NaN code.
attend   softmax(scale q k~^T) v~ in fp64 over the visible keys: j < lens[b], with causal
         j <= i + lens[b] - n.  No visible key: O = 0, LSE = -inf.
"""
from __future__ import annotations

import math

import numpy as np

from .fp8 import E4M3_MAX, e4m3_decode, e4m3_encode


def pow2_scale(amax: float) -> float:
    if amax <= 0:
        return 0.0
    m, e = math.frexp(amax)                 # amax = m 2^e, 1/2 <= m < 1; 448 = 0.875 * 2^9
    return max(math.ldexp(1.0, e - 9 if m <= 0.875 else e - 8), 2.0 ** -126)


def encode(x, s) -> np.ndarray:
    """e4m3 codes of x / s (x, s fp64 holding fp32 values), by the rules above."""
    x = np.asarray(x, dtype=np.float64)
    y = (x / s if s > 0 else x).astype(np.float32)
    nan = np.isnan(y)
    y = np.where(nan, np.float32(0), np.clip(y, -E4M3_MAX, E4M3_MAX))
    sign = np.where(np.signbit(x), 0x80, 0).astype(np.uint8)
    return np.where(nan, sign | 0x7F, e4m3_encode(y)).astype(np.uint8)


def append(x, codes, scale, table, cu, lens) -> None:
    """x [H, total, d] values into codes, scale (numpy arrays, changed in place)."""
    x = np.asarray(x, dtype=np.float64)
    H, P = codes.shape[1], codes.shape[2]
    for b in range(len(lens)):
        n = int(cu[b + 1] - cu[b])
        start = int(lens[b]) - n
        pos = start
        while pos < lens[b]:
            blk, slot = divmod(pos, P)
            end = min(int(lens[b]), (blk + 1) * P)
            page = int(table[b][blk])
            rows = x[:, cu[b] + pos - start:cu[b] + end - start]
            for h in range(H):
                mag = np.abs(rows[h])
                s = pow2_scale(float(np.max(np.where(np.isfinite(mag), mag, 0.0), initial=0.0)))
                if slot > 0:
                    s_old = float(scale[page, h])
                    s = max(s, s_old)
                    if s > s_old:
                        old = (e4m3_decode(codes[page, h, :slot]).astype(np.float32) * np.float32(s_old)).astype(np.float64)
                        codes[page, h, :slot] = encode(old, s)
                scale[page, h] = s
                codes[page, h, slot:slot + end - pos] = encode(rows[h], s)
            pos = end


def rows(codes, scale, table_row, n: int, h: int) -> np.ndarray:
    """The first n dequantised rows of one sequence and head, fp64 [n, d]."""
    P = codes.shape[2]
    out = np.empty((n, codes.shape[3]))
    for blk in range((n + P - 1) // P):
        page, m = int(table_row[blk]), min(P, n - blk * P)
        out[blk * P:blk * P + m] = e4m3_decode(codes[page, h, :m]) * float(scale[page, h])
    return out


def attend(q, k_codes, v_codes, k_scale, v_scale, table, cu, lens, causal: bool, scale: float):
    """q [Hq, total, d] values -> (O, LSE, W, Z) in fp64: the result, sum_j p_j |v_j| per element
    of O, and the largest scale * sum_c |q_c k_jc| of each row's visible keys (what an error bound
    needs)."""
    q = np.asarray(q, dtype=np.float64)
    Hq, T, d = q.shape
    g = Hq // k_codes.shape[1]
    O, W = np.zeros((Hq, T, d)), np.zeros((Hq, T, d))
    L, Z = np.full((Hq, T), -np.inf), np.zeros((Hq, T))
    for b in range(len(lens)):
        n, nk = int(cu[b + 1] - cu[b]), int(lens[b])
        if n == 0 or nk == 0:
            continue
        sl = np.s_[int(cu[b]):int(cu[b + 1])]
        for h in range(Hq // g):
            kk = rows(k_codes, k_scale, table[b], nk, h)
            vv = rows(v_codes, v_scale, table[b], nk, h)
            for hq in range(h * g, (h + 1) * g):
                s = scale * (q[hq, sl] @ kk.T)
                z = scale * (np.abs(q[hq, sl]) @ np.abs(kk).T)
                if causal:
                    hidden = np.arange(nk)[None, :] > np.arange(n)[:, None] + nk - n
                    s, z = np.where(hidden, -np.inf, s), np.where(hidden, 0.0, z)
                m = s.max(axis=1, keepdims=True)
                p = np.exp(s - m)
                l = p.sum(axis=1, keepdims=True)
                O[hq, sl] = (p / l) @ vv
                W[hq, sl] = (p / l) @ np.abs(vv)
                L[hq, sl] = (m + np.log(l))[:, 0]
                Z[hq, sl] = z.max(axis=1)
    return O, L, W, Z
