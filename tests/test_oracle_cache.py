"""Pins of the cache and rotary oracles: against other ways of writing the same definitions."""
import numpy as np
import pytest
import torch

import oracle.cache as oc
import oracle.rope as orope
from cache_cases import bf16, empty_cache, filled, offsets, page_tables
from oracle.fp8 import attn_fwd_values, e4m3_decode


@pytest.mark.parametrize("amax,want", [(448.0, 1.0), (449.0, 2.0), (224.0, 0.5), (1.75, 2.0 ** -8), (1.7500001, 2.0 ** -7),
                                       (0.0, 0.0), (1e-44, 2.0 ** -126), (3.3e38, 2.0 ** 120)])
def test_pow2_scale(amax, want):
    assert oc.pow2_scale(amax) == want
    if want > 2.0 ** -126:
        assert amax / want <= 448.0 < 2 * amax / want


def test_append_matches_torch_conversion():
    """All at once into fresh pages: torch's float8 conversion of x / s."""
    lens, P, H, d = [37, 16, 1], 16, 2, 64
    table, pages = page_tables(lens, P, 3)
    codes, scale = empty_cache(pages, H, P, d)
    x = bf16(np.random.RandomState(0).randn(H, sum(lens), d) * 3)
    oc.append(x.float().numpy(), codes, scale, table, offsets(lens), lens)
    cu = offsets(lens)
    for b, n in enumerate(lens):
        for blk in range(-(-n // P)):
            rows = x[:, cu[b] + blk * P:min(cu[b] + (blk + 1) * P, cu[b + 1])].float()
            for h in range(H):
                s = scale[table[b, blk], h]
                want = (rows[h] / float(s)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
                assert (codes[table[b, blk], h, :rows.shape[1]] == want).all()


def test_append_one_by_one_ends_as_all_at_once():
    """The scale of a page is a power of two: the order of arrival leaves no trace in values
    that stay above the subnormals."""
    P, H, d, n = 32, 1, 64, 29
    table, pages = page_tables([n], P)
    x = bf16(np.exp2(np.arange(n) / 4.0)[None, :, None] * np.sign(np.random.RandomState(1).randn(H, n, d)))
    at_once, s1 = empty_cache(pages, H, P, d)
    oc.append(x.float().numpy(), at_once, s1, table, [0, n], [n])
    one, s2 = empty_cache(pages, H, P, d)
    for i in range(n):
        oc.append(x[:, i:i + 1].float().numpy(), one, s2, table, [0, 1], [i + 1])
    page = table[0, 0]
    assert s1[page, 0] == s2[page, 0]
    a, b = e4m3_decode(at_once[page, 0, :n]), e4m3_decode(one[page, 0, :n])
    big = np.abs(a) >= 2.0 ** -5
    assert big.sum() > n * d // 2 and (a[big] == b[big]).all()
    assert np.abs(a - b).max() <= 2.0 ** -9


def test_append_nonfinite_and_zero():
    P, H, d = 16, 1, 64
    table, pages = page_tables([3], P)
    codes, scale = empty_cache(pages, H, P, d)
    x = np.zeros((1, 3, d))
    oc.append(x[:, :1], codes, scale, table, [0, 1], [1])
    assert scale[table[0, 0], 0] == 0 and (codes[table[0, 0], 0, 0] == 0).all()
    x[0, 1, :4] = [np.inf, -np.inf, np.nan, 7.0]
    oc.append(x[:, 1:2], codes, scale, table, [0, 1], [2])
    assert scale[table[0, 0], 0] == 2.0 ** -6
    assert e4m3_decode(codes[table[0, 0], 0, 1, :2]).tolist() == [448.0, -448.0]
    assert np.isnan(e4m3_decode(codes[table[0, 0], 0, 1, 2])) and e4m3_decode(codes[table[0, 0], 0, 1, 3]) == 448.0


def test_attend_matches_dense_attention():
    lens, ns, Hq, H, P, d = [50, 33], [50, 33], 4, 2, 16, 64
    c = filled(lens, ns, Hq, H, P, d, seed=4)
    O, L, W, Z = oc.attend(c["q"].float().numpy(), c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], c["table"],
                           c["cu"], c["lens"], True, 0.125)
    for b, n in enumerate(lens):
        sl = slice(c["cu"][b], c["cu"][b + 1])
        k = np.stack([oc.rows(c["k_cache"], c["k_scale"], c["table"][b], n, h) for h in range(H)])[None]
        v = np.stack([oc.rows(c["v_cache"], c["v_scale"], c["table"][b], n, h) for h in range(H)])[None]
        o, l = attn_fwd_values(c["q"][:, sl].float().numpy()[None], k, v, True, 0.125)
        np.testing.assert_allclose(O[:, sl], o[0], atol=1e-12)
        np.testing.assert_allclose(L[:, sl], l[0], atol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_matrix(interleaved):
    """The rotation as an explicit matrix per position; its transpose is the gradient's."""
    d, rot, m = 16, 12, 1.25
    f = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    for p in (0, 1, 777):
        R = np.eye(d)
        for j in range(rot // 2):
            a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
            c, s = m * np.cos(p * f[j]), m * np.sin(p * f[j])
            R[a, a], R[a, b], R[b, b], R[b, a] = c, -s, c, s
        x = np.random.RandomState(p).randn(1, 1, 1, d)
        np.testing.assert_allclose(orope.rotate(x, f, [[p]], interleaved, m)[0, 0, 0], R @ x[0, 0, 0], atol=1e-12)
        np.testing.assert_allclose(orope.rotate(x, f, [[p]], interleaved, m, True)[0, 0, 0], R.T @ x[0, 0, 0], atol=1e-12)
