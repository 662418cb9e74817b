"""The oracle of the cache and the host side of its calls where they are easily wrong."""
import ctypes

import numpy as np
import pytest

import oracle.cache as oc
from cache_cases import empty_cache, page_tables
from oracle.fp8 import e4m3_decode


@pytest.mark.parametrize("first", [[np.inf, -np.inf, np.nan, 0.0], [np.inf, 0.0, -0.0, 0.0]])
@pytest.mark.parametrize("second", [7.0, 1e-30, 3e38])
def test_a_kept_row_reads_the_same_when_its_page_gets_its_first_scale(first, second):
    """A row without a finite value other than 0 leaves scale 0 and codes that read 0 (or NaN).  What
    it reads is decode(code) * scale, before and after the page's scale grows."""
    P, H, d = 16, 1, 64
    table, pages = page_tables([2], P)
    codes, scale = empty_cache(pages, H, P, d)
    x = np.zeros((1, 2, d))
    x[0, 0, :4], x[0, 1] = first, np.float32(second)
    oc.append(x[:, :1], codes, scale, table, [0, 1], [1])
    page = table[0, 0]
    with np.errstate(invalid="ignore"):
        was = e4m3_decode(codes[page, 0, 0]) * float(scale[page, 0])
    assert scale[page, 0] == 0 and (was[~np.isnan(was)] == 0).all()
    oc.append(x[:, 1:], codes, scale, table, [0, 1], [2])
    now = e4m3_decode(codes[page, 0, 0]) * float(scale[page, 0])
    assert scale[page, 0] > 0
    np.testing.assert_array_equal(now, was)


@pytest.fixture(scope="module")
def A():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import attention_attn_fwd_09_gb300 as A
    return A


@pytest.mark.parametrize("fn", ["attn_rope", "attn_rope_bwd"])
@pytest.mark.parametrize("which", ["q", "k"])
@pytest.mark.parametrize("out", [
    (4096, 64, 64),         # heads and tokens coincide
    (4096, 64, 128),        # head 2 is token 1
    (64, 256, 64),          # a batch element is a token
    (4096, -64, 64), (4096, 0, 64), (4096, 100, 32), (1 << 62, 1 << 62, 64),
])
def test_rotary_outputs_whose_rows_overlap_are_refused(A, fn, which, out):
    """No stride is short, but two rows of the output share an element (3 heads, 4 tokens, 2 sequences)."""
    fine, d = (3 * 4 * 64, 4 * 64, 64), 64
    outs = out + fine if which == "q" else fine + out
    st = (ctypes.c_longlong * 12)(*(fine + fine + outs))
    p = [ctypes.c_void_p(0x10000 * i) for i in (1, 2, 3, 4, 5)]
    rc = getattr(A._lib, fn)(p[0], p[1], p[2], p[3], p[4], None, 2, 3, 3, 4, d, d, 0, 1.0, st, None)
    assert rc == -1 and "overlap" in A.attn_last_error()


@pytest.mark.parametrize("rot,base,trained,factor", [(128, 1e4, 8192, 4.0), (64, 1e6, 32768, 8.0), (128, 5e5, 4096, 2.0), (96, 1e4, 2048, 1.5)])
def test_yarn_frequencies_of_released_checkpoints(A, rot, base, trained, factor):
    """The blend runs linearly over the pairs, from the last one with 32 turns or more over the trained length
    to the first with one or fewer; here these pairs are found by counting turns.  ramp="turns" blends linearly
    in the turns instead."""
    f = base ** (-2.0 * np.arange(rot // 2) / rot)
    turns = trained * f / (2 * np.pi)
    first, last = int(np.flatnonzero(turns >= 32)[-1]), int(np.flatnonzero(turns <= 1)[0])
    assert 0 < first < last < rot // 2 - 1
    compressed = np.clip((np.arange(rot // 2) - first) / (last - first), 0, 1)
    got, m = A.attn_rope_freqs(rot, base, "yarn", factor, trained, device="cpu")
    np.testing.assert_allclose(got.numpy(), f * (1 - compressed) + f / factor * compressed, rtol=1e-13)
    assert abs(m - (0.1 * np.log(factor) + 1)) < 1e-15
    same = A.attn_rope_freqs(rot, base, "yarn", factor, trained, device="cpu", ramp="pairs")[0]
    assert (same == got).all()
    left = np.clip((turns - 1) / 31, 0, 1)
    got, _ = A.attn_rope_freqs(rot, base, "yarn", factor, trained, device="cpu", ramp="turns")
    np.testing.assert_allclose(got.numpy(), f * left + f / factor * (1 - left), rtol=1e-13)


def test_yarn_refusals_and_far_ends(A):
    for bad in (dict(ramp="other"), dict(beta_slow=0.0), dict(beta_slow=-1.0), dict(beta_fast=1.0)):
        with pytest.raises(ValueError):
            A.attn_rope_freqs(64, scaling="yarn", factor=2.0, trained_length=1024, device="cpu", **bad)
    f = 1e4 ** (-2.0 * np.arange(32) / 64)
    short = A.attn_rope_freqs(64, scaling="yarn", factor=2.0, trained_length=64, device="cpu")[0].numpy()   # no pair makes 32 turns
    assert short[0] == 1.0 and (np.diff(short / f) <= 1e-12).all() and abs(short[-1] / f[-1] - 0.5) < 1e-12
    long = A.attn_rope_freqs(64, scaling="yarn", factor=2.0, trained_length=1 << 40, device="cpu")[0].numpy()
    np.testing.assert_allclose(long, f, rtol=1e-13)                                                         # all make more


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", [(8, 2), (32, 1), (5, 5)])
def test_workspace_does_not_fall_as_the_bound_grows(A, heads, d):
    sizes = [A.attn_fwd_kv_fp8_workspace_size(3, *heads, total, mq, d) for total in (3, 70) for mq in range(1, 60)]
    assert sizes[:59] == sizes[59:] == sorted(sizes[:59]) and sizes[0] > 0
