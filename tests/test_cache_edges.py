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
