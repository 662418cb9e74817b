"""The oracle of the cache and the host side of its calls where they are easily wrong."""
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
