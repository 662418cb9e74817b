"""Sizes at the ends of their ranges for the calls over parts of the 8-bit cache: counts near 2^31, tables without
entries.  Each call ends in a refusal before anything is launched."""
import pytest

from test_cache_abi import attend
from test_cache_parts_abi import A, ODD, listed, prefix, select  # noqa: F401  (A: the fixture)

TOP = 0x7fffffff


def test_counts_near_the_int_range_are_refused(A):  # noqa: F811
    """The kernels step past the end of a list by up to 1024 entries: that has to stay below 2^31."""
    for count in (TOP, TOP - 127, 0x7fff0001):
        assert select(A, count=count, ws=None) == -1 and listed(A, count=count, ws=None) == -1
        assert select(A, count=count, first=count, last=0, ws=None) == -1
    assert select(A, count=0x7fff0000, ws=None) == -4 and listed(A, count=0x7fff0000, ws=None) == -4


def test_a_table_without_columns_may_be_null(A):  # noqa: F811
    """An empty tensor has no address.  (The refusals that follow show that the pointer was let through.)"""
    assert attend(A, t=None, width=0, ws=None) == -4 and attend(A, t=None, width=1, ws=None) == -1
    assert listed(A, t=None, width=0, ws=None) == -4 and listed(A, t=None, width=1, ws=None) == -1
    assert prefix(A, pt=None, pwidth=0, ws=None) == -4 and prefix(A, pt=None, pwidth=1, ws=None) == -1
    assert prefix(A, t=None, width=0, ws=None) == -4 and prefix(A, t=None, width=1, ws=None) == -1
    assert select(A, t=None, width=0, out=ODD) == -3 and select(A, t=None, width=1, out=ODD) == -1


def test_more_lists_than_a_launch_has_blocks(A):  # noqa: F811
    """Refused with the other sizes, and no workspace size, which would pass 64 bits and wrap."""
    assert select(A, Hq=40000, H=40000, T=60000, mq=1, pages=1, ws=None) == -2
    assert select(A, Hq=40000, H=40000, T=50000, mq=1, pages=1, ws=None) == -4
    for sizes in ((40000, 60000, 5), (65535, 0x7fff0000, 1 << 27), (1, 1, 1 << 27), (65535, 32768, 1 << 30)):
        with pytest.raises(A.AttnError):
            A.attn_select_pages_fp8_workspace_size(*sizes)
    assert A.attn_select_pages_fp8_workspace_size(8, 4096, 8192) < 16.3 * 8 * 4096 * 8192
