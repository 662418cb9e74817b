"""Listed pages and shared prefixes: pages that only later queries see, tables without entries, offsets of a
second part that are wrong."""
import numpy as np
import pytest
import torch

import oracle.sparse as osp
from cache_cases import bf16, check, filled
from test_cache_parts_gpu import DEV, INVALID, cache_args, check_prefix, dev, prefixed, run_pages, run_prefix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def A():
    import attention_attn_fwd_09_gb300 as A
    A.attn_set_debug_knobs()
    A.attn_device_status(True)
    yield A


@pytest.fixture(autouse=True)
def clean_status(A):
    yield
    assert A.attn_device_status(True) == 0


def same(A, c, pages, d):
    o, lse = run_pages(A, c, pages)
    check(o, lse, osp.attend_pages(c["q"].float().numpy(), c, pages, True, d ** -0.5), d)


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_drafts_that_share_a_list_across_a_page_border(A, P, d):
    """Drafts of which the first ones end a page: the next page is masked for them, wherever it is listed."""
    H, n = 2, 4
    c = filled([2 * P + 2, 5 * P + 1], [n, n], 8, H, P, d, seed=P + d)      # they see 2, 2, 3, 3 and 5, 5, 5, 6 pages
    for first, second in (([0, 1, 2, -1], [0, 2, 4, 5]), ([2, 0, -1, -1], [5, 1, 0, -1]), ([-1, 1, 2, -1], [5, -1, 4, -1]),
                          ([2, -1, -1, -1], [5, -1, -1, -1])):              # (the last: nothing that some queries see)
        pages = np.empty((H, 2 * n, 4), np.int32)
        pages[:, :n], pages[:, n:] = first, second
        same(A, c, pages, d)


def test_a_page_behind_the_sequence_and_one_too_far_back_in_the_list(A):
    P, H, d = 32, 2, 64
    c = filled([2 * P + 1, 40], [3, 1], 4, H, P, d, seed=5)                 # the first sequence's queries see 2, 2, 3 pages
    good = np.full((H, 4, 4), -1, np.int32)
    good[:, :3, :3], good[:, 3, :2] = [0, 1, 2], [0, 1]
    same(A, c, good, d)
    for where, entry in (((0, 0, 1), 3), ((0, 0, 2), 3), ((1, 1, 3), 0), ((0, 0, 2), 1), ((1, 3, 0), 2)):
        pages = good.copy()
        pages[where] = entry
        run_pages(A, c, pages)
        assert A.attn_device_status(True) == INVALID, (where, entry)
