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


def test_tables_without_entries(A):
    """Lengths of 0 need no pages: tables of no columns are as good as any."""
    c, pre = prefixed([0, 0], [40, 7, 90], [1, 1, 2], [1, 3], 8, 2, 32, 64, seed=1)
    none = np.zeros((2, 0), np.int32)
    want = run_prefix(A, c, pre)
    check_prefix(A, c, {**pre, "table": none})
    got = run_prefix(A, c, {**pre, "table": none})
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    c, pre = prefixed([300], [0] * 20, [2] * 20, [40], 8, 2, 32, 64, seed=2)            # by tiles
    check_prefix(A, {**c, "table": np.zeros((20, 0), np.int32)}, pre, causal=False)
    empty = filled([0, 0], [1, 2], 8, 2, 32, 64, seed=3)
    empty["table"] = none
    args = [dev(empty["q"]), *cache_args(empty), dev(none), dev(empty["cu"]), dev(empty["lens"])]
    for o, lse in (A.attn_fwd_kv_fp8(*args, 2, causal=False), A.attn_fwd_kv_fp8(*[bf16(np.ones((32, 3, 64))).to(DEV), *args[1:]], 2, causal=False),
                   A.attn_fwd_kv_fp8_pages(*args, dev(np.full((2, 3, 4), -1, np.int32)), causal=False)):
        assert (o == 0).all() and torch.isneginf(lse).all()
    bounds = torch.zeros(empty["k_cache"].shape[0], 2, 2, 64, dtype=torch.uint8, device=DEV)
    lists = A.attn_select_pages_fp8(args[0], bounds, args[3], dev(none), args[6], args[7], 32, 4, 2, causal=False)
    assert (lists == -1).all()


@pytest.mark.parametrize("Hq,H,P,d", [(4, 2, 32, 64), (16, 1, 128, 128)])
def test_tiles_of_both_parts_write_nothing_when_the_second_is_wrong(A, Hq, H, P, d):
    """One launch of tiles for both parts: offsets and lengths of either part that break a rule."""
    ns = [20, 30]
    c, pre = prefixed([100, 70], [20, 33], ns, [15, 35], Hq, H, P, d, seed=5)
    check_prefix(A, c, pre)
    o = torch.full((Hq, 50, d), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((Hq, 50), 7.0, device=DEV)
    big = 1 << 20
    for mine, front in ((dict(cu=[0, 20, 49]), {}), (dict(cu=[1, 20, 50]), {}), (dict(cu=[0, 51, 50]), {}), (dict(lens=[20, 29]), {}),
                        (dict(lens=[-1, 33]), {}), (dict(lens=[20, big]), {}), ({}, dict(cu=[0, 15, 51])), ({}, dict(lens=[100, -1])),
                        ({}, dict(lens=[big, 70]))):
        as32 = lambda x: {n: np.asarray(v, np.int32) for n, v in x.items()}
        run_prefix(A, {**c, **as32(mine)}, {**pre, **as32(front)}, o=o, lse=lse, max_prefix_q=35, max_q=30)
        assert A.attn_device_status(True) == INVALID and (o == 7).all() and (lse == 7).all(), (mine, front)
    run_prefix(A, c, pre, o=o, lse=lse, max_prefix_q=35, max_q=29)          # a bound that is too small
    assert A.attn_device_status(True) == INVALID and (o == 7).all()
