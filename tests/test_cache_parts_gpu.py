"""attn_fwd_kv_fp8_pages and attn_fwd_kv_fp8_prefix against the fp64 oracle, within bounds that are
derived from the number formats (cache_cases.bounds, and below for the joint of two parts)."""
import numpy as np
import pytest
import torch

import oracle.cache as oc
import oracle.sparse as osp
from cache_cases import bf16, bounds, check, filled, offsets, page_tables

pytestmark = pytest.mark.gpu
DEV = "cuda"
INVALID, TIMEOUT = -1, -6


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


def dev(x):
    return torch.as_tensor(x).to(DEV)


def cache_args(c):
    return [dev(c[n]) for n in ("k_cache", "v_cache", "k_scale", "v_scale")]


# ------------------------------------------------------------------ listed pages
def lists(c, P, Hkv, count, causal, seed=0, holes=True):
    """Distinct pages that each query sees, shuffled, with negative entries between; a query sees its
    last page often enough."""
    rng = np.random.RandomState(seed)
    at = osp.queries(c["cu"], c["lens"], causal)
    out = np.full((Hkv, len(at), count), -1, np.int32)
    for h in range(Hkv):
        for t, (b, seen) in enumerate(at):
            n = -(-seen // P)
            pick = rng.permutation(n)[:rng.randint(0, min(n, count) + 1) if holes else count]
            if n and count and len(pick) and rng.rand() < 0.7:
                pick[0] = n - 1 if n - 1 not in pick else pick[0]
            room = min(n, count)
            where = rng.permutation(room)[:len(pick)]
            out[h, t, np.sort(where) if holes else np.arange(len(pick))] = pick
    return out


def run_pages(A, c, pages, causal=True, scale=None, **kw):
    return A.attn_fwd_kv_fp8_pages(dev(c["q"]), *cache_args(c), dev(c["table"]), dev(c["cu"]), dev(c["lens"]), dev(pages),
                                   causal=causal, scale=scale, **kw)


def check_pages(A, c, pages, causal=True, scale=None):
    d = c["q"].shape[2]
    o, lse = run_pages(A, c, pages, causal, scale)
    check(o, lse, osp.attend_pages(c["q"].float().numpy(), c, pages, causal, d ** -0.5 if scale is None else scale), d)


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,H", [(8, 2), (7, 1), (3, 3)])
def test_pages_lengths_and_holes(A, P, d, Hq, H):
    """One token and drafts, lengths from 1 to several pages, lists with holes, empty ones too."""
    c = filled([1, P, P + 1, 5 * P + 3, 9 * P - 1], [1, 2, 1, 4, 3], Hq, H, P, d, seed=P + d + Hq)
    check_pages(A, c, lists(c, P, H, 7, True, seed=P))
    check_pages(A, c, lists(c, P, H, 3, False, seed=P + 1), causal=False, scale=0.3)


@pytest.mark.parametrize("Hq,H", [(16, 1), (20, 1), (32, 1), (17, 1), (48, 2)])
def test_pages_wide_groups(A, Hq, H):
    c = filled([200, 77], [2, 1], Hq, H, 32, 128, seed=Hq)
    check_pages(A, c, lists(c, 32, H, 5, True, seed=1))


@pytest.mark.parametrize("P,d", [(16, 64), (32, 128), (128, 128)])
def test_all_pages_listed_is_the_whole_attention(A, P, d):
    c = filled([700, 1, 333], [1, 1, 2], 8, 2, P, d, seed=3)
    n = -(-700 // P)
    pages = np.tile(np.arange(n, dtype=np.int32), (2, 4, 1))
    for t, (b, seen) in enumerate(osp.queries(c["cu"], c["lens"], True)):
        pages[:, t, -(-seen // P):] = -1
    o, lse = run_pages(A, c, pages)
    check(o, lse, oc.attend(c["q"].float().numpy(), c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], c["table"],
                            c["cu"], c["lens"], True, d ** -0.5), d)


def test_pages_long_lists_cut_between_blocks(A):
    """Few units of many pieces (partial results are joined), then many units."""
    c = filled([9000], [1], 4, 1, 64, 128, seed=5)
    check_pages(A, c, lists(c, 64, 1, 130, True, holes=False))
    c = filled([900] * 40, [1] * 40, 16, 4, 16, 64, seed=6)
    check_pages(A, c, lists(c, 16, 4, 20, True, holes=False))


def test_pages_more_queries_than_threads(A):
    ns = [0, 150, 1, 0, 33, 2]
    c = filled([40, 160, 1, 0, 90, 17], ns, 2, 1, 16, 64, seed=8)
    check_pages(A, c, lists(c, 16, 1, 4, True))


def test_pages_no_keys_no_lists(A):
    c = filled([0, 5, 0], [2, 1, 1], 4, 2, 16, 64, seed=9)
    check_pages(A, c, np.full((2, 4, 3), -1, np.int32), causal=False)
    o, lse = run_pages(A, c, np.zeros((2, 4, 0), np.int32), causal=False)
    assert (o == 0).all() and torch.isneginf(lse).all()
    o, lse = A.attn_fwd_kv_fp8_pages(torch.empty(4, 0, 64, dtype=torch.bfloat16, device=DEV), *cache_args(c), dev(c["table"]),
                                     dev(np.zeros(4, np.int32)), dev(c["lens"]), dev(np.zeros((2, 0, 3), np.int32)))
    assert o.shape == (4, 0, 64) and lse.shape == (4, 0)


@pytest.mark.parametrize("P", [16, 64])
def test_pages_nan_behind_what_a_query_sees(A, P):
    """NaN rows inside a listed page but behind the query's own position reach later queries only."""
    d, H, n = 64, 1, 3
    c = filled([2 * P + 5], [n], 4, H, P, d, seed=2)
    page, slot = c["table"][0][2], 4                                       # the last key: only the last query sees it
    c["v_cache"][page, 0, slot, :3] = 0x7F
    c["k_cache"][page, 0, slot] = 0x7F
    pages = np.tile(np.array([0, 2, -1], np.int32), (H, n, 1))
    o, lse = run_pages(A, c, pages)
    O, L, W, Z = osp.attend_pages(c["q"].float().numpy(), {**c, "lens": c["lens"]}, pages, True, d ** -0.5)
    assert torch.isnan(o[:, 2]).all()
    check(o[:, :2], lse[:, :2], tuple(x[:, :2] for x in (O, L, W, Z)), d)


def test_pages_device_checks(A):
    P, H = 32, 2
    c = filled([100, 40], [1, 2], 4, H, P, 64, seed=4)
    good = lists(c, P, H, 4, True, holes=False)
    for where, entry in (((1, 0, 1), 4), ((0, 2, 0), 2), ((0, 1, 3), 0), ((0, 1, 2), 1), ((0, 0, 0), 2 ** 31 - 1)):
        pages = good.copy()
        pages[where] = entry                                               # behind the last page, or one too many
        run_pages(A, c, pages)
        assert A.attn_device_status(True) == INVALID, (where, entry)
    for entry in (-1, c["k_cache"].shape[0], 2 ** 31 - 1):                 # a bad page of the table, listed
        table = c["table"].copy()
        table[0, 0] = entry
        pages = np.full((H, 3, 4), -1, np.int32)
        pages[:, 0, 0] = 0
        run_pages(A, {**c, "table": table}, pages)
        assert A.attn_device_status(True) == INVALID
        pages[:, 0, 0] = 1                                                 # not listed: not read
        check_pages(A, {**c, "table": np.where(table == entry, c["table"], table)}, pages)
        run_pages(A, {**c, "table": table}, pages)
        assert A.attn_device_status(True) == 0
    o = torch.full((4, 3, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    for cu, lens in (([0, 1, 2], c["lens"]), ([0, 4, 3], c["lens"]), ([1, 1, 3], c["lens"]), (c["cu"], [100, 1]),
                     (c["cu"], [-1, 40]), (c["cu"], [1 << 20, 40])):
        run_pages(A, {**c, "cu": np.asarray(cu, np.int32), "lens": np.asarray(lens, np.int32)}, good, o=o)
        assert A.attn_device_status(True) == INVALID and (o == 7).all()


# ------------------------------------------------------------------ shared prefixes
def prefixed(prefix, lens, ns, members, Hq, H, P, d, seed=0):
    """One cache for prefixes and sequences: filled() with the prefixes as further sequences."""
    c = filled(list(prefix) + list(lens), [0] * len(prefix) + list(ns), Hq, H, P, d, seed=seed)
    G = len(prefix)
    pre = dict(table=np.ascontiguousarray(c["table"][:G]), cu=offsets(members), lens=c["lens"][:G].copy())
    c.update(table=np.ascontiguousarray(c["table"][G:]), cu=offsets(ns), lens=c["lens"][G:].copy())
    return c, pre


def run_prefix(A, c, pre, causal=True, max_prefix_q=None, max_q=None, **kw):
    return A.attn_fwd_kv_fp8_prefix(dev(c["q"]), *cache_args(c), dev(pre["table"]), dev(pre["cu"]), dev(pre["lens"]),
                                    int(np.diff(pre["cu"]).max()) if max_prefix_q is None else max_prefix_q, dev(c["table"]),
                                    dev(c["cu"]), dev(c["lens"]), int(np.diff(c["cu"]).max()) if max_q is None else max_q,
                                    causal=causal, **kw)


def check_prefix(A, c, pre, causal=True, **kw):
    """A part's own bound (cache_cases.bounds), and the joint's: a part's weight 2^(lse_a - lse) is off by
    what its log2 sum is, the score's error e_s, 2^-16 of the sum, 2^-21 of the logarithm and two roundings of
    up to 2^-24 of its size each, and by 2^-22 of the exponential; relatively, on every element of W."""
    d = c["q"].shape[2]
    o, lse = run_prefix(A, c, pre, causal, **kw)
    O, L, W, Z = osp.attend_prefix(c["q"].float().numpy(), c, pre["table"], pre["cu"], pre["lens"], causal, d ** -0.5)
    bo, bl = bounds(O, L, W, Z, d)
    e_s = (d + 8) * 2.0 ** -24 * Z + 2.0 ** -22 * Z
    size = np.abs(np.where(np.isfinite(L), L, 0.0)) / np.log(2.0) + 32    # a part's log2 sum, where it weighs
    e_j = 2 * (e_s + 2.0 ** -16 + 2.0 ** -21 + 2.0 ** -22 + 2.0 ** -23 * size)
    bo, bl = bo + e_j[..., None] * W, bl + e_j
    o, lse = o.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    none = np.isneginf(L)
    assert np.isfinite(o).all() and (np.isneginf(lse) == none).all()
    worst = np.max(np.abs(o - O) / bo)
    assert worst <= 1, f"O off by {worst:.3g} of its bound"
    worst = np.max(np.abs(np.where(none, 0.0, lse) - np.where(none, 0.0, L)) / bl)
    assert worst <= 1, f"LSE off by {worst:.3g} of its bound"


SHAPES = [  # prefix lengths, own lengths, queries, queries per prefix
    ([300], [5, 70, 1], [1, 1, 1], [3]),                                   # few rows everywhere
    ([1000, 0, 77], [9, 40, 200, 3, 64], [1, 1, 1, 1, 1], [2, 1, 2]),      # one prefix is empty
    ([2111], list(range(1, 41)), [1] * 40, [40]),                          # tiles, then few rows
    ([513, 129], [60, 250, 131], [31, 40, 1], [50, 22]),                   # tiles everywhere; borders inside a sequence
    ([64], [300], [100], [100]),
    ([1], [1], [1], [1]),
    ([30, 0, 77, 400, 5], [64], [20], [4] * 5),                            # few rows behind each prefix, tiles of one sequence
    ([700], [1 + 7 * (i % 9) for i in range(160)], [1] * 160, [160]),      # tiles, then more units of few rows than SMs
]


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("Hq,H,P,d", [(8, 2, 16, 64), (4, 4, 128, 128), (7, 1, 64, 128), (16, 2, 32, 64)])
def test_prefix(A, shape, Hq, H, P, d):
    prefix, lens, ns, members = SHAPES[shape]
    c, pre = prefixed(prefix, lens, ns, members, Hq, H, P, d, seed=shape)
    check_prefix(A, c, pre)


@pytest.mark.parametrize("ns,members,Hq,lens", [([2, 1], [3], 4, [70, 5]), ([20, 9], [29], 4, [70, 40]), ([1] * 100, [100], 4, [70] + [5] * 99),
                                                ([20], [4] * 5, 2, [70])])
def test_prefix_nan_values_reach_the_queries_that_see_them(A, ns, members, Hq, lens):
    """A NaN among a sequence's own values reaches its queries from there on; one in a prefix all behind it."""
    H, P, d = 2, 32, 64
    G = len(members)
    c, pre = prefixed([90] * G, lens, ns, members, Hq, H, P, d, seed=17)
    ref = lambda cc: osp.attend_prefix(cc["q"].float().numpy(), cc, pre["table"], pre["cu"], pre["lens"], True, d ** -0.5)[0]
    clean = ref(c)
    at = lens[0] - 1                                       # the first sequence's last key: its last query's alone
    own = {**c, "v_cache": c["v_cache"].copy()}
    own["v_cache"][c["table"][0, at // P], 1, at % P, 7:9] = 0x7F
    o = run_prefix(A, own, pre)[0].float().cpu().numpy()
    want = np.zeros(o.shape, bool)
    want[Hq // 2:, ns[0] - 1, 7:9] = True
    assert (np.isnan(o) == want).all()
    front = {**c, "v_cache": c["v_cache"].copy()}
    front["v_cache"][pre["table"][G - 1, 1], 0, 3, 60] = 0xFF
    o = run_prefix(A, front, pre)[0].float().cpu().numpy()
    want = np.zeros(o.shape, bool)
    want[:Hq // 2, pre["cu"][G - 1]:, 60] = True
    assert (np.isnan(o) == want).all()
    assert np.abs(o - clean)[~want].max() < 0.1


def test_prefix_bounds_larger_than_needed_and_not_causal(A):
    c, pre = prefixed([700, 130], [40, 0, 9], [2, 1, 3], [3, 3], 8, 2, 32, 128, seed=11)
    check_prefix(A, c, pre, causal=False)
    check_prefix(A, c, pre, causal=False, max_prefix_q=6, max_q=6)


@pytest.mark.parametrize("members", [[1], [40]])
def test_prefix_and_own_keys_both_empty(A, members):
    """O = 0 and LSE = -inf where no part has a key; elsewhere one part alone counts."""
    n = members[0]
    c, pre = prefixed([0], [0, 30] if n > 1 else [0], [n - 1, 1] if n > 1 else [1], members, 4, 1, 16, 64, seed=12)
    check_prefix(A, c, pre, causal=False)
    c, pre = prefixed([50], [0], [n], members, 4, 1, 16, 64, seed=13)
    check_prefix(A, c, pre, causal=False)


def test_prefix_equals_the_whole_attention(A):
    """A prefix of whole pages and the rest, against attn_fwd_kv_fp8 over all of it: the same keys, so
    both within their bounds of the same oracle; here of one another, which is twice a bound at most."""
    P, d, shared, own = 64, 128, 640, [70, 1, 200]
    c, pre = prefixed([shared], own, [1, 1, 1], [3], 8, 2, P, d, seed=21)
    width = shared // P + c["table"].shape[1]
    table = np.full((3, width), -1, np.int32)
    table[:, :shared // P] = pre["table"][0, :shared // P]
    table[:, shared // P:] = c["table"]
    whole = {**c, "table": table, "lens": c["lens"] + shared}
    o, lse = A.attn_fwd_kv_fp8(dev(c["q"]), *cache_args(c), dev(table), dev(c["cu"]), dev(whole["lens"]), 1)
    check_prefix(A, c, pre)
    O, L, W, Z = osp.attend_prefix(c["q"].float().numpy(), c, pre["table"], pre["cu"], pre["lens"], True, d ** -0.5)
    check(o, lse, (O, L, W, Z), d)


def test_prefix_device_checks_write_nothing(A):
    c, pre = prefixed([100], [20, 33], [1, 2], [3], 4, 2, 32, 64, seed=4)
    for members in (1, 30):                                                # the first part by few rows or tiles
        o = torch.full((4, 3, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((4, 3), 7.0, device=DEV)
        kw = dict(o=o, lse=lse, max_prefix_q=3, max_q=3 if members > 1 else 2)
        for bad in (dict(pre=dict(cu=[0, 2])), dict(pre=dict(cu=[1, 3])), dict(pre=dict(lens=[-1])), dict(pre=dict(lens=[1 << 20])),
                    dict(c=dict(cu=[0, 1, 2])), dict(c=dict(lens=[20, 1])), dict(c=dict(lens=[20, 1 << 20]))):
            cc = {**c, **{n: np.asarray(x, np.int32) for n, x in bad.get("c", {}).items()}}
            pp = {**pre, **{n: np.asarray(x, np.int32) for n, x in bad.get("pre", {}).items()}}
            run_prefix(A, cc, pp, **kw)
            assert A.attn_device_status(True) == INVALID and (o == 7).all() and (lse == 7).all(), bad
    run_prefix(A, c, pre, max_prefix_q=2)                                  # a bound that is too small
    assert A.attn_device_status(True) == INVALID
    table = pre["table"].copy()
    table[0, 1] = -5
    run_prefix(A, c, {**pre, "table": table})
    assert A.attn_device_status(True) == INVALID


@pytest.mark.parametrize("ns,members,lens", [([1] * 80, [80], [9] * 80), ([20], [4] * 5, [30])])
def test_prefix_by_two_kernels_device_checks_write_nothing(A, ns, members, lens):
    """Tiles then few rows (more units than SMs), and few rows then tiles: a launch for each part."""
    G, B, T = len(members), len(ns), sum(ns)
    c, pre = prefixed([50] * G, lens, ns, members, 8, 2, 32, 64, seed=6)
    check_prefix(A, c, pre)
    o = torch.full((8, T, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((8, T), 7.0, device=DEV)
    cu, mine = pre["cu"].copy(), c["cu"].copy()
    cu[-1] -= 1
    mine[-1] += 1
    for p, q in ((dict(cu=cu), {}), (dict(lens=np.full(G, -1)), {}), ({}, dict(cu=mine)), ({}, dict(lens=np.full(B, 1 << 20)))):
        as32 = lambda d: {n: np.asarray(x, np.int32) for n, x in d.items()}
        run_prefix(A, {**c, **as32(q)}, {**pre, **as32(p)}, o=o, lse=lse, max_prefix_q=max(members), max_q=max(ns))
        assert A.attn_device_status(True) == INVALID and (o == 7).all() and (lse == 7).all()


def test_prefix_tiles_device_checks_write_nothing(A):
    ns = [20, 30]
    c, pre = prefixed([100], [20, 33], ns, [50], 4, 2, 32, 64, seed=5)
    o = torch.full((4, 50, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((4, 50), 7.0, device=DEV)
    for cu, lens in (([0, 49], [100]), ([0, 50], [-3])):
        run_prefix(A, c, {**pre, "cu": np.asarray(cu, np.int32), "lens": np.asarray(lens, np.int32)}, o=o, lse=lse,
                   max_prefix_q=50)
        assert A.attn_device_status(True) == INVALID and (o == 7).all() and (lse == 7).all()


# ------------------------------------------------------------------ how they are called
@pytest.mark.parametrize("which", ["pages", "prefix", "prefix_tiles", "prefix_two"])
def test_captured_replayed_and_on_another_stream(A, which):
    if which == "pages":
        c = filled([500, 90], [1, 2], 8, 2, 32, 128, seed=31)
        pages = lists(c, 32, 2, 6, True, seed=1)
        args = [dev(c["q"]), *cache_args(c), dev(c["table"]), dev(c["cu"]), dev(c["lens"]), dev(pages)]
        call, size = A.attn_fwd_kv_fp8_pages, A.attn_fwd_kv_fp8_pages_workspace_size(8, 2, 3, 128)
    else:
        n, B = {"prefix": (1, 2), "prefix_tiles": (30, 2), "prefix_two": (1, 90)}[which]
        c, pre = prefixed([400], [30 + i % 2 * 20 for i in range(B)], [n] * B, [B * n], 8, 2, 32, 128, seed=32)
        args = [dev(c["q"]), *cache_args(c), dev(pre["table"]), dev(pre["cu"]), dev(pre["lens"]), B * n, dev(c["table"]),
                dev(c["cu"]), dev(c["lens"]), n]
        call, size = A.attn_fwd_kv_fp8_prefix, A.attn_fwd_kv_fp8_prefix_workspace_size(8, 2, B * n, B * n, n, 128)
    want = call(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(*args, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    outs, graphs = [], []
    for _ in range(2):                                                     # two graphs, a workspace each
        o, lse, ws = torch.empty_like(want[0]), torch.empty_like(want[1]), torch.empty(size, dtype=torch.uint8, device=DEV)
        call(*args, o=o, lse=lse, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(*args, o=o, lse=lse, workspace=ws)
        outs.append((o, lse, ws))
        graphs.append(g)
    for k in range(3):
        args[0].mul_(-1)                                                   # new queries, lengths as they were
        want = call(*args)
        torch.cuda.synchronize()
        for o, lse, ws in outs:
            o.fill_(3)
            ws.fill_(0xAB)
        streams = [torch.cuda.Stream() for _ in graphs]
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, lse, _ in outs:
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("which", ["pages", "prefix", "prefix_tiles", "prefix_two"])
def test_a_wait_that_runs_out(A, which):
    n, B = {"prefix_tiles": (20, 1), "prefix_two": (1, 90)}.get(which, (1, 1))
    c, pre = prefixed([400], [50] * B, [n] * B, [n * B], 8, 2, 32, 128, seed=33)
    A.attn_set_debug_knobs(wait_limit_ns=2_000_000)
    A.attn_set_test_hooks(skip_first_kv_load=True)
    try:
        if which == "pages":
            run_pages(A, c, np.zeros((2, n * B, 1), np.int32))
        else:
            run_prefix(A, c, pre)
        assert A.attn_device_status(True) == TIMEOUT
    finally:
        A.attn_set_test_hooks(False)
        A.attn_set_debug_knobs()
    check_prefix(A, c, pre)
