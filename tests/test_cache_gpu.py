"""attn_kv_append_fp8 and attn_fwd_kv_fp8 against the fp64 oracle: codes and scales exactly,
attention within the bounds derived in cache_cases.bounds."""
import numpy as np
import pytest
import torch

import oracle.cache as oc
import oracle.rope as orope
from cache_cases import bf16, check, empty_cache, filled, offsets, page_tables

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


# ------------------------------------------------------------------ append
class Cache:
    """The same cache on the GPU and in the oracle."""

    def __init__(self, A, table, pages, H, P, d, seed=0):
        self.A, self.table = A, table
        self.host = {n: empty_cache(pages, H, P, d, seed + i) for i, n in enumerate("kv")}
        self.gpu = {n: (dev(c.copy()), dev(s.copy())) for n, (c, s) in self.host.items()}
        self.dtable = dev(table)

    def append(self, k, v, ns, lens, views=None):
        cu = offsets(ns)
        for n, x in (("k", k), ("v", v)):
            oc.append(x.float().numpy(), *self.host[n], self.table, cu, lens)
        gk, gv = views if views else (k.to(DEV), v.to(DEV))
        self.A.attn_kv_append_fp8(gk, gv, self.gpu["k"][0], self.gpu["v"][0], self.gpu["k"][1], self.gpu["v"][1],
                                  self.dtable, dev(cu), dev(np.asarray(lens, np.int32)))

    def same(self):
        for n in "kv":
            for got, want in zip(self.gpu[n], self.host[n]):
                got = got.cpu().numpy()
                assert (got == want).all(), (n, np.argwhere(got != want)[:5])


def kv(rng, H, T, d, gain=1.0):
    return bf16(rng.randn(H, T, d) * gain), bf16(rng.randn(H, T, d) * gain * 3)


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_append_prompts_then_tokens(A, P, d):
    """Prompts of odd lengths, then single tokens of growing size (scales grow, earlier codes are
    rounded again), then a piece that crosses pages; every byte of the cache compared, so what
    lies behind the last row and other sequences' pages stay as they were."""
    rng = np.random.RandomState(P + d)
    H, ns = 2, [1, P, 2 * P + 3, 17, 0]
    extra = [2, P + 5, 9, 1, 3]
    final = [n + 4 + e for n, e in zip(ns, extra)]
    table, pages = page_tables(final, P, P)
    c = Cache(A, table, pages, H, P, d)
    lens = list(ns)
    c.append(*kv(rng, H, sum(ns), d), ns, lens)
    c.same()
    for step in range(4):
        lens = [n + 1 for n in lens]
        c.append(*kv(rng, H, 5, d, gain=2.0 ** (2 * step - 2)), [1] * 5, lens)
        c.same()
    lens = [n + e for n, e in zip(lens, extra)]
    c.append(*kv(rng, H, sum(extra), d), extra, lens)
    c.same()


@pytest.mark.parametrize("P,H,d,ns", [
    (16, 8, 64, [2600, 17, 1]), (32, 9, 128, [3000, 1500, 0, 33]), (16, 33, 128, [520, 100]),     # many small pages
    (128, 9, 128, [1] * 40 + [97]), (64, 3, 64, [1, 0, 1] * 20 + [70]),                          # a piece among single rows
])
def test_append_many_rows_in_one_page_of_a_warp(A, P, H, d, ns):
    rng = np.random.RandomState(P + H)
    had = rng.randint(0, 2 * P, len(ns))
    lens = [int(h) + n for h, n in zip(had, ns)]
    table, pages = page_tables(lens, P, 3)
    c = Cache(A, table, pages, H, P, d)
    c.append(*kv(rng, H, int(had.sum()), d, gain=0.25), had.tolist(), had.tolist())
    c.same()
    k, v = kv(rng, H, sum(ns), d)
    k[0, :, 5] = float("inf")
    v[H - 1, ::3, d - 1] = float("nan")
    c.append(k, v, ns, lens)
    c.same()


def test_append_strided_projection(A):
    """K, V as views of a fused projection, [tokens, heads, d]."""
    rng = np.random.RandomState(1)
    H, P, d, ns = 3, 32, 128, [33, 5]
    table, pages = page_tables(ns, P)
    c = Cache(A, table, pages, H, P, d)
    proj = bf16(rng.randn(38, 4 + 2 * H, d))
    k, v = proj[:, 4:4 + H].transpose(0, 1), proj[:, 4 + H:].transpose(0, 1)
    on = proj.to(DEV)
    c.append(k, v, ns, ns, views=(on[:, 4:4 + H].transpose(0, 1), on[:, 4 + H:].transpose(0, 1)))
    c.same()


def test_append_nonfinite_zero_and_extreme_rows(A):
    H, P, d = 1, 16, 64
    table, pages = page_tables([9], P)
    c = Cache(A, table, pages, H, P, d)
    x = np.zeros((1, 9, d), np.float32)
    x[0, 1, :5] = [np.inf, -np.inf, np.nan, 7.0, -0.0]
    x[0, 2] = 1e-38
    x[0, 3, 0] = 3e38
    x[0, 5, 1] = 1e-40
    x = bf16(x)
    for i in range(4):                                     # one by one: 0, then non-finite, tiny, huge
        c.append(x[:, i:i + 1], x[:, 8 - i:9 - i], [1], [i + 1])
        c.same()
    c.append(x[:, 4:], x[:, :5], [5], [9])
    c.same()


def test_append_many_sequences(A):
    """More sequences than a block has threads, some without new rows."""
    rng = np.random.RandomState(8)
    B, H, P, d = 700, 1, 16, 64
    ns = rng.randint(0, 4, B).tolist()
    before = rng.randint(0, 20, B).tolist()
    lens = [a + b for a, b in zip(ns, before)]
    table, pages = page_tables(lens, P)
    c = Cache(A, table, pages, H, P, d)
    c.append(*kv(rng, H, sum(before), d), before, before)
    c.append(*kv(rng, H, sum(ns), d), ns, lens)
    c.same()


def test_append_refuses_bad_offsets_and_pages(A):
    rng = np.random.RandomState(2)
    H, P, d, lens = 2, 16, 64, [20, 7]
    table, pages = page_tables(lens, P)
    k, v = (t.to(DEV) for t in kv(rng, H, 27, d))
    good = np.asarray(offsets(lens))
    for cu, ln, tab in (([1, 20, 27], lens, table), ([0, 28, 27], lens, table), ([0, 20, 26], lens, table), (good, [19, 7], table),
                        (good, [20, 3 * P + 1], table), (good, [-1, 7], table)):
        c = Cache(A, np.asarray(tab), pages, H, P, d)
        A.attn_kv_append_fp8(k, v, c.gpu["k"][0], c.gpu["v"][0], c.gpu["k"][1], c.gpu["v"][1], c.dtable,
                             dev(np.asarray(cu, np.int32)), dev(np.asarray(ln, np.int32)))
        assert A.attn_device_status(True) == INVALID
        c.same()                                            # nothing written
    for entry in (-1, pages, 2 ** 31 - 1, -2 ** 31):        # the first page of sequence 0 is bad; the others are written
        bad = table.copy()
        c = Cache(A, bad, pages, H, P, d)
        c.append(*(t.cpu() for t in (k, v)), lens, lens)
        page = bad[0, 0]
        bad[0, 0] = entry
        fresh = Cache(A, bad, pages, H, P, d)
        A.attn_kv_append_fp8(k, v, fresh.gpu["k"][0], fresh.gpu["v"][0], fresh.gpu["k"][1], fresh.gpu["v"][1], dev(bad),
                             dev(good), dev(np.asarray(lens, np.int32)))
        assert A.attn_device_status(True) == INVALID
        for n in "kv":
            for got, want, was in zip(fresh.gpu[n], c.host[n], fresh.host[n]):
                got = got.cpu().numpy()
                assert (got[page] == was[page]).all()
                others = np.arange(pages) != page
                assert (got[others] == want[others]).all()


# ------------------------------------------------------------------ attention
def attend(A, c, max_q=None, causal=True, scale=None, **kw):
    d = c["q"].shape[2]
    ns = np.diff(c["cu"])
    o, lse = A.attn_fwd_kv_fp8(c["q"].to(DEV), dev(c["k_cache"]), dev(c["v_cache"]), dev(c["k_scale"]), dev(c["v_scale"]),
                               dev(c["table"]), dev(c["cu"]), dev(c["lens"]), int(max(ns)) if max_q is None else max_q,
                               causal=causal, scale=scale, **kw)
    return o, lse


def reference(c, causal=True, scale=None):
    d = c["q"].shape[2]
    return oc.attend(c["q"].float().numpy(), c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], c["table"], c["cu"],
                     c["lens"], causal, d ** -0.5 if scale is None else scale)


def run_check(A, c, causal=True, scale=None, max_q=None):
    o, lse = attend(A, c, max_q, causal, scale)
    check(o, lse, reference(c, causal, scale), c["q"].shape[2])


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", [(1, 1), (4, 4), (8, 2), (7, 1), (6, 2), (16, 1), (12, 4)])
def test_decode(A, P, d, heads):
    """One query per sequence; lengths around every tile and page border."""
    lens = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 500]
    run_check(A, filled(lens, [1] * len(lens), *heads, P, d, seed=P + d))


@pytest.mark.parametrize("n", [2, 3, 4, 5, 8])
@pytest.mark.parametrize("heads", [(4, 4), (8, 2), (8, 1), (3, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_drafts(A, n, heads, causal):
    lens = [n, n + 1, 16, 100, 129, 300]
    run_check(A, filled(lens, [n] * len(lens), *heads, 32, 128, seed=n), causal)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,P", [((4, 1), 16), ((2, 2), 64), ((6, 2), 128), ((8, 1), 32), ((5, 1), 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_pieces(A, d, heads, P, causal):
    """Pieces of prompts of ragged sizes, whole prompts and single tokens in one call."""
    lens, ns = [130, 257, 64, 300, 1, 129, 511, 40], [130, 100, 1, 3, 1, 128, 257, 0]
    run_check(A, filled(lens, ns, *heads, P, d, seed=P), causal)


@pytest.mark.parametrize("case", [
    dict(lens=[2000], ns=[1], heads=(8, 2)),               # few rows over many keys: split and joined
    dict(lens=[3001, 1], ns=[1, 1], heads=(4, 1)),
    dict(lens=[2500, 30, 700], ns=[70, 30, 1], heads=(4, 1)),
    dict(lens=[1500], ns=[300], heads=(2, 1)),
    dict(lens=[900] * 40, ns=[1] * 40, heads=(8, 8)),
    dict(lens=[40] * 300, ns=[1] * 300, heads=(2, 2)),     # more units than CTAs
])
def test_long_and_many(A, case):
    run_check(A, filled(case["lens"], case["ns"], *case["heads"], 64, 128, seed=9))


@pytest.mark.parametrize("d,P", [(64, 16), (128, 32), (128, 128)])
@pytest.mark.parametrize("heads,n", [((4, 1), 5), ((8, 1), 16), ((2, 1), 40), ((12, 1), 10)])
def test_units_of_one_tile(A, heads, n, d, P):
    """Up to 128 rows per sequence and K/V head: two tiles share a unit's key blocks, odd and even
    numbers of them, cut between CTAs or not, alone and beside units of two tiles."""
    lens = [n, 128, 129, 256, 257, 300, 640, 641, 5000]
    run_check(A, filled(lens, [n] * len(lens), *heads, P, d, seed=n + P))
    ns = [n, 128, 1, 200, 2, 0, n, 500, n]
    run_check(A, filled(lens, ns, *heads, P, d, seed=n + P + 1))
    run_check(A, filled([3, 130, 700, 0, 1500], [n] * 5, *heads, P, d, seed=n), causal=False)
    run_check(A, filled([9001], [n], *heads, P, d, seed=n))


@pytest.mark.parametrize("n", [1, 40])
def test_no_visible_key(A, n):
    """Sequences without keys (not causal): O = 0 and LSE = -inf; without queries: nothing."""
    c = filled([0, 50, 0, 33], [n, n, 0, 2], 4, 2, 16, 64, seed=3)
    o, lse = attend(A, c, causal=False)
    assert (o[:, :n] == 0).all() and torch.isneginf(lse[:, :n]).all()
    check(o, lse, reference(c, False), 64)


@pytest.mark.parametrize("n", [1, 5, 60])
def test_magnitudes(A, n):
    """Large scores (a softmax that is nearly one key), scales that differ by 2^20 between pages
    and heads, zero pages, large and tiny queries."""
    for gain, qs in ((8.0, 1.0), (1.0, 2.0 ** 40), (2.0 ** -30, 1.0), (1.0, 2.0 ** -100)):
        c = filled([200, 64, 130], [n, min(n, 64), n], 4, 2, 16, 128, seed=5, gain=gain)
        c["q"] = bf16(c["q"].float().numpy() * qs)
        run_check(A, c, scale=128 ** -0.5 if qs < 2 else 128 ** -0.5 / qs)
    c = filled([200, 64, 130], [n, min(n, 64), n], 4, 2, 16, 128, seed=6)
    rng = np.random.RandomState(0)
    f = np.exp2(rng.randint(-10, 11, c["v_scale"].shape)).astype(np.float32)
    f[rng.rand(*f.shape) < 0.2] = 0
    c["v_scale"] = c["v_scale"] * f
    c["k_scale"] = (c["k_scale"] * np.exp2(rng.randint(-3, 2, f.shape))).astype(np.float32)
    c["k_scale"][rng.rand(*f.shape) < 0.2] = 0
    c["k_scale"][c["k_scale"] > 1e6] = 1.0
    run_check(A, c)
    c["v_scale"] *= np.float32(1.7)                        # scales that are no powers of two
    c["k_scale"] *= np.float32(0.3)
    run_check(A, c)


@pytest.mark.parametrize("n", [1, 33])
def test_nonfinite_keys_and_queries(A, n):
    """A NaN key or query reaches its own rows and heads only; infinite queries likewise."""
    c = filled([100, 90], [n, n], 4, 2, 32, 64, seed=8)
    c["k_cache"][c["table"][0, 1], 1, 3, 5] = 0x7F         # sequence 0, key 35, K/V head 1
    q = c["q"].float().numpy()
    q[0, n, 7] = np.nan                                    # sequence 1, first row, head 0
    q[3, n, 2] = np.inf
    clean = dict(c, q=bf16(np.where(np.isfinite(q), q, 0)))
    clean["k_cache"] = c["k_cache"].copy()
    clean["k_cache"][c["table"][0, 1], 1, 3, 5] = 0
    c["q"] = bf16(q)
    o, lse = attend(A, c, causal=False)
    o2, lse2 = attend(A, clean, causal=False)
    assert torch.isnan(o[2:, :n]).all() and torch.isnan(o[0, n]).all() and torch.isnan(o[3, n]).all()
    ok = torch.ones(4, 2 * n, dtype=torch.bool, device=DEV)
    ok[2:, :n], ok[0, n], ok[3, n] = False, False, False
    assert torch.equal(o[ok], o2[ok]) and torch.equal(lse[ok], lse2[ok])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P", [16, 128])
@pytest.mark.parametrize("n,heads,lens", [
    (5, (6, 2), [9, 40, 129, 600]),        # few rows
    (16, (1, 1), [16, 47, 3000, 31]),
    (40, (6, 2), [40, 90, 600, 130]),      # tiles
    (300, (2, 2), [300, 513, 2700, 300]),  # several units of queries, cut between CTAs
])
def test_nan_keys_and_values_that_some_queries_do_not_see(A, n, heads, lens, P, d):
    """NaN in keys and values: the queries that see the row are NaN (a value: in its column), the
    others' results are the ones without it, bit for bit."""
    Hq, H = heads
    g = Hq // H
    clean = filled(lens, [n] * len(lens), Hq, H, P, d, seed=n)
    c = dict(clean, k_cache=clean["k_cache"].copy(), v_cache=clean["v_cache"].copy())
    clean["v_cache"] = clean["v_cache"].copy()
    want = torch.zeros(Hq, n * len(lens), d, dtype=torch.bool)
    want_lse = torch.zeros(Hq, n * len(lens), dtype=torch.bool)
    rng = np.random.RandomState(n + P)
    # (sequence, key from the end, K/V head, column, in K)
    spots = [(0, 0, 0, 3, False), (0, 2, H - 1, d - 1, False), (0, n - 1, 0, 17, False), (1, n // 2, 0, 0, False),
             (1, n // 2, 0, 1, False), (2, 1, 0, 5, True), (2, n // 2, H - 1, 40, False), (2, lens[2] - 1, H - 1, 31, False),
             (2, lens[2] // 2, 0, 32, False)] + [(2, int(rng.randint(n)), 0, int(rng.randint(d)), False) for _ in range(4)]
    for b, back, h, col, in_k in spots:
        key = lens[b] - 1 - back
        page, row = c["table"][b, key // P], key % P
        c["k_cache" if in_k else "v_cache"][page, h, row, col] = 0x7F if col & 1 else 0xFF
        if not in_k:
            clean["v_cache"][page, h, row, col] = 0
        sees = np.arange(n) + lens[b] - n >= key
        for hq in range(h * g, (h + 1) * g):
            rows = torch.arange(b * n, (b + 1) * n)[torch.from_numpy(sees)]
            if in_k:
                want[hq, rows] = True
                want_lse[hq, rows] = True
            else:
                want[hq, rows, col] = True
    o, lse = attend(A, c)
    o0, lse0 = attend(A, clean)
    assert not torch.isnan(o0).any()
    assert torch.equal(torch.isnan(o).cpu(), want) and torch.equal(torch.isnan(lse).cpu(), want_lse)
    assert torch.equal(o[~want.to(DEV)], o0[~want.to(DEV)]) and torch.equal(lse[~want_lse.to(DEV)], lse0[~want_lse.to(DEV)])
    again, _ = attend(A, clean)            # nothing of it stays
    assert torch.equal(again, o0)


def test_rows_behind_the_last_key_do_not_matter(A):
    """Stale codes, NaN codes and scales in the cache where no sequence reads: the same bits."""
    for n, lens in ((1, [1, 17, 130]), (50, [50, 77, 200])):
        c = filled(lens, [n] * 3, 8, 2, 64, 128, seed=4)
        a = attend(A, c)
        d = {k: v.copy() if isinstance(v, np.ndarray) else v for k, v in c.items()}
        used = np.zeros(c["k_cache"].shape[0], dtype=bool)
        for b, ln in enumerate(lens):
            for blk in range(-(-ln // 64)):
                used[c["table"][b, blk]] = True
                m = min(64, ln - blk * 64)
                for name in ("k_cache", "v_cache"):
                    d[name][c["table"][b, blk], :, m:] = 0x7F
        for name in ("k_cache", "v_cache"):
            d[name][~used] = 0xFF
        for name in ("k_scale", "v_scale"):
            d[name][~used] = np.nan
        b = attend(A, d)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_shared_pages_and_loose_bound(A):
    """Two sequences over the same pages (a shared prefix), and max_q larger than needed."""
    c = filled([128, 128, 96], [1, 1, 2], 4, 2, 32, 64, seed=2)
    c["table"][1] = c["table"][0]
    run_check(A, c)
    run_check(A, c, max_q=4)
    run_check(A, c, max_q=3)


@pytest.mark.parametrize("heads,n", [((17, 1), 1), ((130, 1), 2), ((256, 1), 1), ((256, 1), 3), ((384, 2), 1), ((85, 1), 4)])
def test_wide_groups(A, heads, n):
    """Groups wider than a 128-row tile, and sizes that leave rows of a 256-row unit unused."""
    run_check(A, filled([n, 129, 300], [n] * 3, *heads, 32, 64, seed=heads[0]))


@pytest.mark.parametrize("n,B", [(1, 900), (6, 150)])
def test_many_sequences(A, n, B):
    """More sequences than threads, with and without queries."""
    rng = np.random.RandomState(B)
    lens = rng.randint(n, 60, B)
    ns = np.where(rng.rand(B) < 0.3, 0, rng.randint(1, n + 1, B))
    run_check(A, filled(lens.tolist(), ns.tolist(), 4, 1, 16, 64, seed=B))


def test_nothing_to_do(A):
    c = filled([40, 7], [2, 0], 4, 2, 16, 64)
    empty = dict(c, q=c["q"][:, :0], cu=np.zeros(3, np.int32))
    o, lse = attend(A, empty, max_q=1)
    assert o.shape == (4, 0, 64) and lse.shape == (4, 0)


@pytest.mark.parametrize("n", [1, 8, 80])
def test_a_wait_that_runs_out(A, n):
    """The first K copy of every CTA is never issued: the waits end, the status says so, and the
    next call is right."""
    c = filled([700, 300], [n, n], 8, 2, 64, 128, seed=17)
    want = attend(A, c)
    torch.cuda.synchronize()
    A.attn_set_debug_knobs(wait_limit_ns=20_000_000)
    A.attn_set_test_hooks(True)
    try:
        attend(A, c)
        assert A.attn_device_status(True) == TIMEOUT
    finally:
        A.attn_set_test_hooks(False)
        A.attn_set_debug_knobs()
    got = attend(A, c)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_debug_synchronisation_reports_bad_offsets(A):
    """sync_check: the call itself raises what the device check found."""
    c = filled([40, 50], [20, 3], 4, 2, 16, 64, seed=1)
    A.attn_set_debug_knobs(sync_check=True)
    try:
        attend(A, c)
        with pytest.raises(A.AttnError) as e:
            attend(A, dict(c, lens=np.array([10, 50], np.int32)))            # fewer keys than queries
        assert e.value.code == INVALID
        A.attn_device_status(True)
        with pytest.raises(A.AttnError) as e:
            attend(A, dict(c, table=c["table"] + 1000))
        assert e.value.code == INVALID and "page table" in str(e.value)
    finally:
        A.attn_set_debug_knobs()
        A.attn_device_status(True)


def test_bad_offsets_and_pages(A):
    c = filled([40, 50], [2, 3], 4, 2, 16, 64, seed=1)
    for key, val in (("cu", [0, 2, 4]), ("cu", [1, 2, 5]), ("cu", [0, 6, 5]), ("lens", [1, 50]), ("lens", [40, 65 + 16]),
                     ("lens", [-1, 50])):
        bad = dict(c, **{key: np.asarray(val, np.int32)})
        o, lse = torch.full((4, 5, 64), 3.0, dtype=torch.bfloat16, device=DEV), torch.full((4, 5), 3.0, device=DEV)
        attend(A, bad, max_q=3, o=o, lse=lse)
        assert A.attn_device_status(True) == INVALID
        assert (o == 3).all() and (lse == 3).all()
    attend(A, c, max_q=2)
    assert A.attn_device_status(True) == INVALID
    good = attend(A, c)
    for entry in (-1, c["k_cache"].shape[0], 2 ** 31 - 1, -2 ** 31):
        bad = dict(c, table=c["table"].copy())
        bad["table"][0, 1] = entry
        o, lse = attend(A, bad)
        assert A.attn_device_status(True) == INVALID
        assert torch.equal(o[:, 2:], good[0][:, 2:]) and torch.equal(lse[:, 2:], good[1][:, 2:])


def test_repeatable(A):
    for ns in ([1] * 3, [70, 1, 200]):
        c = filled([1000, 300, 1700], ns, 8, 2, 64, 128, seed=12)
        a, b = attend(A, c), attend(A, c)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("d", [64, 128])
def test_many_short_units(A, d):
    """Units of one to three key blocks behind one another in a CTA, over and over: no result of one
    unit meets the values of the next."""
    rng = np.random.RandomState(d)
    lens = rng.randint(30, 380, 500)
    c = filled(lens.tolist(), np.minimum(lens, rng.randint(17, 65, 500)).tolist(), 8, 2, 128, d, seed=d)
    g = {k: dev(c[k]) for k in ("k_cache", "v_cache", "k_scale", "v_scale", "table", "cu", "lens")}
    q = c["q"].to(DEV)
    call = lambda: A.attn_fwd_kv_fp8(q, g["k_cache"], g["v_cache"], g["k_scale"], g["v_scale"], g["table"], g["cu"],
                                     g["lens"], 64)
    o, lse = call()
    check(o, lse, reference(c), d)
    for _ in range(40):
        o2, lse2 = call()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_pages_past_32_bits(A):
    """Pages whose byte offset passes 2^32 (and element offset 2^31)."""
    P, H, d = 128, 8, 128                                  # 128 KiB a page
    pages = (5 << 30) // (P * H * d)
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("needs 24 GB free")
    small = filled([300, 129], [1, 2], 8, 8, P, d, seed=3)
    far = np.array([pages - 1, pages - 2, 3, pages // 2 + 1, pages - 7, 0])
    c = dict(small)
    kc, vc = (torch.zeros((pages, H, P, d), dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros((pages, H), device=DEV) for _ in range(2))
    table, at = small["table"].copy(), 0
    for b in range(2):
        for i in range(3 if b == 0 else 2):
            old, new = small["table"][b, i], int(far[at])
            for dst, src in ((kc, "k_cache"), (vc, "v_cache"), (ks, "k_scale"), (vs, "v_scale")):
                dst[new] = dev(small[src][old])
            table[b, i] = new
            at += 1
    o, lse = A.attn_fwd_kv_fp8(c["q"].to(DEV), kc, vc, ks, vs, dev(table), dev(c["cu"]), dev(c["lens"]), 2)
    check(o, lse, reference(small), d)
    # and an appended row lands there
    host = (kc[int(table[1, 1])].cpu().numpy()[None], ks[int(table[1, 1])].cpu().numpy()[None])
    k, v = kv(np.random.RandomState(0), H, 1, d)
    A.attn_kv_append_fp8(k.to(DEV), v.to(DEV), kc, vc, ks, vs, dev(table[1:]), dev(np.array([0, 1], np.int32)),
                         dev(np.array([130], np.int32)))
    oc.append(k.float().numpy(), *host, np.array([[9, 0]]), [0, 1], [130])
    assert (kc[int(table[1, 1])].cpu().numpy() == host[0][0]).all()
    assert (ks[int(table[1, 1])].cpu().numpy() == host[1][0]).all()


def test_streams(A):
    c = filled([1000, 300], [1, 1], 8, 2, 64, 128, seed=12)
    want = attend(A, c)
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        torch.cuda.synchronize()
        got = attend(A, c, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("n", [1, 70])
def test_graph_with_growing_lengths(A, n):
    """Captured once with its buffers, replayed on other queries and longer sequences: what eager
    calls give, bit for bit, for both kernels."""
    c = filled([900, 300, 1500], [n] * 3, 8, 2, 64, 128, seed=31)
    q, lens = c["q"].to(DEV), dev(c["lens"] - 200)
    cache = [dev(c[k]) for k in ("k_cache", "v_cache", "k_scale", "v_scale", "table", "cu")]
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
    ws = torch.empty(A.attn_fwd_kv_fp8_workspace_size(3, 8, 2, 3 * n, n, 128), dtype=torch.uint8, device=DEV)
    call = lambda **kw: A.attn_fwd_kv_fp8(q, *cache, lens, n, **kw)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(o=o, lse=lse, workspace=ws)
        call(o=o, lse=lse, workspace=ws)                   # a workspace serves one call after another
    for step in range(3):
        g.replay()
        torch.cuda.synchronize()
        want = call()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        check(o, lse, reference(dict(c, q=q.cpu(), lens=lens.cpu().numpy())), 128)
        q.copy_(torch.randn(q.shape).to(torch.bfloat16))
        lens += 100
        ws.fill_(0xFF)


@pytest.mark.parametrize("n", [1, 90])
def test_two_calls_at_once(A, n):
    """Two streams, each with its own workspace."""
    cs = [filled([4000, 2000], [n, n], 8, 2, 64, 128, seed=20 + i) for i in range(2)]
    want = [attend(A, c) for c in cs]
    args = [[c["q"].to(DEV)] + [dev(c[k]) for k in ("k_cache", "v_cache", "k_scale", "v_scale", "table", "cu", "lens")] for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i] = A.attn_fwd_kv_fp8(*args[i], n, stream=s)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_binding_refusals(A):
    c = filled([40], [2], 4, 2, 16, 64)
    good = dict(q=c["q"].to(DEV), **{k: dev(c[k]) for k in ("k_cache", "v_cache", "k_scale", "v_scale")}, page_table=dev(c["table"]),
                cu_seqlens_q=dev(c["cu"]), kv_lens=dev(c["lens"]))
    for k, bad in (("q", good["q"].float()), ("q", good["q"][:, :, :32]), ("k_cache", good["k_cache"][..., :32]),
                   ("v_cache", good["v_cache"][1:]), ("k_scale", good["k_scale"].double()), ("v_scale", good["v_scale"][:, :1]),
                   ("page_table", good["page_table"].long()), ("page_table", good["page_table"][0]), ("cu_seqlens_q", good["cu_seqlens_q"][:1]),
                   ("kv_lens", good["kv_lens"].long()), ("kv_lens", good["kv_lens"].cpu()), ("k_cache", good["k_cache"][0])):
        with pytest.raises(ValueError):
            A.attn_fwd_kv_fp8(**{**good, k: bad}, max_q=2)
    for kw in (dict(o=good["q"].float()), dict(lse=torch.zeros(4, 3, device=DEV)), dict(workspace=torch.zeros(4))):
        with pytest.raises(ValueError):
            A.attn_fwd_kv_fp8(**good, max_q=2, **kw)
    for mq in (0, 3):
        with pytest.raises(A.AttnError):
            A.attn_fwd_kv_fp8(**good, max_q=mq)


# ------------------------------------------------------------------ as a decoder uses them
@pytest.mark.parametrize("P,heads,d", [(16, (8, 2), 128), (128, (4, 4), 64)])
def test_decoder_steps(A, P, heads, d):
    """Prompts in two pieces, then single tokens: rotate, append, attend, from a fused
    projection, against the oracles fed with the same projections; then the same token step
    captured once in a graph and replayed with the lengths advanced on the device."""
    rng = np.random.RandomState(P)
    Hq, H = heads
    B, first, second, steps = 3, [20, 1, 37], [30, 140, 3], 4
    total = [a + b + steps + 2 for a, b in zip(first, second)]
    table, pages = page_tables(total, P)
    c = Cache(A, table, pages, H, P, d)
    f, m = A.attn_rope_freqs(d, scaling="yarn", factor=2.0, trained_length=128)
    lens = [0] * B

    def step(ns, proj, dproj, dpos, dcu, dlens, n_max):
        T = proj.shape[0]
        q, k, v = dproj[:, :Hq].transpose(0, 1), dproj[:, Hq:Hq + H].transpose(0, 1), dproj[:, Hq + H:].transpose(0, 1)
        rq, rk = A.attn_rope(q, k, f, dpos, mscale=m)
        A.attn_kv_append_fp8(rk, v, c.gpu["k"][0], c.gpu["v"][0], c.gpu["k"][1], c.gpu["v"][1], c.dtable, dcu, dlens)
        o, lse = A.attn_fwd_kv_fp8(rq, c.gpu["k"][0], c.gpu["v"][0], c.gpu["k"][1], c.gpu["v"][1], c.dtable, dcu, dlens, n_max)
        return rq, rk, o, lse

    def verify(ns, proj, got):
        """The rotation against its oracle; the rest against oracles fed with the rotated rows."""
        rq, rk, o, lse = got
        pos = np.concatenate([np.arange(ln - n, ln) for ln, n in zip(lens, ns)])[None]
        x = proj.float().numpy().transpose(1, 0, 2).astype(np.float64)
        want = orope.rotate(x[None, :Hq + H], f.cpu().numpy(), pos, False, m)[0]
        both = np.concatenate([t.float().cpu().numpy() for t in (rq, rk)])
        assert (np.abs(both - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -16).all()
        cu = offsets(ns)
        oc.append(rk.float().cpu().numpy(), *c.host["k"], table, cu, lens)
        oc.append(x[Hq + H:], *c.host["v"], table, cu, lens)
        c.same()
        ref = oc.attend(rq.float().cpu().numpy(), c.host["k"][0], c.host["v"][0], c.host["k"][1], c.host["v"][1], table, cu,
                        lens, True, d ** -0.5)
        check(o, lse, ref, d)

    for ns in (first, second) + ([1] * B,) * 2:
        lens = [a + b for a, b in zip(lens, ns)]
        proj = bf16(rng.randn(sum(ns), Hq + 2 * H, d))
        pos = np.concatenate([np.arange(ln - n, ln) for ln, n in zip(lens, ns)]).astype(np.int32)
        verify(ns, proj, step(ns, proj, proj.to(DEV), dev(pos), dev(offsets(ns)), dev(np.asarray(lens, np.int32)), max(ns)))

    ns = [1] * B
    dproj = torch.zeros((B, Hq + 2 * H, d), dtype=torch.bfloat16, device=DEV)
    dcu, dlens = dev(offsets(ns)), dev(np.asarray(lens, np.int32) + 1)
    dpos = dlens - 1
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(ns, dproj, dproj, dpos, dcu, dlens, 1)
    for i in range(steps):
        proj = bf16(rng.randn(B, Hq + 2 * H, d))
        dproj.copy_(proj)
        lens = [n + 1 for n in lens]
        g.replay()
        torch.cuda.synchronize()
        verify(ns, proj, got)
        dlens += 1
        dpos += 1
