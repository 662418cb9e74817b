"""attn_select_pages_fp8 against the definition in 64 bits (sums without rounding): the lists are whole
numbers and have to be equal, near ties, exact ties, NaN and infinities included."""
import numpy as np
import pytest
import torch

import oracle.sparse as osp
from cache_cases import bf16, offsets, page_tables
from oracle.fp8 import e4m3_decode

pytestmark = pytest.mark.gpu
DEV = "cuda"
INVALID = -1


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


def made(lens, ns, Hq, H, P, d, seed=0, spread=40):
    """Random bounds (any finite codes, lo <= hi), scales around 2^-3 and random queries."""
    rng = np.random.RandomState(seed)
    table, pages = page_tables(lens, P, seed)
    codes = rng.randint(0, spread, (pages, H, 2, d)) + 60 - spread // 2
    codes = (codes | (rng.randint(0, 2, codes.shape) << 7)).astype(np.uint8)
    x = e4m3_decode(codes)
    swap = x[:, :, :1] > x[:, :, 1:]
    codes = np.where(swap, codes[:, :, ::-1], codes)
    scale = np.exp2(rng.randint(-5, -2, (pages, H))).astype(np.float32)
    return dict(bounds=codes, scale=scale, table=table, cu=offsets(ns), lens=np.asarray(lens, np.int32),
                q=bf16(rng.randn(Hq, int(sum(ns)), d)), P=P)


def run(A, c, count, first, last, causal=True, max_q=None, **kw):
    n = int(np.diff(c["cu"]).max()) if max_q is None else max_q
    return A.attn_select_pages_fp8(dev(c["q"]), dev(c["bounds"]), dev(c["scale"]), dev(c["table"]), dev(c["cu"]), dev(c["lens"]),
                                   c["P"], count, n, first=first, last=last, causal=causal, **kw)


def check(A, c, count, first, last, causal=True, **kw):
    got = run(A, c, count, first, last, causal, **kw).cpu().numpy()
    want = osp.select_pages(c["q"].float().numpy(), e4m3_decode(c["bounds"]), c["scale"], c["table"], c["cu"], c["lens"], c["P"],
                            count, first, last, causal)
    assert (got == want).all(), np.argwhere((got != want).any(-1))[:5]


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,H", [(8, 2), (3, 3), (7, 1), (16, 1), (20, 1), (64, 2)])
def test_lengths_and_groups(A, P, d, Hq, H):
    c = made([1, P, 3 * P + 1, 20 * P - 1, 41 * P + 5], [1, 2, 1, 5, 3], Hq, H, P, d, seed=P + d + Hq)
    check(A, c, 9, 1, 2)
    check(A, c, 5, 0, 0, causal=False)
    check(A, c, 4, 3, 1)                                   # nothing left to choose
    check(A, c, 1, 0, 1)
    check(A, c, 30, 2, 5, max_q=int(c["cu"][-1]))          # a bound larger than needed


def test_long_tables_and_many_chunks(A):
    c = made([16 * 1500 + 3], [1], 4, 1, 16, 64, seed=1)
    check(A, c, 100, 1, 2)
    check(A, c, 1400, 10, 20)
    c = made([16 * 300, 16 * 40, 5] * 9, [1, 2, 1] * 9, 4, 2, 16, 128, seed=2)
    check(A, c, 33, 1, 1)


def test_more_pages_than_shared_memory_holds(A):
    c = made([16 * 11000 - 7], [2], 2, 1, 16, 64, seed=3)
    check(A, c, 50, 1, 1)


def test_more_sequences_than_threads(A):
    ns = [1, 0, 2] * 120
    c = made([16 * (3 + i % 9) + i % 16 for i in range(360)], ns, 2, 1, 16, 64, seed=4)
    check(A, c, 4, 1, 1)


def test_equal_scores_go_by_number(A):
    """Pages that are copies of one another, of a few kinds, and all alike."""
    for kinds in (1, 2, 5):
        c = made([16 * 700], [1], 4, 2, 16, 64, seed=5 + kinds)
        which = np.random.RandomState(kinds).randint(0, kinds, len(c["bounds"]))
        c["bounds"], c["scale"] = c["bounds"][which], c["scale"][which]
        check(A, c, 40, 1, 2)
        check(A, c, 400, 0, 0)


def test_scores_that_32_bits_cannot_tell_apart(A):
    """Pages that differ in the smallest code of one column only, where the query is small too: the order of
    their scores is far below the rounding of an fp32 sum."""
    rng = np.random.RandomState(7)
    c = made([32 * 300], [2], 4, 1, 32, 128, seed=8)
    c["bounds"][:] = c["bounds"][:1]
    c["scale"][:] = 0.25
    c["bounds"][:, :, 1, 77] = rng.randint(0, 8, len(c["bounds"]))[:, None]        # 0 .. 7 x 2^-9
    c["bounds"][:, :, 0, 77] = 0x80
    q = c["q"].float()
    q[:, :, 77] = 2.0 ** -18
    c["q"] = q.to(torch.bfloat16)
    check(A, c, 50, 1, 1)
    check(A, c, 200, 0, 3)


def test_zero_keys_and_zero_queries(A):
    c = made([16 * 90, 16 * 20], [1, 1], 4, 2, 16, 64, seed=9)
    c["scale"][:] = 0
    check(A, c, 12, 1, 2)
    c = made([16 * 90], [1], 4, 2, 16, 64, seed=9)
    c["q"].zero_()
    check(A, c, 12, 0, 1)


def test_nan_and_infinities(A):
    base = made([16 * 120, 16 * 50], [1, 2], 4, 2, 16, 64, seed=10)
    nan = {**base, "bounds": base["bounds"].copy()}
    for p in (3, 40, 41, 77):                              # pages with a NaN column are listed first
        nan["bounds"][base["table"][0, p], :, :, 5] = 0x7F
    check(A, nan, 12, 1, 2)
    check(A, nan, 3, 0, 1)                                 # more of them than there is room for
    nan["bounds"][base["table"][0, :120], 1] = 0x7F
    check(A, nan, 12, 1, 2)
    for value in (float("inf"), float("-inf"), float("nan")):
        c = {**base, "q": base["q"].clone()}
        c["q"][1, 0, 3] = value
        check(A, c, 12, 1, 2)
    c = {**base, "q": (base["q"].float() * 1e38).to(torch.bfloat16), "scale": base["scale"] * np.float32(64)}   # past fp32's range
    check(A, c, 12, 1, 2)
    c = {**base, "q": (base["q"].float() * 1e-38).to(torch.bfloat16)}
    check(A, c, 12, 1, 2)


def test_device_checks(A):
    c = made([16 * 30, 40], [1, 2], 4, 2, 16, 64, seed=11)
    out = torch.full((2, 3, 6), 77, dtype=torch.int32, device=DEV)
    for cu, lens in (([0, 1, 2], c["lens"]), ([0, 4, 3], c["lens"]), ([1, 1, 3], c["lens"]), (c["cu"], [480, 1]),
                     (c["cu"], [-1, 40]), (c["cu"], [1 << 20, 40])):
        run(A, {**c, "cu": np.asarray(cu, np.int32), "lens": np.asarray(lens, np.int32)}, 6, 1, 1, max_q=2, pages=out)
        assert A.attn_device_status(True) == INVALID and (out == 77).all()
    run(A, c, 6, 1, 1, max_q=1, pages=out)                 # a bound that is too small
    assert A.attn_device_status(True) == INVALID and (out == 77).all()
    for entry in (-1, len(c["bounds"]), 2 ** 31 - 1):
        table = c["table"].copy()
        table[0, 9] = entry
        run(A, {**c, "table": table}, 6, 1, 1)
        assert A.attn_device_status(True) == INVALID


def test_no_keys_and_no_queries(A):
    c = made([0, 30], [1, 1], 4, 2, 16, 64, seed=12)
    check(A, c, 5, 1, 1, causal=False)
    got = A.attn_select_pages_fp8(torch.empty(4, 0, 64, dtype=torch.bfloat16, device=DEV), dev(c["bounds"]), dev(c["scale"]),
                                  dev(c["table"]), dev(np.zeros(3, np.int32)), dev(c["lens"]), 16, 5, 1)
    assert got.shape == (2, 0, 5)


def test_captured_replayed_and_on_another_stream(A):
    c = made([16 * 200, 16 * 77], [1, 3], 8, 2, 16, 128, seed=13)
    args = [dev(c[n]) for n in ("q", "bounds", "scale", "table", "cu", "lens")] + [16, 20, 3]
    size = A.attn_select_pages_fp8_workspace_size(2, 4, c["table"].shape[1])
    want = A.attn_select_pages_fp8(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = A.attn_select_pages_fp8(*args, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    runs = []
    for _ in range(2):                                     # two graphs, a workspace each
        out, ws = torch.empty_like(want), torch.empty(size, dtype=torch.uint8, device=DEV)
        A.attn_select_pages_fp8(*args, pages=out, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            A.attn_select_pages_fp8(*args, pages=out, workspace=ws)
        runs.append((g, out, ws, torch.cuda.Stream()))
    for _ in range(3):
        args[0].copy_(args[0].roll(1, 2) * -1)
        want = A.attn_select_pages_fp8(*args)
        torch.cuda.synchronize()
        for g, out, ws, s in runs:
            out.fill_(0)
            ws.fill_(0xFF)                                 # NaN everywhere
        torch.cuda.synchronize()
        for g, out, ws, s in runs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, want) for _, out, _, _ in runs)
