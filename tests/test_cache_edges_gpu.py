"""Cached attention, append and rotary positions where they are easily wrong: results joined within a
block, streams given as numbers, pages of scale 0, queries with one dominating or infinite component,
loose bounds, empty sequences among large units."""
import numpy as np
import pytest
import torch

import oracle.cache as oc
from cache_cases import bf16, check, filled, offsets, page_tables
from test_cache_gpu import Cache, attend, dev, kv, reference, run_check

pytestmark = pytest.mark.gpu
DEV = "cuda"


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


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,n", [((8, 1), 1), ((16, 1), 1), ((4, 1), 4)])
def test_warps_join_the_same_way_every_time(A, heads, n, d):
    """Few rows, many units per block, the four warps' maxima and V scales far apart: whoever reads
    another warp's statistics reads them before the slot is used again, so that every run gives the
    same bits."""
    rng = np.random.RandomState(d + n)
    lens = rng.randint(n + 1, 200, 400)
    c = filled(lens.tolist(), [n] * 400, *heads, 32, d, seed=n + d, gain=2.0)
    c["v_scale"] = (c["v_scale"] * np.exp2(rng.randint(-6, 7, c["v_scale"].shape))).astype(np.float32)
    g = {k: dev(c[k]) for k in ("k_cache", "v_cache", "k_scale", "v_scale", "table", "cu", "lens")}
    q = c["q"].to(DEV)
    call = lambda: A.attn_fwd_kv_fp8(q, g["k_cache"], g["v_cache"], g["k_scale"], g["v_scale"], g["table"], g["cu"],
                                     g["lens"], n)
    o, lse = call()
    check(o, lse, reference(c), d)
    for _ in range(100):
        o2, lse2 = call()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_stream_zero_is_the_default_stream(A):
    """The number 0 (cuda_stream of the default stream) names the default stream for the three
    operators, as it does for the library's other calls: what they do comes after what is already on it."""
    zero = torch.cuda.default_stream().cuda_stream
    assert zero == 0
    c = filled([700, 300], [2, 2], 8, 2, 64, 128, seed=2)
    want = attend(A, c)
    f, m = A.attn_rope_freqs(128)
    x = bf16(np.random.RandomState(0).randn(2, 4, 128)).to(DEV)
    want_x, _ = A.attn_rope(x, None, f)
    g = {k: dev(c[k]) for k in ("k_cache", "v_cache", "k_scale", "v_scale", "table", "cu", "lens")}
    q, qx = torch.zeros_like(c["q"], device=DEV), torch.zeros_like(x)
    src, busy = c["q"].to(DEV), torch.randn(4096, 4096, device=DEV)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):                          # the current stream is another one
        with A._there(q.device, zero):
            assert torch.cuda.current_stream().cuda_stream == 0
        with torch.cuda.stream(torch.cuda.default_stream()):
            for _ in range(20):
                busy = (busy @ busy).clamp_(-1, 1)         # the inputs are written late
            q.copy_(src)
            qx.copy_(x)
        o, lse = A.attn_fwd_kv_fp8(q, g["k_cache"], g["v_cache"], g["k_scale"], g["v_scale"], g["table"], g["cu"],
                                   g["lens"], 2, stream=zero)
        y, _ = A.attn_rope(qx, None, f, stream=zero)
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1]) and torch.equal(y, want_x)
    table, pages = page_tables([4], 16)
    cache = Cache(A, table, pages, 2, 16, 128)
    late = torch.zeros_like(qx)
    with torch.cuda.stream(side):
        with torch.cuda.stream(torch.cuda.default_stream()):
            for _ in range(20):
                busy = (busy @ busy).clamp_(-1, 1)
            late.copy_(x)
        A.attn_kv_append_fp8(late, late, cache.gpu["k"][0], cache.gpu["v"][0], cache.gpu["k"][1], cache.gpu["v"][1],
                             cache.dtable, dev(offsets([4])), dev(np.array([4], np.int32)), stream=zero)
    torch.cuda.synchronize()
    for n in "kv":
        oc.append(x.float().cpu().numpy(), *cache.host[n], table, offsets([4]), [4])
    cache.same()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P,n", [(16, 1), (128, 1), (16, 9), (128, 100)])
def test_append_to_a_page_of_scale_zero(A, P, n, d):
    """A first row without a finite value other than 0, then finite rows (few and many: both kernels).
    The first row reads the same values before and after, byte for byte as the oracle has it."""
    rng = np.random.RandomState(P + n)
    table, pages = page_tables([1 + n], P)
    c = Cache(A, table, pages, 2, P, d)
    x = np.zeros((2, 1, d), np.float32)
    x[:, 0, :6] = [np.inf, -np.inf, np.nan, 0.0, -0.0, np.inf]
    y = np.where(np.isnan(x), x, -x)
    c.append(bf16(x), bf16(y), [1], [1])
    c.same()
    assert (c.gpu["k"][1][int(table[0, 0])] == 0).all()
    c.append(*kv(rng, 2, n, d), [n], [1 + n])
    c.same()
    first = c.gpu["k"][0][int(table[0, 0]), :, 0].cpu().numpy()
    assert (first[:, [0, 1, 5]] & 0x7F == 0).all() and (first[:, 2] & 0x7F == 0x7F).all()


def check_with_query_error(o, lse, c, scale, bits):
    """As cache_cases.check, with components of q off by up to 2^-bits of their row's largest: a score is
    then off by 2^-bits scale max_c |q_c| sum_c |k_jc| more."""
    O, L, W, Z = reference(c, scale=scale)
    d, g = c["q"].shape[2], c["q"].shape[0] // c["k_cache"].shape[1]
    peak = np.abs(c["q"].float().numpy()).max(axis=-1).astype(np.float64)                  # [Hq, T]
    more = np.zeros_like(peak)
    for b, n in enumerate(c["lens"]):
        sl = slice(c["cu"][b], c["cu"][b + 1])
        for h in range(peak.shape[0]):
            k = oc.rows(c["k_cache"], c["k_scale"], c["table"][b], int(n), h // g)
            more[h, sl] = 2.0 ** -bits * scale * peak[h, sl] * np.abs(k).sum(axis=1).max()
    # (bounds multiplies Z by this)
    check(o, lse, (O, L, W, Z + more / ((d + 8) * 2.0 ** -24 + 2.0 ** -22)), d)


def one_large_component(n, factor, d, P, heads):
    """Queries whose column 5 is `factor` times the others, keys that are 0 there: the scores are made of
    the small components alone."""
    lens = [n + 3, 200, 129]
    c = filled(lens, [n] * 3, *heads, P, d, seed=n + d)
    q = c["q"].float().numpy()
    q[..., 5] *= factor
    c["q"] = bf16(q)
    c["k_cache"][..., 5] = 0
    return c


@pytest.mark.parametrize("factor", [10, 50, 200, 1000, 30000])
@pytest.mark.parametrize("n,heads,P,d", [(5, (4, 1), 32, 128), (40, (4, 1), 16, 64), (90, (4, 1), 128, 128), (70, (6, 2), 64, 64)])
def test_queries_with_one_large_component_on_the_tiles(A, n, heads, P, d, factor):
    c = one_large_component(n, factor, d, P, heads)
    o, lse = attend(A, c)
    check_with_query_error(o, lse, c, d ** -0.5, 21)


@pytest.mark.parametrize("n", [5, 90])
def test_query_components_stay_exact_down_to_2_13_of_the_largest(A, n):
    """128 beside 127 * 2^-10 (2^-10 of it) and 151 * 2^-13 (in the last binade that is held exactly), with
    all bits of a bf16 in use: the small ones make the score, so what cache_cases.bounds claims for exact
    operands holds."""
    c = filled([n + 3, n + 200], [n] * 2, 4, 1, 32, 128, seed=1)
    q = np.zeros(c["q"].shape, np.float32)
    q[..., 0], q[..., 1], q[..., 2] = 128, 127 * 2.0 ** -10, 151 * 2.0 ** -13
    c["q"] = bf16(q)
    c["k_cache"][..., 0] = 0
    run_check(A, c, scale=1.0)


@pytest.mark.parametrize("factor", [10, 1000, 30000, 2.0 ** 27])
@pytest.mark.parametrize("n,heads,P,d", [(1, (8, 2), 16, 128), (4, (4, 1), 32, 128), (2, (3, 1), 128, 64)])
def test_queries_with_one_large_component_on_few_rows(A, n, heads, P, d, factor):
    c = one_large_component(n, factor, d, P, heads)
    o, lse = attend(A, c)
    check_with_query_error(o, lse, c, d ** -0.5, 39)


@pytest.mark.parametrize("n", [1, 4, 5, 40, 90])
def test_queries_at_both_ends_of_the_exponent(A, n):
    """Rows whose largest component is in bf16's last binade, or near its first normal one, with a scale that
    makes ordinary scores of them."""
    for e in (127, 126, 100, -90):
        c = filled([n + 3, 70 + n], [n] * 2, 4, 1, 32, 128, seed=3)
        q = c["q"].float().numpy()
        q = np.sign(q) * np.minimum(np.abs(q), 1.9)
        q[..., 0] = 1.9                                    # a row's largest, in its exponent's binade
        c["q"] = bf16(q * 2.0 ** e)
        c["k_scale"] = (c["k_scale"] * 2.0 ** (-60 if e > 0 else 60)).astype(np.float32)
        c["k_scale"][c["k_scale"] > 2.0 ** 90] = 0         # of pages that nobody uses
        run_check(A, c, scale=128 ** -0.5 * 2.0 ** ((60 if e > 0 else -60) - e))


@pytest.mark.parametrize("n", [1, 4, 5, 40, 90])
@pytest.mark.parametrize("what", [-np.inf, np.inf])
def test_an_infinite_query_is_nan_where_it_sees_a_key(A, n, what):
    """softmax of scores that are all -inf, or infinite in part, is NaN; a row that sees no key is still 0."""
    c = filled([n + 3, 70 + n, 0], [n] * 3, 4, 1, 32, 128, seed=1)
    c["k_cache"][..., 3] = 0x30                            # the same sign at every key
    clean = attend(A, c, causal=False)
    q = c["q"].float().numpy()
    for row in (0, 2 * n):                                 # of the first sequence, and of the one without keys
        q[0, row] = 0
        q[0, row, 3] = what
    o, lse = attend(A, dict(c, q=bf16(q)), causal=False)
    assert torch.isnan(o[0, 0]).all() and torch.isnan(lse[0, 0])
    assert (o[0, 2 * n] == 0).all() and torch.isneginf(lse[0, 2 * n])
    keep = torch.ones(lse.shape, dtype=torch.bool, device=DEV)
    keep[0, 0] = keep[0, 2 * n] = False
    assert torch.equal(o[keep], clean[0][keep]) and torch.equal(lse[keep], clean[1][keep])


def test_rotary_outputs_in_wider_and_permuted_layouts(A):
    """Outputs whose rows lie apart in any order of the strides: every other head of a wider buffer, tokens
    outermost, batch innermost of the three."""
    x = bf16(np.random.RandomState(3).randn(2, 3, 5, 64)).to(DEV)
    f, m = A.attn_rope_freqs(64)
    want, _ = A.attn_rope(x, None, f)
    wide = torch.full((2, 5, 6, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    for view in (wide[:, :, ::2].transpose(1, 2), torch.empty((5, 3, 2, 64), dtype=torch.bfloat16, device=DEV).permute(2, 1, 0, 3),
                 torch.empty((3, 5, 2, 64), dtype=torch.bfloat16, device=DEV).permute(2, 0, 1, 3)):
        y, _ = A.attn_rope(x, None, f, q_out=view)
        assert y is view and torch.equal(y, want)
    assert (wide[:, :, 1::2] == 9.0).all()
    buf = torch.zeros(4096, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(A.AttnError, match="overlap"):
        A.attn_rope(x, None, f, q_out=buf.as_strided((2, 3, 5, 64), (1024, 64, 64, 1)))
    assert (buf == 0).all()


@pytest.mark.parametrize("bound", [3, 4, 5, 64, 512])
def test_a_constant_bound_over_short_steps(A, bound):
    """A server keeps the workspace of its largest piece and passes min(bound, packed queries): steps with
    fewer rows than the bound, down to a single token, give what the tightest bound gives."""
    for ns, lens in (([1], [300]), ([1, 1], [40, 700]), ([3, 1, 2], [3, 90, 500])):
        c = filled(lens, ns, 8, 2, 32, 64, seed=len(ns))
        ws = torch.full((A.attn_fwd_kv_fp8_workspace_size(len(ns), 8, 2, sum(ns), bound, 64),), 0xFF, dtype=torch.uint8, device=DEV)
        o, lse = attend(A, c, max_q=min(bound, sum(ns)), workspace=ws)
        check(o, lse, reference(c), 64)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", [(4, 1), (8, 2)])
def test_sequences_without_keys_among_units_of_two_tiles(A, heads, d):
    """Units of 256 rows beside sequences without keys, without queries, and short ones (not causal)."""
    lens, ns = [0, 300, 0, 700, 0, 5, 0], [200, 300, 0, 130, 1, 0, 70]
    c = filled(lens, ns, *heads, 64, d, seed=3)
    o, lse = attend(A, c, causal=False)
    check(o, lse, reference(c, False), d)
    for b, n in enumerate(lens):
        if n == 0:
            sl = slice(c["cu"][b], c["cu"][b + 1])
            assert (o[:, sl] == 0).all() and torch.isneginf(lse[:, sl]).all()
