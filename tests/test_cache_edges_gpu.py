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
