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
