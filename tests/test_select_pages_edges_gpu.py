"""attn_select_pages_fp8 where scores are tiny or their terms far apart: lists still equal those of 64-bit scores."""
import numpy as np
import pytest
import torch

from test_select_pages_gpu import check, made

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


@pytest.mark.parametrize("down", [20, 30, 40, 44, 48, 52, 56, 60, 80, 110])
@pytest.mark.parametrize("Hq,H,d", [(4, 2, 64), (20, 1, 128)])
def test_scores_below_the_fp32_range(A, down, Hq, H, d):
    """q around 2^-100 and scales down to 2^-115: scores, and bounds on their error, below the smallest fp32 number."""
    c = made([16 * 120, 16 * 50], [1, 2], Hq, H, 16, d, seed=down)
    c["q"] = (c["q"].float() * 2.0 ** -100).to(torch.bfloat16)
    c["scale"] = c["scale"] * np.float32(2.0 ** -down)
    check(A, c, 12, 1, 2)
