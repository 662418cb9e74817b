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


@pytest.mark.parametrize("small", [34, 44, 48, 50, 52, 90, 240])
@pytest.mark.parametrize("Hq,H,d", [(4, 2, 64), (4, 1, 128), (7, 1, 128)])
def test_terms_far_apart(A, small, Hq, H, d):
    """A few large components against columns that all pages share, the others 2^-small of them: the order of
    pages lies in the last bits of 64-bit scores, or below them (then by number).  small = 240: of the smallest
    ones q can hold."""
    c = made([32 * 300], [2], Hq, H, 32, d, seed=small)
    c["bounds"][:, :, :, :4] = c["bounds"][:1, :, :, :4]
    c["scale"][:] = 0.25
    q = c["q"].float() * (2.0 ** 120 if small == 240 else 1.0)
    q[..., 4:] *= 2.0 ** -small
    c["q"] = q.to(torch.bfloat16)
    check(A, c, 50, 1, 1)
    check(A, c, 200, 0, 3)


def test_terms_far_apart_that_cancel(A):
    """The large terms cancel, all but exactly: what is left decides."""
    c = made([32 * 300], [2], 2, 1, 32, 128, seed=3)
    b = c["bounds"]
    b[:, :, 1, 0] = b[:, :, 0, 0] = 0x38                   # 1, in every page
    b[:, :, 1, 5] = b[:, :, 0, 5] = 0x38
    q = c["q"].float() * 2.0 ** -45
    q[..., 0], q[..., 5] = 1.5, -1.5
    c["q"] = q.to(torch.bfloat16)
    check(A, c, 50, 1, 1)
