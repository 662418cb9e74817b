"""Bounds that attn_rope_kv_append_fp8 keeps when rows are given up again, as drafts that were not taken."""
import numpy as np
import pytest
import torch

from cache_cases import offsets

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_given_up_still_count_until_the_page_starts_anew(P, d):
    import attention_attn_fwd_09_gb300 as A
    H, e4m3 = 2, torch.float8_e4m3fn
    rng = np.random.RandomState(P + d)
    kc, vc = (torch.zeros(3, H, P, d, dtype=torch.uint8, device=DEV) for _ in "kv")
    ks, vs = (torch.zeros(3, H, device=DEV) for _ in "kv")
    bounds = torch.full((3, H, 2, d), 0x7F, dtype=torch.uint8, device=DEV)
    table = torch.tensor([[2, 0]], dtype=torch.int32, device=DEV)

    def append(n, length, span):
        x = torch.as_tensor(rng.uniform(-span, span, (H, n, d)).astype(np.float32)).to(torch.bfloat16)
        x[:, 0, 0] = 448                                   # the scale is 1 throughout: codes are the values, rounded
        on = x.to(DEV)
        A.attn_rope_kv_append_fp8(None, on, on, None, kc, vc, ks, vs, table, torch.as_tensor(offsets([n])).to(DEV),
                                  torch.tensor([length], dtype=torch.int32, device=DEV), k_bounds=bounds)
        assert A.attn_device_status(True) == 0
        return x.to(e4m3).float()

    def kept():
        return bounds[2].view(e4m3).float().cpu()

    first = append(6, 6, 100.0)
    second = append(2, 5, 10.0)                            # three rows given up, two others in their place
    rows = kc[2].view(e4m3).float().cpu()[:, :5]
    assert torch.equal(rows, torch.cat((first[:, :3], second), 1))
    both = torch.cat((first, second), 1)
    assert torch.equal(kept(), torch.stack((both.amin(1), both.amax(1)), 1))
    assert (kept()[:, 0] <= rows.amin(1)).all() and (kept()[:, 1] >= rows.amax(1)).all()
    third = append(4, 4, 5.0)                              # from the page's first row on
    assert torch.equal(kept(), torch.stack((third.amin(1), third.amax(1)), 1))
