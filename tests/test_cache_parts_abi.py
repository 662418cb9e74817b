"""Refusals of the rotating append, page selection, listed-page and shared-prefix attention entry points:
the documented status before anything touches the GPU, and the binding's own checks."""
import ctypes

import pytest
import torch

FAKE, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10002)
BIG, EIGHT = ctypes.c_void_p(0x20000), ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def A():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import attention_attn_fwd_09_gb300 as A
    return A


def append(A, q=FAKE, qo=BIG, k=FAKE, v=FAKE, f=FAKE, pos=None, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, bounds=FAKE, t=FAKE, cu=FAKE,
           ln=FAKE, B=1, Hq=4, H=2, T=3, d=64, rot=64, inter=0, m=1.0, pages=4, P=16, width=2, strides=None):
    st = (ctypes.c_longlong * 8)(*strides) if strides else None
    return A._lib.attn_rope_kv_append_fp8(q, qo, k, v, f, pos, kc, vc, ks, vs, bounds, t, cu, ln, B, Hq, H, T, d, rot, inter, m,
                                          pages, P, width, st, None)


def select(A, q=FAKE, kc=FAKE, ks=FAKE, t=FAKE, cu=FAKE, ln=FAKE, out=FAKE, B=1, Hq=4, H=2, T=3, mq=3, d=64, pages=4, P=16,
           width=2, count=4, first=1, last=1, causal=1, ws=FAKE, wsn=1 << 40):
    return A._lib.attn_select_pages_fp8(q, kc, ks, t, cu, ln, out, B, Hq, H, T, mq, d, pages, P, width, count, first, last,
                                        causal, ws, wsn, None)


def listed(A, q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, t=FAKE, cu=FAKE, ln=FAKE, lists=FAKE, o=FAKE, lse=FAKE, B=1, Hq=4,
           H=2, T=3, count=4, d=64, pages=4, P=16, width=2, causal=1, scale=0.125, ws=FAKE, wsn=1 << 40):
    return A._lib.attn_fwd_kv_fp8_pages(q, kc, vc, ks, vs, t, cu, ln, lists, o, lse, B, Hq, H, T, count, d, pages, P, width,
                                        causal, scale, ws, wsn, None)


def prefix(A, q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, pt=FAKE, pcu=FAKE, pln=FAKE, t=FAKE, cu=FAKE, ln=FAKE, o=FAKE, lse=FAKE,
           G=1, B=1, Hq=4, H=2, T=3, pq=3, mq=3, d=64, pages=4, P=16, pwidth=2, width=2, causal=1, scale=0.125, ws=FAKE,
           wsn=1 << 40):
    return A._lib.attn_fwd_kv_fp8_prefix(q, kc, vc, ks, vs, pt, pcu, pln, t, cu, ln, o, lse, G, B, Hq, H, T, pq, mq, d, pages, P,
                                         pwidth, width, causal, scale, ws, wsn, None)


@pytest.mark.parametrize("call", [append, select, listed, prefix])
def test_common_refusals(A, call):
    assert call(A, d=192) == -2 and call(A, d=96) == -2
    assert call(A, P=24) == -2 and call(A, P=256) == -2 and call(A, P=0) == -2
    for bad in (dict(B=-1), dict(T=-1), dict(B=0), dict(H=0), dict(pages=-1), dict(width=-1), dict(width=1 << 28),
                dict(T=0x7fffffff), dict(kc=None), dict(ks=None), dict(t=None), dict(cu=None), dict(ln=None),
                dict(q=None), dict(pages=1 << 30, H=4), dict(Hq=-1)):
        assert call(A, **bad) == -1, bad
        assert A.attn_last_error()
    assert call(A, kc=EIGHT) == -3 and call(A, t=ODD) == -3 and call(A, ks=ODD) == -3 and call(A, cu=ODD) == -3
    assert call(A, B=0, T=0, **({"G": 0} if call is prefix else {})) == 0 and call(A, T=0) == 0


def test_append_refusals(A):
    for bad in (dict(rot=66), dict(rot=-2), dict(rot=63), dict(m=float("inf")), dict(m=float("nan")), dict(f=None), dict(k=None),
                dict(v=None), dict(qo=None), dict(pages=0), dict(width=0), dict(rot=0),          # queries, but no rotation
                dict(strides=[64, 32, 64, 128, 64, 128, 64, 32]),                               # rows of q_out overlap
                dict(qo=FAKE, strides=[64, 256, 64, 128, 64, 128, 256, 64])):                    # in place, other strides
        assert append(A, **bad) == -1, bad
    assert append(A, k=EIGHT) == -3 and append(A, bounds=EIGHT) == -3 and append(A, f=ctypes.c_void_p(0x10004)) == -3
    assert append(A, pos=ODD) == -3 and append(A, q=ctypes.c_void_p(0x10001)) == -3
    assert append(A, strides=[64, 256, 64, 132, 64, 128, 64, 256]) == -3       # a token stride of k that is no multiple of 8


def test_select_refusals(A):
    for bad in (dict(count=0), dict(first=-1), dict(last=-1), dict(first=3, last=2), dict(first=1 << 30, last=1 << 30, count=4),
                dict(mq=0), dict(mq=4), dict(Hq=3), dict(out=None), dict(pages=0)):
        assert select(A, **bad) == -1, bad
    assert select(A, Hq=514) == -2 and select(A, Hq=65536) == -2
    assert select(A, q=EIGHT) == -3 and select(A, out=ODD) == -3
    assert select(A, ws=None) == -4 and select(A, wsn=64) == -4 and select(A, ws=EIGHT) == -3
    for bad in ((0, 1, 1), (1, -1, 1), (1, 1, -1)):
        with pytest.raises(A.AttnError):
            A.attn_select_pages_fp8_workspace_size(*bad)
    assert A.attn_select_pages_fp8_workspace_size(2, 0, 5) == 0


def test_listed_refusals(A):
    for bad in (dict(Hq=3), dict(scale=0.0), dict(scale=float("nan")), dict(count=-1), dict(lists=None), dict(o=None),
                dict(lse=None), dict(vc=None), dict(pages=0)):
        assert listed(A, **bad) == -1, bad
    assert listed(A, Hq=65536) == -2 and listed(A, Hq=514) == -2
    assert listed(A, q=EIGHT) == -3 and listed(A, o=EIGHT) == -3 and listed(A, lists=ODD) == -3
    assert listed(A, ws=None) == -4 and listed(A, wsn=64) == -4 and listed(A, ws=EIGHT) == -3
    for bad in ((0, 2, 3, 64), (3, 2, 3, 64), (4, 2, -1, 64), (4, 2, 3, 96)):
        with pytest.raises(A.AttnError):
            A.attn_fwd_kv_fp8_pages_workspace_size(*bad)
    assert A.attn_fwd_kv_fp8_pages_workspace_size(4, 2, 0, 64) == 0


def test_prefix_refusals(A):
    for bad in (dict(Hq=3), dict(scale=0.0), dict(G=0), dict(G=-1), dict(pq=0), dict(pq=4), dict(mq=0), dict(mq=4), dict(pt=None),
                dict(pcu=None), dict(pln=None), dict(o=None), dict(lse=None), dict(pages=0), dict(pwidth=-1),
                dict(pwidth=1 << 28)):
        assert prefix(A, **bad) == -1, bad
    assert prefix(A, Hq=65536) == -2 and prefix(A, Hq=514) == -2
    assert prefix(A, pt=ODD) == -3 and prefix(A, pcu=ODD) == -3 and prefix(A, pln=ODD) == -3 and prefix(A, o=EIGHT) == -3
    assert prefix(A, ws=None) == -4 and prefix(A, wsn=64) == -4 and prefix(A, ws=EIGHT) == -3
    for bad in ((0, 2, 3, 1, 1, 64), (3, 2, 3, 1, 1, 64), (4, 2, -1, 1, 1, 64), (4, 2, 3, -1, 1, 64), (4, 2, 3, 1, -1, 64), (4, 2, 3, 1, 1, 96)):
        with pytest.raises(A.AttnError):
            A.attn_fwd_kv_fp8_prefix_workspace_size(*bad)
    assert A.attn_fwd_kv_fp8_prefix_workspace_size(4, 2, 0, 1, 1, 64) == 0


@pytest.mark.parametrize("heads", [(8, 2), (32, 1), (5, 5)])
def test_prefix_workspace_does_not_fall_as_the_bounds_grow(A, heads):
    size = lambda pq, mq, T=70: A.attn_fwd_kv_fp8_prefix_workspace_size(*heads, T, pq, mq, 64)
    for mq in (1, 3, 40):
        sizes = [size(pq, mq) for pq in range(1, 60)]
        assert sizes == sorted(sizes)
    assert size(3, 1, 70) <= size(3, 1, 71)


def test_binding_refuses_cpu_tensors(A):
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k"):
        A.attn_rope_kv_append_fp8(x, x, x, None, None, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="q"):
        A.attn_select_pages_fp8(x, None, None, None, None, None, 16, 4, 1)
    with pytest.raises(ValueError, match="q"):
        A.attn_fwd_kv_fp8_pages(x, None, None, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="q"):
        A.attn_fwd_kv_fp8_prefix(x, None, None, None, None, None, None, None, 1, None, None, None, 1)
