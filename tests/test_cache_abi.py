"""Refusals of the rotary, cache append and cached attention entry points: the documented
status before anything touches the GPU, and the binding's own checks."""
import ctypes

import pytest
import torch

FAKE, ODD, HALF = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10002), ctypes.c_void_p(0x10001)


@pytest.fixture(scope="module")
def A():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import attention_attn_fwd_09_gb300 as A
    return A


def rope(A, q=FAKE, k=FAKE, qo=ctypes.c_void_p(0x20000), ko=ctypes.c_void_p(0x30000), f=FAKE, pos=None, B=1, Hq=2, Hk=1,
         N=4, d=64, rot=64, inter=0, m=1.0, strides=None, fn="attn_rope"):
    st = (ctypes.c_longlong * 12)(*strides) if strides else None
    return getattr(A._lib, fn)(q, k, qo, ko, f, pos, B, Hq, Hk, N, d, rot, inter, m, st, None)


@pytest.mark.parametrize("fn", ["attn_rope", "attn_rope_bwd"])
def test_rope_refusals(A, fn):
    assert rope(A, fn=fn, d=96) == -2
    for bad in (dict(rot=0), dict(rot=3), dict(rot=66), dict(m=float("inf")), dict(m=float("nan")), dict(Hq=0), dict(Hk=-1),
                dict(B=-1), dict(N=-1), dict(q=None), dict(k=None), dict(f=None), dict(Hq=40000, Hk=40000),
                dict(strides=[0, 64, 64, 0, 64, 64, 0, 64, 32, 0, 64, 64]),      # output rows overlap
                dict(strides=[0, 64, 64, 0, 64, 64, 0, 0, 64, 0, 64, 64]),
                dict(qo=FAKE, strides=[0, 64, 128, 0, 64, 64, 0, 256, 64, 0, 64, 64])):   # in place, other strides
        assert rope(A, fn=fn, **bad) == -1, bad
        assert A.attn_last_error()
    assert rope(A, fn=fn, N=0x7fffffff, Hq=1, Hk=0) == -1
    assert rope(A, fn=fn, q=HALF) == -3
    assert rope(A, fn=fn, f=ctypes.c_void_p(0x10004)) == -3
    assert rope(A, fn=fn, pos=ODD) == -3
    assert rope(A, fn=fn, B=0) == 0 and rope(A, fn=fn, N=0) == 0


def append(A, k=FAKE, v=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, t=FAKE, cu=FAKE, ln=FAKE, B=1, H=2, T=3, d=64, pages=4,
           P=16, width=2, strides=None):
    st = (ctypes.c_longlong * 4)(*strides) if strides else None
    return A._lib.attn_kv_append_fp8(k, v, kc, vc, ks, vs, t, cu, ln, B, H, T, d, pages, P, width, st, None)


def attend(A, q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, t=FAKE, cu=FAKE, ln=FAKE, o=FAKE, lse=FAKE, B=1, Hq=4, H=2, T=3,
           mq=3, d=64, pages=4, P=16, width=2, causal=1, scale=0.125, ws=FAKE, wsn=1 << 40):
    return A._lib.attn_fwd_kv_fp8(q, kc, vc, ks, vs, t, cu, ln, o, lse, B, Hq, H, T, mq, d, pages, P, width, causal, scale,
                                  ws, wsn, None)


@pytest.mark.parametrize("call", [append, attend])
def test_cache_refusals(A, call):
    assert call(A, d=192) == -2 and call(A, d=96) == -2
    assert call(A, P=24) == -2 and call(A, P=256) == -2 and call(A, P=0) == -2
    for bad in (dict(B=-1), dict(T=-1), dict(B=0), dict(H=0), dict(pages=-1), dict(width=-1), dict(width=1 << 28),
                dict(T=0x7fffffff), dict(kc=None), dict(ks=None), dict(t=None), dict(cu=None), dict(ln=None),
                dict(pages=1 << 30, H=4)):
        assert call(A, **bad) == -1, bad
    assert call(A, kc=ctypes.c_void_p(0x10008)) == -3
    assert call(A, t=ODD) == -3 and call(A, ks=ODD) == -3
    assert call(A, B=0, T=0) == 0 and call(A, T=0) == 0


def test_append_refusals(A):
    assert append(A, k=ctypes.c_void_p(0x10008)) == -3
    assert append(A, strides=[64, 132, 64, 128]) == -3          # a token stride that is no multiple of 8
    assert append(A, k=None) == -1 and append(A, pages=0) == -1 and append(A, width=0) == -1


def test_attend_refusals(A):
    for bad in (dict(Hq=3), dict(scale=0.0), dict(scale=float("nan")), dict(mq=0), dict(mq=4), dict(q=None), dict(o=None),
                dict(lse=None)):
        assert attend(A, **bad) == -1, bad
    assert attend(A, q=ctypes.c_void_p(0x10008)) == -3 and attend(A, o=ctypes.c_void_p(0x10008)) == -3
    assert attend(A, Hq=65536, H=2) == -2
    assert attend(A, Hq=514, H=2) == -2                         # more than 256 query heads per K/V head
    assert attend(A, ws=None) == -4 and attend(A, wsn=64) == -4 and attend(A, ws=ctypes.c_void_p(0x10008)) == -3


def test_workspace_size_refusals(A):
    for bad in ((-1, 4, 2, 3, 1, 64), (1, 3, 2, 3, 1, 64), (1, 4, 2, -1, 1, 64), (1, 4, 2, 3, -1, 64), (1, 4, 2, 3, 1, 96)):
        with pytest.raises(A.AttnError):
            A.attn_fwd_kv_fp8_workspace_size(*bad)
    assert A.attn_fwd_kv_fp8_workspace_size(0, 4, 2, 0, 0, 64) == 0


def test_binding_refuses_cpu_tensors(A):
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    f, m = A.attn_rope_freqs(64, device="cpu")
    with pytest.raises(ValueError, match="q"):
        A.attn_rope(x, None, f)
    with pytest.raises(ValueError, match="k"):
        A.attn_kv_append_fp8(x[0], x[0], None, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="q"):
        A.attn_fwd_kv_fp8(x[0], None, None, None, None, None, None, None, 1)


def test_rope_freqs(A):
    f, m = A.attn_rope_freqs(64, base=500.0, device="cpu")
    assert f.dtype is torch.float64 and m == 1.0 and torch.allclose(f, 500.0 ** (-torch.arange(0, 64, 2).double() / 64))
    g, m = A.attn_rope_freqs(64, base=500.0, scaling="linear", factor=4.0, device="cpu")
    assert m == 1.0 and torch.allclose(g, f / 4)
    g, m = A.attn_rope_freqs(64, base=500.0, scaling="ntk", factor=4.0, device="cpu")
    assert m == 1.0 and g[0] == 1.0 and abs(g[-1] / (f[-1] / 4) - 1) < 1e-12      # the slowest pair: compressed exactly
    g, m = A.attn_rope_freqs(64, base=500.0, scaling="yarn", factor=4.0, trained_length=1024, device="cpu")
    turns = 1024 * f / 6.283185307179586
    assert abs(m - (0.1 * 1.3862943611198906 + 1)) < 1e-15
    assert torch.equal(g[turns >= 32], f[turns >= 32]) and torch.allclose(g[turns <= 1], f[turns <= 1] / 4)
    assert (g <= f).all() and (g >= f / 4).all()
    for bad in (dict(rot=63), dict(rot=0), dict(base=1.0), dict(factor=0.5), dict(scaling="yarn"), dict(scaling="other"),
                dict(rot=2, scaling="ntk")):
        with pytest.raises(ValueError):
            A.attn_rope_freqs(**{"rot": 64, "device": "cpu", **bad})
