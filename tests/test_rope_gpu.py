"""attn_rope and attn_rope_bwd against the fp64 oracle.

Bound per element: the cosine and sine come from an angle exact to 2^-32 turns (2^-29.3
radians) and an fp32 evaluation (2 ulp: 2^-23 at most in value), times m; products and sum
round three times in fp32; the result rounds to bf16 by 2^-8 of itself.  So
2^-8 |y| + (|a| + |b|) |m| 2^-20."""
import numpy as np
import pytest
import torch

import oracle.rope as orope
from cache_cases import bf16

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def A():
    import attention_attn_fwd_09_gb300 as A
    A.attn_device_status(True)
    yield A
    assert A.attn_device_status(True) == 0


def partner_sum(x, rot, inter):
    x = np.abs(x)
    s = x.copy()
    if inter:
        t = x[..., 0:rot:2] + x[..., 1:rot:2]
        s[..., 0:rot:2], s[..., 1:rot:2] = t, t
    else:
        t = x[..., :rot // 2] + x[..., rot // 2:rot]
        s[..., :rot // 2], s[..., rot // 2:rot] = t, t
    return s


def check(y, x, f, pos, inter, m, backward):
    x = x.float().cpu().numpy().astype(np.float64)
    rot = 2 * f.numel()
    want = orope.rotate(x, f.cpu().numpy(), pos, inter, m, backward)
    got = y.float().cpu().numpy().astype(np.float64)
    tol = 2.0 ** -8 * np.abs(want) + partner_sum(x, rot, inter) * abs(m) * 2.0 ** -20 + 1e-38
    assert (np.abs(got - want) <= tol).all(), np.max(np.abs(got - want) / tol)
    assert (got[..., rot:] == x[..., rot:]).all()


def rows(rng, *shape):
    return bf16(rng.randn(*shape)).to(DEV)


@pytest.mark.parametrize("d,rot", [(64, 64), (64, 24), (128, 128), (128, 64), (128, 40), (128, 2), (128, 90), (192, 192), (256, 256),
                                   (256, 72), (192, 96)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("backward", [False, True])
def test_widths(A, d, rot, inter, backward):
    rng = np.random.RandomState(d + rot)
    B, N, Hq, Hk = 2, 13, 3, 1
    q, k = rows(rng, B, Hq, N, d), rows(rng, B, Hk, N, d)
    f, m = A.attn_rope_freqs(rot, scaling="yarn", factor=3.0, trained_length=512)
    pos = torch.as_tensor(rng.randint(0, 5000, (B, N)).astype(np.int32), device=DEV)
    call = A.attn_rope_bwd if backward else A.attn_rope
    qo, ko = call(q, k, f, pos, interleaved=inter, mscale=m)
    check(qo, q, f, pos.cpu().numpy(), inter, m, backward)
    check(ko, k, f, pos.cpu().numpy(), inter, m, backward)


@pytest.mark.parametrize("N", [1, 7, 8, 9, 300, 1500])
@pytest.mark.parametrize("H", [(1, 0), (5, 1), (8, 8), (32, 8)])
def test_lengths_and_heads(A, N, H):
    rng = np.random.RandomState(N)
    d, f = 128, A.attn_rope_freqs(128)[0]
    q, k = rows(rng, 1, H[0], N, d), (rows(rng, 1, H[1], N, d) if H[1] else None)
    qo, ko = A.attn_rope(q, k, f)
    pos = np.arange(N)[None]
    check(qo, q, f, pos, False, 1.0, False)
    if H[1]:
        check(ko, k, f, pos, False, 1.0, False)
    else:
        assert ko is None


def test_far_positions(A):
    """Positions up to 2^31 - 1, where an fp32 angle has no correct digit, and negative ones."""
    rng = np.random.RandomState(3)
    d = 64
    p = np.array([[0, 1, 2 ** 20 + 1, 2 ** 24 + 1, 123456789, 2 ** 31 - 1, -1, -77777, -2 ** 31]], np.int32)
    q = rows(rng, 1, 2, p.shape[1], d)
    f, m = A.attn_rope_freqs(d, scaling="linear", factor=1.5)
    qo, _ = A.attn_rope(q, None, f, torch.as_tensor(p, device=DEV))
    # The phase of a position p carries p 2^-53 relative error of f in fp64: 2^31 * 2^-52 radians, below the bound.
    check(qo, q, f, p, False, 1.0, False)


def test_projection_views_in_and_out(A):
    """Q, K as views of a fused projection; gradients written back into such a layout."""
    rng = np.random.RandomState(5)
    B, N, Hq, Hk, d = 2, 37, 4, 2, 128
    proj = rows(rng, B, N, Hq + 2 * Hk, d)
    before = proj.clone()
    q, k = proj[:, :, :Hq].transpose(1, 2), proj[:, :, Hq:Hq + Hk].transpose(1, 2)
    f, m = A.attn_rope_freqs(64)
    qo, ko = A.attn_rope(q, k, f)
    assert qo.is_contiguous() and ko.is_contiguous() and torch.equal(proj, before)
    pos = np.tile(np.arange(N), (B, 1))
    check(qo, q, f, pos, False, 1.0, False)
    check(ko, k, f, pos, False, 1.0, False)
    grad = torch.full_like(proj, 7.0)
    gq, gk = grad[:, :, :Hq].transpose(1, 2), grad[:, :, Hq:Hq + Hk].transpose(1, 2)
    A.attn_rope_bwd(qo, ko, f, q_out=gq, k_out=gk)
    check(gq, qo, f, pos, False, 1.0, True)
    check(gk, ko, f, pos, False, 1.0, True)
    assert (grad[:, :, Hq + Hk:] == 7.0).all()


@pytest.mark.parametrize("shift,rot", [(8, 32), (4, 32), (2, 32), (1, 32), (8, 8), (0, 6)])
@pytest.mark.parametrize("inter", [False, True])
def test_alignments(A, shift, rot, inter):
    """Rows that start on 16, 8, 4 and 2 bytes."""
    rng = np.random.RandomState(shift)
    H, T, d = 3, 11, 64
    buf = rows(rng, T, H * d + shift)
    x = buf[:, shift:shift + H * d].unflatten(1, (H, d)).transpose(0, 1)
    f = A.attn_rope_freqs(rot)[0]
    pos = torch.arange(T, dtype=torch.int32, device=DEV) * 3
    y, _ = A.attn_rope(x, None, f, pos, interleaved=inter)
    check(y[None], x[None], f, pos.cpu().numpy()[None], inter, 1.0, False)


@pytest.mark.parametrize("inter,rot", [(False, 128), (True, 128), (False, 40), (True, 6)])
def test_in_place(A, inter, rot):
    rng = np.random.RandomState(9)
    qkv = rows(rng, 29, 6, 128)
    x = qkv.clone()
    q, k = qkv[:, :3].transpose(0, 1), qkv[:, 3:5].transpose(0, 1)
    f = A.attn_rope_freqs(rot)[0]
    A.attn_rope(q, k, f, interleaved=inter, q_out=q, k_out=k)
    pos = np.arange(29)[None]
    check(q[None], x[:, :3].transpose(0, 1)[None], f, pos, inter, 1.0, False)
    check(k[None], x[:, 3:5].transpose(0, 1)[None], f, pos, inter, 1.0, False)
    assert torch.equal(qkv[:, 5], x[:, 5])


def test_backward_is_the_gradient(A):
    """<dy, R x> = <R^T dy, x>, and central differences of a scalar of the rotated rows."""
    rng = np.random.RandomState(11)
    d, N = 64, 5
    x, dy = rows(rng, 1, 1, N, d), rows(rng, 1, 1, N, d)
    f, m = A.attn_rope_freqs(48, scaling="yarn", factor=2.0, trained_length=64)
    y, _ = A.attn_rope(x, None, f, interleaved=True, mscale=m)
    dx, _ = A.attn_rope_bwd(dy, None, f, interleaved=True, mscale=m)
    a, b = float((dy.double() * y.double()).sum()), float((dx.double() * x.double()).sum())
    # each side: bf16 roundings of N d products
    size = float((dy.double() * y.double()).abs().sum() + (dx.double() * x.double()).abs().sum())
    assert abs(a - b) <= 2.0 ** -8 * size
    pos = np.arange(N)[None]
    xd, dyd = x.double().cpu().numpy(), dy.double().cpu().numpy()
    fn = lambda z: float((orope.rotate(z, f.cpu().numpy(), pos, True, m) * dyd).sum())
    for n, c in ((0, 0), (1, 1), (2, 30), (4, 47), (3, 60)):
        e = np.zeros_like(xd)
        e[0, 0, n, c] = 1e-3
        slope = (fn(xd + e) - fn(xd - e)) / 2e-3
        assert abs(float(dx[0, 0, n, c]) - slope) <= 2.0 ** -8 * abs(slope) + 2.0 ** -18 * 8


def test_nonfinite_stay_in_their_pair(A):
    x = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16, device=DEV)
    x[0, 0, 0, 3], x[0, 0, 1, 60] = float("inf"), float("nan")
    y, _ = A.attn_rope(x, None, A.attn_rope_freqs(64)[0])
    bad = ~torch.isfinite(y[0, 0])
    assert bad[0].nonzero().flatten().tolist() == [3, 35] and bad[1].nonzero().flatten().tolist() == [28, 60]


def test_empty_and_single(A):
    f = A.attn_rope_freqs(64)[0]
    for shape in ((0, 2, 5, 64), (1, 2, 0, 64)):
        q, k = A.attn_rope(torch.empty(shape, dtype=torch.bfloat16, device=DEV), None, f)
        assert q.shape == shape
    x = rows(np.random.RandomState(0), 2, 1, 64)
    y, _ = A.attn_rope(x, None, f, torch.tensor([5], dtype=torch.int32, device=DEV))
    check(y[None], x[None], f, [[5]], False, 1.0, False)


def test_binding_refusals(A):
    f = A.attn_rope_freqs(64)[0]
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    for args in ((x.half(), None, f), (x, x[:, :3], f), (x, None, f.float()), (x, None, f, torch.zeros(3, dtype=torch.int32, device=DEV)),
                 (x, None, f, torch.zeros(4, dtype=torch.int64, device=DEV)), (x, None, f.cpu()), (x.transpose(1, 2), None, f),
                 (x, None, f.view(2, 16)), (x[0], None, f)):
        with pytest.raises(ValueError):
            A.attn_rope(*args)
    with pytest.raises(A.AttnError):
        A.attn_rope(x, None, A.attn_rope_freqs(66)[0])


def test_streams_and_graph(A):
    """On another stream than the current one, and captured and replayed on new inputs."""
    rng = np.random.RandomState(2)
    f = A.attn_rope_freqs(128)[0]
    q, k = rows(rng, 4, 65, 128), rows(rng, 2, 65, 128)
    want = A.attn_rope(q, k, f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, side.cuda_stream):
        got = A.attn_rope(q, k, f, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out = [torch.empty_like(t) for t in (q, k)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        A.attn_rope(q, k, f, q_out=out[0], k_out=out[1])
    q.copy_(rows(rng, 4, 65, 128))
    g.replay()
    torch.cuda.synchronize()
    check(out[0][None], q[None], f, np.arange(65)[None], False, 1.0, False)


def test_rows_past_32_bits(A):
    """A token stride that takes the last rows' offsets past 2^32 bytes and 2^31 elements."""
    n, step = 5, 1 << 29                                  # 5 rows, 1 GiB apart: 5 GiB
    free, _ = torch.cuda.mem_get_info()
    if free < 16 << 30:
        pytest.skip("needs 16 GB free")
    buf = torch.zeros(n * step + 256, dtype=torch.bfloat16, device=DEV)
    x = buf.as_strided((1, n, 64), (64, step, 1))
    x.copy_(rows(np.random.RandomState(1), 1, n, 64))
    f = A.attn_rope_freqs(64)[0]
    y, _ = A.attn_rope(x, None, f)
    check(y[None], x[None], f, np.arange(n)[None], False, 1.0, False)
    z, _ = A.attn_rope(y, None, f, q_out=buf.as_strided((1, n, 64), (64, step, 1), 128))
    check(z[None], y[None], f, np.arange(n)[None], False, 1.0, False)


def test_an_output_for_no_k_is_refused(A):
    q = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16, device="cuda")
    f, _ = A.attn_rope_freqs(64)
    with pytest.raises(ValueError, match="k_out"):
        A.attn_rope(q, None, f, k_out=torch.empty_like(q))
    q_out, none = A.attn_rope(q, None, f)
    assert none is None and torch.equal(q_out, q)
