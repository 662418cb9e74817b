"""attn_rope_kv_append_fp8: V and the rows kept exactly as the fp64 oracle has them, rotated K codes
within what the fp32 rotation may move a value, bounds exactly those of the codes, queries as
attn_rope returns them."""
import numpy as np
import pytest
import torch

import oracle.cache as oc
import oracle.sparse as osp
from cache_cases import bf16, empty_cache, offsets, page_tables
from oracle.fp8 import e4m3_decode

pytestmark = pytest.mark.gpu
DEV = "cuda"
INVALID = -1
# y = m (a cos - b sin): the angle is off by 9.4e-8, sine and cosine by 2 ulp (2^-22) and by m's rounding
# (2^-24), the products and their sum by 2^-23 of |a| + |b| together: 9.4e-8 + 2^-22 + 2^-24 + 2^-23 < 5.2e-7.
EPS = 5.2e-7


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


def slack(x, rot, interleaved, m):
    """How far each rotated value may be off: EPS m (|a| + |b|) of its pair."""
    s, r = np.zeros_like(x), np.abs(x[..., :rot])
    if interleaved:
        s[..., 0:rot:2] = s[..., 1:rot:2] = r[..., 0::2] + r[..., 1::2]
    else:
        s[..., :rot // 2] = s[..., rot // 2:rot] = r[..., :rot // 2] + r[..., rot // 2:]
    return s * EPS * abs(m)


def turned(x, f, where, interleaved, m):
    """The rotation in 64 bits, in real numbers (a product of complex ones would make NaN of infinities)."""
    y, t, half = x.copy(), where[:, None].astype(np.float64) * f, len(f)
    a, b = (np.s_[..., 0:2 * half:2], np.s_[..., 1:2 * half:2]) if interleaved else (np.s_[..., :half], np.s_[..., half:2 * half])
    y[a] = m * (x[a] * np.cos(t) - x[b] * np.sin(t))
    y[b] = m * (x[b] * np.cos(t) + x[a] * np.sin(t))
    return y


class Cache:
    def __init__(self, A, pages, table, H, P, d, bounds=True, seed=0):
        self.A, self.table, self.H, self.P, self.d, self.pages = A, table, H, P, d, pages
        self.host = {n: empty_cache(pages, H, P, d, seed + i) for i, n in enumerate("kv")}
        self.gpu = {n: (dev(c.copy()), dev(s.copy())) for n, (c, s) in self.host.items()}
        self.bounds = dev(np.random.RandomState(seed).randint(0, 256, (pages, H, 2, d)).astype(np.uint8)) if bounds else None
        self.used = np.zeros(pages, int)                   # rows of each page that a call wrote

    def append(self, q, k, v, ns, lens, freqs, m=1.0, inter=False, positions=None, views=None, q_out=None, **kw):
        """The call, and everything it may change checked."""
        P, d, cu = self.P, self.d, offsets(ns)
        rot = 0 if freqs is None else 2 * len(freqs)
        before = {n: tuple(t.cpu().numpy().copy() for t in self.gpu[n]) for n in "kv"}
        bounds_before = None if self.bounds is None else self.bounds.cpu().numpy().copy()
        gq, gk, gv = views if views else (None if q is None else q.to(DEV), k.to(DEV), v.to(DEV))
        at = np.concatenate([np.arange(n - x, n) for x, n in zip(ns, lens)]).astype(np.int32) if sum(ns) else np.zeros(0, np.int32)
        where = at if positions is None else positions
        out = self.A.attn_rope_kv_append_fp8(
            gq, gk, gv, None if freqs is None else dev(freqs), self.gpu["k"][0], self.gpu["v"][0], self.gpu["k"][1],
            self.gpu["v"][1], dev(self.table), dev(cu), dev(np.asarray(lens, np.int32)),
            positions=None if positions is None else dev(positions), interleaved=inter, mscale=m, k_bounds=self.bounds,
            q_out=q_out, **kw)
        torch.cuda.synchronize()
        if q is not None:
            want, _ = self.A.attn_rope(q.to(DEV).contiguous(), None, dev(freqs), dev(where), interleaved=inter, mscale=m)
            assert torch.equal(out.contiguous().view(torch.int16), want.view(torch.int16))
        # V: the oracle's append, byte for byte
        codes, scale = before["v"]
        oc.append(v.float().numpy(), codes, scale, self.table, cu, lens)
        for got, want in zip(self.gpu["v"], (codes, scale)):
            got = got.cpu().numpy()
            assert (got == want).all(), np.argwhere(got != want)[:5]
        # K: rotated in 64 bits
        x = k.float().numpy().astype(np.float64)
        with np.errstate(invalid="ignore"):
            y = x if rot == 0 else turned(x, freqs, where, inter, m)
            off = np.zeros_like(x) if rot == 0 else slack(x, rot, inter, m)
        off = np.where(np.isfinite(off), off, 0.0)
        got_c, got_s = (t.cpu().numpy() for t in self.gpu["k"])
        codes, scale = before["k"]
        touched = set()
        for b in range(len(lens)):
            n, start = ns[b], lens[b] - ns[b]
            pos = start
            while pos < lens[b]:
                blk, slot = divmod(pos, P)
                end = min(lens[b], (blk + 1) * P)
                page = int(self.table[b][blk])
                touched.add(page)
                self.used[page] = slot + end - pos
                sl = np.s_[:, cu[b] + pos - start:cu[b] + end - start]
                for h in range(self.H):
                    yy, oo = y[sl][h], off[sl][h]
                    mag = np.where(np.isfinite(yy), np.abs(yy), 0.0)
                    lo_s, hi_s = oc.pow2_scale(float(np.max(mag - oo, initial=0.0))), oc.pow2_scale(float(np.max(mag + oo, initial=0.0)))
                    s_old = float(scale[page, h]) if slot else 0.0
                    s = float(got_s[page, h])
                    assert s in (max(lo_s, s_old), max(hi_s, s_old)), (page, h, s, lo_s, hi_s, s_old)
                    if slot and s > s_old:
                        old = (e4m3_decode(codes[page, h, :slot]).astype(np.float32) * np.float32(s_old)).astype(np.float64)
                        codes[page, h, :slot] = oc.encode(old, s)
                    assert (got_c[page, h, :slot] == codes[page, h, :slot]).all()
                    new = got_c[page, h, slot:slot + end - pos]
                    with np.errstate(invalid="ignore"):
                        low, high, mid = (e4m3_decode(oc.encode(z, s)) for z in (yy - oo, yy + oo, yy))
                        value = e4m3_decode(new)
                    nan = np.isnan(mid)
                    assert (np.isnan(value) == nan).all()
                    ok = nan | ((value >= low) & (value <= high))
                    assert ok.all(), (page, h, np.argwhere(~ok)[:4])
                    codes[page, h, slot:slot + end - pos] = new
                    scale[page, h] = s
                pos = end
        assert (got_c == codes).all() and (got_s == scale).all()        # nothing else has changed
        if self.bounds is not None:
            got_b = self.bounds.cpu().numpy()
            pages = sorted(touched)
            want = osp.page_bounds(codes[pages], self.used[pages])
            value = e4m3_decode(got_b[pages])
            assert ((value == want) | (np.isnan(value) & np.isnan(want))).all()
            rest = np.setdiff1d(np.arange(self.pages), pages)
            assert (got_b[rest] == bounds_before[rest]).all()
        return out


def rows(rng, Hq, H, T, d, gain=1.0):
    return bf16(rng.randn(Hq, T, d)), bf16(rng.randn(H, T, d) * gain), bf16(rng.randn(H, T, d) * gain * 3)


def freqs(A, rot, base=10000.0):
    return A.attn_rope_freqs(rot, base, device="cpu")[0].numpy()


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rot,inter", [("d", False), ("d", True), ("d/2", False), ("d/4+8", False), ("d/4+8", True),
                                       ("6", False), ("2", True), ("0", False)])
def test_prompts_then_tokens(A, P, d, rot, inter):
    """Prompts of odd lengths, single tokens of growing size (scales grow, codes and bounds are rounded
    again), then pieces that cross pages."""
    rot = int(eval(rot.replace("/", "//"), {"d": d}))
    rng = np.random.RandomState(P + d + rot)
    f = freqs(A, rot) if rot else None
    H, Hq, ns = 2, 3 if rot else 0, [1, P, 2 * P + 3, 17, 0]
    extra = [2, P + 5, 9, 1, 3]
    final = [n + 3 + e for n, e in zip(ns, extra)]
    table, pages = page_tables(final, P, P)
    c = Cache(A, pages, table, H, P, d)

    def step(ns, lens, gain=1.0, **kw):
        q, k, v = rows(rng, Hq or 1, H, sum(ns), d, gain)
        c.append(q if rot else None, k, v, ns, lens, f, inter=inter, **kw)

    lens = list(ns)
    step(ns, lens)
    for i in range(3):
        lens = [n + 1 for n in lens]
        step([1] * 5, lens, 2.0 ** (2 * i - 2), m=1.25)
    lens = [n + e for n, e in zip(lens, extra)]
    step(extra, lens)


@pytest.mark.parametrize("P,H,d,ns", [
    (16, 8, 64, [2600, 17, 1]), (32, 9, 128, [3000, 1500, 0, 33]), (16, 33, 128, [520, 100]),     # many small pages
    (128, 9, 128, [1] * 40 + [97]), (64, 3, 64, [1, 0, 1] * 20 + [70]),                          # a piece among single rows
    (128, 2, 128, [1500, 1]), (64, 4, 128, [700, 300]), (128, 1, 64, [513]),                     # a block per page
])
@pytest.mark.parametrize("inter", [False, True])
def test_regimes(A, P, H, d, ns, inter):
    rng = np.random.RandomState(P + H)
    had = rng.randint(0, 2 * P, len(ns))
    lens = [int(h) + n for h, n in zip(had, ns)]
    table, pages = page_tables(lens, P, 3)
    c = Cache(A, pages, table, H, P, d)
    f = freqs(A, d, 500000.0)
    q, k, v = rows(rng, 2, H, int(had.sum()), d, 0.25)
    c.append(q, k, v, had.tolist(), had.tolist(), f, inter=inter)
    q, k, v = rows(rng, 2, H, sum(ns), d)
    k[0, :, 5] = float("inf")
    k[0, ::3, 6] = float("nan")
    v[H - 1, ::3, d - 1] = float("nan")
    far = (rng.randint(0, 500000) + np.arange(sum(ns))).astype(np.int32)
    c.append(q, k, v, ns, lens, f, inter=inter, positions=far)


def test_without_bounds_and_in_place_views_of_a_projection(A):
    rng = np.random.RandomState(1)
    H, Hq, P, d, ns = 3, 4, 32, 128, [33, 5]
    table, pages = page_tables(ns, P)
    c = Cache(A, pages, table, H, P, d, bounds=False)
    proj = bf16(rng.randn(38, Hq + 2 * H, d))
    on = proj.to(DEV)
    split = lambda t: (t[:, :Hq].transpose(0, 1), t[:, Hq:Hq + H].transpose(0, 1), t[:, Hq + H:].transpose(0, 1))
    q, k, v = split(proj)
    out = c.append(q, k, v, ns, ns, freqs(A, d), views=split(on), q_out=split(on)[0])
    assert out.data_ptr() == on.data_ptr()
    assert torch.equal(on[:, Hq:], proj[:, Hq:].to(DEV))


@pytest.mark.parametrize("P", [16, 128])
def test_zero_extreme_and_nonfinite_rows(A, P):
    H, d = 1, 64
    table, pages = page_tables([20], P)
    c = Cache(A, pages, table, H, P, d)
    x = np.zeros((1, 20, d), np.float32)
    x[0, 1, :5] = [np.inf, -np.inf, np.nan, 7.0, -0.0]
    x[0, 2] = 1e-38
    x[0, 3, 0] = 3e38
    x[0, 5, 1] = 1e-40
    x[0, 6:] = np.random.RandomState(0).randn(14, d)
    x = bf16(x)
    f = freqs(A, 32)
    for i in range(4):                                     # one by one: 0, then non-finite, tiny, huge
        c.append(None, x[:, i:i + 1], x[:, 8 - i:9 - i], [1], [i + 1], f)
    c.append(None, x[:, 4:9], x[:, :5], [5], [9], f)
    c.append(None, x[:, 9:], x[:, 9:], [11], [20], f)


@pytest.mark.parametrize("rot,inter,lead", [(128, False, 0), (40, False, 0), (40, True, 0), (128, True, 0), (36, False, 0), (128, False, 1)])
@pytest.mark.parametrize("B", [5, 300])
def test_queries_of_a_few_rows(A, rot, inter, lead, B):
    """Few rows' queries: the same bits as attn_rope's whether or not they go in the same launch (rows off 16
    bytes, and a rotated part that is no multiple of 8 columns, do not), some sequences without rows."""
    rng = np.random.RandomState(B + rot)
    H, Hq, P, d = 1, 37, 16, 128
    ns = [0, 1, 1, 3, 1] if B == 5 else rng.randint(0, 3, B).tolist()
    lens = [n + int(x) for n, x in zip(ns, rng.randint(0, 30, B))]
    table, pages = page_tables(lens, P)
    c = Cache(A, pages, table, H, P, d)
    T = sum(ns)
    q, k, v = rows(rng, Hq, H, T, d)
    flat = torch.empty(Hq * T * d + 8, dtype=torch.bfloat16, device=DEV)
    view = flat[lead:lead + Hq * T * d].view(Hq, T, d)
    view.copy_(q)
    c.used[:] = 0
    for b, n in enumerate(lens):                           # the rows before: whatever is there
        for blk in range(-(-n // P)):
            c.used[table[b, blk]] = 0
    c.bounds = None
    c.append(q, k, v, ns, lens, freqs(A, rot), inter=inter, m=0.75, views=(view, k.to(DEV), v.to(DEV)))


def test_many_sequences(A):
    """More sequences than a block has threads, some without new rows."""
    rng = np.random.RandomState(8)
    B, H, P, d = 700, 1, 16, 64
    ns = rng.randint(0, 4, B).tolist()
    before = rng.randint(0, 20, B).tolist()
    lens = [a + b for a, b in zip(ns, before)]
    table, pages = page_tables(lens, P)
    c = Cache(A, pages, table, H, P, d)
    f = freqs(A, d)
    for n, at in ((before, before), (ns, lens)):
        q, k, v = rows(rng, 1, H, sum(n), d)
        c.append(q, k, v, n, at, f)


def test_equals_the_two_calls_where_rounding_cannot_differ(A):
    """Keys that the rotation leaves exact (angles of 0): the same bytes as attn_kv_append_fp8."""
    rng = np.random.RandomState(4)
    H, P, d, ns = 2, 32, 64, [40, 3]
    table, pages = page_tables(ns, P)
    c = Cache(A, pages, table, H, P, d)
    q, k, v = rows(rng, 2, H, 43, d)
    c.append(q, k, v, ns, ns, freqs(A, d), positions=np.zeros(43, np.int32))
    kc, vc, ks, vs = (torch.zeros_like(t) for t in (*(c.gpu[n][0] for n in "kv"), *(c.gpu[n][1] for n in "kv")))
    A.attn_kv_append_fp8(k.to(DEV), v.to(DEV), kc, vc, ks, vs, dev(table), dev(offsets(ns)), dev(np.asarray(ns, np.int32)))
    for b, n in enumerate(ns):
        for t in range(n):
            page = table[b, t // P]
            assert torch.equal(kc[page, :, t % P], c.gpu["k"][0][page, :, t % P]) and torch.equal(ks[page], c.gpu["k"][1][page])


def test_bad_offsets_and_pages(A):
    rng = np.random.RandomState(2)
    H, P, d, lens = 2, 16, 64, [20, 7]
    table, pages = page_tables(lens, P)
    q, k, v = (t.to(DEV) for t in rows(rng, 2, H, 27, d))
    f, good = dev(freqs(A, d)), offsets(lens)
    for cu, ln in (([1, 20, 27], lens), ([0, 28, 27], lens), ([0, 20, 26], lens), (good, [19, 7]), (good, [20, 3 * P + 1]),
                   (good, [-1, 7])):
        c = Cache(A, pages, table, H, P, d)
        was = [t.clone() for t in (*c.gpu["k"], *c.gpu["v"], c.bounds)]
        A.attn_rope_kv_append_fp8(q, k, v, f, c.gpu["k"][0], c.gpu["v"][0], c.gpu["k"][1], c.gpu["v"][1], dev(table),
                                  dev(np.asarray(cu, np.int32)), dev(np.asarray(ln, np.int32)), k_bounds=c.bounds)
        assert A.attn_device_status(True) == INVALID
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(was, (*c.gpu["k"], *c.gpu["v"], c.bounds)))
    for entry in (-1, pages, 2 ** 31 - 1):
        bad = table.copy()
        bad[0, 0] = entry
        c = Cache(A, pages, bad, H, P, d)
        was = {n: c.gpu[n][0].clone() for n in "kv"}
        A.attn_rope_kv_append_fp8(q, k, v, f, c.gpu["k"][0], c.gpu["v"][0], c.gpu["k"][1], c.gpu["v"][1], dev(bad), dev(good),
                                  dev(np.asarray(lens, np.int32)), k_bounds=c.bounds)
        assert A.attn_device_status(True) == INVALID
        page = int(table[0, 0])
        assert all(torch.equal(was[n][page], c.gpu[n][0][page]) for n in "kv")
        assert not torch.equal(was["k"][int(table[1, 0])], c.gpu["k"][0][int(table[1, 0])])


def test_captured_replayed_and_on_another_stream(A):
    """Growing lengths in one graph: what it appends is what eager calls append."""
    rng = np.random.RandomState(6)
    B, Hq, H, P, d = 5, 4, 2, 16, 64
    start = [0, 15, 16, 30, 3]
    table, pages = page_tables([n + 8 for n in start], P)
    f = freqs(A, d)
    q, k, v = rows(rng, Hq, H, B, d)
    on = [t.to(DEV) for t in (q, k, v)]
    made = [Cache(A, pages, table, H, P, d) for _ in range(2)]
    lens = dev(np.asarray(start, np.int32))
    tab, cu, fd = dev(table), dev(offsets([1] * B)), dev(f)
    out = torch.empty_like(on[0])
    call = lambda c, **kw: A.attn_rope_kv_append_fp8(*on, fd, c.gpu["k"][0], c.gpu["v"][0], c.gpu["k"][1], c.gpu["v"][1], tab,
                                                     cu, lens, k_bounds=c.bounds, **kw)
    lens += 1
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(made[0], stream=side)
    side.synchronize()
    want = call(made[1])
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        call(made[0], q_out=out)
    for i in range(6):
        lens += 1
        on[1].mul_(1.5)
        on[0].mul_(-1.25)
        g.replay()
        want = call(made[1])
        assert torch.equal(out, want)
    torch.cuda.synchronize()
    for a, b in zip((*made[0].gpu["k"], *made[0].gpu["v"], made[0].bounds), (*made[1].gpu["k"], *made[1].gpu["v"], made[1].bounds)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
