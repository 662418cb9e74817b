"""The cache's calls together, as a server makes them: prompts and tokens appended with rotation and
bounds, pages chosen, attention over them or behind a shared prefix, step by step in one graph; each
step against the fp64 oracle of what the cache holds."""
import numpy as np
import pytest
import torch

import oracle.cache as oc
import oracle.sparse as osp
from cache_cases import bf16, check, offsets, page_tables
from oracle.fp8 import e4m3_decode
from test_cache_parts_gpu import SHAPES, check_prefix  # noqa: F401  (the joint's bound)

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def A():
    import attention_attn_fwd_09_gb300 as A
    A.attn_set_debug_knobs()
    A.attn_device_status(True)
    yield A
    assert A.attn_device_status(True) == 0


class Server:
    def __init__(self, A, lens, steps, Hq, H, P, d, seed=0, spare=0):
        self.A, self.Hq, self.H, self.P, self.d = A, Hq, H, P, d
        self.table, self.pages = page_tables([n + steps for n in lens], P, seed, spare=spare + 2)
        u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device=DEV)
        self.k, self.v, self.bounds = u8(self.pages, H, P, d), u8(self.pages, H, P, d), u8(self.pages, H, 2, d)
        self.ks, self.vs = (torch.zeros(self.pages, H, device=DEV) for _ in range(2))
        self.freqs, self.m = A.attn_rope_freqs(d, 10000.0)
        self.rng = np.random.RandomState(seed + 5)

    def projected(self, T):
        """A fused projection's output, [tokens, heads, d], as the views the calls take."""
        x = bf16(self.rng.randn(T, self.Hq + 2 * self.H, self.d)).to(DEV)
        return x[:, :self.Hq].transpose(0, 1), x[:, self.Hq:self.Hq + self.H].transpose(0, 1), x[:, self.Hq + self.H:].transpose(0, 1)

    def append(self, q, k, v, table, cu, lens, **kw):
        return self.A.attn_rope_kv_append_fp8(q, k, v, self.freqs, self.k, self.v, self.ks, self.vs, table, cu, lens,
                                              mscale=self.m, k_bounds=self.bounds, **kw)

    def cache(self):
        return self.k, self.v, self.ks, self.vs

    def state(self, table, cu, lens, q):
        """What the oracle reads."""
        return dict(k_cache=self.k.cpu().numpy(), v_cache=self.v.cpu().numpy(), k_scale=self.ks.cpu().numpy(),
                    v_scale=self.vs.cpu().numpy(), table=table.cpu().numpy(), cu=cu.cpu().numpy(), lens=lens.cpu().numpy(), q=q.cpu())


def i32(x):
    return torch.tensor(np.asarray(x, np.int32), device=DEV)


@pytest.mark.parametrize("Hq,H,P,d", [(8, 2, 16, 64), (4, 1, 32, 128)])
def test_sparse_decoding_in_a_graph(A, Hq, H, P, d):
    """Prompts, then single tokens: append, choose 5 pages, attend over them, one graph replayed for
    every token while the lengths grow past page borders; queries and lists against the oracle."""
    lens, steps, count = [3, 9 * P - 2, 20 * P + 1], 6, 5
    s = Server(A, lens, steps, Hq, H, P, d, seed=P)
    table, kv_lens = i32(s.table), i32(lens)
    q, k, v = s.projected(sum(lens))
    cu = i32(offsets(lens))
    qr = s.append(q, k, v, table, cu, kv_lens)
    whole, _ = A.attn_fwd_kv_fp8(qr, *s.cache(), table, cu, kv_lens, max(lens))
    assert torch.isfinite(whole).all()
    one = i32([0, 1, 2, 3])
    row = [t.clone() for t in s.projected(3)]
    out = torch.empty((Hq, 3, d), dtype=torch.bfloat16, device=DEV)
    pages = torch.empty((H, 3, count), dtype=torch.int32, device=DEV)
    o, lse = torch.empty_like(out), torch.empty((Hq, 3), device=DEV)
    ws = [torch.empty(max(n, 16), dtype=torch.uint8, device=DEV) for n in
          (A.attn_select_pages_fp8_workspace_size(H, 3, s.table.shape[1]), A.attn_fwd_kv_fp8_pages_workspace_size(Hq, H, 3, d))]

    def step():
        kv_lens.add_(1)
        s.append(*row, table, one, kv_lens, q_out=out)
        A.attn_select_pages_fp8(out, s.bounds, s.ks, table, one, kv_lens, P, count, 1, first=1, last=2, pages=pages, workspace=ws[0])
        A.attn_fwd_kv_fp8_pages(out, *s.cache(), table, one, kv_lens, pages, o=o, lse=lse, workspace=ws[1])

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(steps - 1):
        for t, x in zip(row, s.projected(3)):
            t.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        c = s.state(table, one, kv_lens, out)
        qn = out.float().cpu().numpy()
        want = osp.select_pages(qn, e4m3_decode(s.bounds.cpu().numpy()), c["k_scale"], c["table"], c["cu"], c["lens"], P, count, 1, 2, True)
        assert (pages.cpu().numpy() == want).all()
        used = np.zeros(s.pages, int)
        for b, n in enumerate(c["lens"]):
            for blk in range(-(-int(n) // P)):
                used[s.table[b, blk]] = min(P, int(n) - blk * P)
        live = used > 0
        assert (e4m3_decode(s.bounds.cpu().numpy())[live] == osp.page_bounds(c["k_cache"][live], used[live])).all()
        check(o, lse, osp.attend_pages(qn, c, want, True, d ** -0.5), d)
    assert A.attn_device_status(True) == 0


@pytest.mark.parametrize("Hq,H,P,d", [(8, 2, 32, 64), (6, 6, 64, 128)])
def test_questions_behind_a_shared_document(A, Hq, H, P, d):
    """One document appended once, then questions of several sequences behind it (positions go on from its
    end), then their answers token by token."""
    doc, asked, steps = 5 * P + 7, [4, 1, 19, 2], 3
    s = Server(A, [doc, *asked], steps, Hq, H, P, d, seed=3)
    front, own = i32(s.table[:1]), i32(s.table[1:])
    q, k, v = s.projected(doc)
    s.append(q, k, v, front, i32([0, doc]), i32([doc]))
    lens, ns = np.array(asked), asked
    for _ in range(steps + 1):
        T = sum(ns)
        cu, kv_lens, pos = i32(offsets(ns)), i32(lens), np.concatenate([np.arange(n - x, n) for n, x in zip(lens, ns)]) + doc
        q, k, v = s.projected(T)
        qr = s.append(q, k, v, own, cu, kv_lens, positions=i32(pos))
        pre = dict(table=s.table[:1], cu=np.array([0, T], np.int32), lens=np.array([doc], np.int32))
        check_prefix(A, s.state(own, cu, kv_lens, qr), pre)
        ns = [1] * len(asked)
        lens = lens + 1


def test_every_page_listed_and_a_prefix_of_none_are_the_whole_attention(A):
    """Three ways to the same keys: within their bounds of one oracle."""
    Hq, H, P, d, lens = 8, 2, 64, 128, [500, 64, 129]
    s = Server(A, lens, 0, Hq, H, P, d, seed=9)
    table, kv_lens, cu = i32(s.table), i32(lens), i32(offsets(lens))
    q, k, v = s.projected(sum(lens))
    qr = s.append(q, k, v, table, cu, kv_lens)
    last = torch.stack([qr[:, n - 1] for n in np.cumsum(lens)], 1).contiguous()
    one = i32([0, 1, 2, 3])
    c = s.state(table, one, kv_lens, last)
    ref = oc.attend(last.float().cpu().numpy(), c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], c["table"], c["cu"],
                    c["lens"], True, d ** -0.5)
    pages = A.attn_select_pages_fp8(last, s.bounds, s.ks, table, one, kv_lens, P, 8, 1)
    check(*A.attn_fwd_kv_fp8(last, *s.cache(), table, one, kv_lens, 1), ref, d)
    check(*A.attn_fwd_kv_fp8_pages(last, *s.cache(), table, one, kv_lens, pages), ref, d)
    none = i32([[-1]])
    o, lse = A.attn_fwd_kv_fp8_prefix(last, *s.cache(), none, i32([0, 3]), i32([0]), 3, table, one, kv_lens, 1)
    check(o, lse, ref, d)
