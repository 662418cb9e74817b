"""Operators of a server that reads less of its cache, with the cases they are timed and checked on.

Four operators over a paged e4m3 cache, each in its plain form (elementary torch operations, 32
bits or more, rounded once at the end) and as the package's own call:

  append  rotary positions of new Q and K rows, K and V written into the cache on the way (K is
          rounded once, to its code), and each page's smallest and largest code per column kept
  select  the pages each query is to read: of a page's bounds and a query, the largest score any
          of its keys could have; the best pages, the first and the last ones, in ascending order
  pages   attention over listed pages only, a list for each query and K/V head
  prefix  attention of sequences that share long prefixes, each followed by its own keys
"""
import math
import random

import torch

own = False  # True: run() makes the package's calls; False: the plain forms

E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One decoding step of 64 sequences: a token each, most pages partly filled, bounds kept.
        dict(name="append_step_b64", op="append", batch=64, heads=32, kv_heads=8, d=128, rot=128, interleaved=False,
             page=64, keys=8192, new=1, even=False, bounds=True, shift=0),
        # Ragged pieces of prompts behind a shared prefix (positions of their own), 64-wide heads of
        # which half turns, pairs interleaved, small pages.
        dict(name="append_ragged_d64", op="append", batch=16, heads=16, kv_heads=4, d=64, rot=32, interleaved=True,
             page=16, keys=4000, new=300, even=False, bounds=True, shift=4096),
        # Two whole prompts of 8192 tokens.
        dict(name="append_prompt_8k", op="append", batch=2, heads=32, kv_heads=8, d=128, rot=128, interleaved=False,
             page=128, keys=8192, new=8192, even=True, bounds=True, shift=0),
        # One conversation far into its context: nothing to hide the latency behind.
        dict(name="select_one_32k", op="select", batch=1, heads=32, kv_heads=8, d=128, page=64, keys=32768, new=1,
             even=True, count=64, first=1, last=2),
        # A busy server: 64 sequences of very different lengths, some shorter than the budget.
        dict(name="select_step_ragged_32k", op="select", batch=64, heads=32, kv_heads=8, d=128, page=32, keys=32768,
             new=1, even=False, count=128, first=1, last=2),
        # Four drafted tokens at once, one K/V head for 32 query heads, small pages.
        dict(name="select_draft_mqa", op="select", batch=8, heads=32, kv_heads=1, d=64, page=16, keys=16001, new=4,
             even=True, count=100, first=2, last=4),
        # The lists of one conversation read: 4096 of its 32768 keys.
        dict(name="pages_one_32k", op="pages", batch=1, heads=32, kv_heads=8, d=128, page=64, keys=32768, new=1,
             even=True, count=64),
        # The same for a batch of 64.
        dict(name="pages_step_ragged_32k", op="pages", batch=64, heads=32, kv_heads=8, d=128, page=32, keys=32768, new=1,
             even=False, count=128),
        # Drafted tokens, groups of 7 heads, 64-wide, small pages, a list for each token.
        dict(name="pages_draft_d64", op="pages", batch=8, heads=28, kv_heads=4, d=64, page=16, keys=9001, new=4, even=False,
             count=75),
        # Eight samples of one prompt, a few hundred tokens into their answers.
        dict(name="prefix_step_b8", op="prefix", batch=8, heads=32, kv_heads=8, d=128, page=64, prefix="8192", keys=300, new=1,
             even=False),
        # A long shared document and 64 questions about it.
        dict(name="prefix_step_b64_32k", op="prefix", batch=64, heads=32, kv_heads=8, d=128, page=64, prefix="32768", keys=1024,
             new=1, even=False),
        # Several system prompts at once (one sequence group has none), pieces of questions.
        dict(name="prefix_groups_pieces", op="prefix", batch=24, heads=16, kv_heads=2, d=64, page=32, prefix="5000 0 16001",
             keys=700, new=60, even=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "select", "pages", "prefix"])
    d = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 7, 8, 20])
    heads = kv_heads * (group if kv_heads < 8 else min(group, 4))
    page = rng.choice([16, 32, 64, 128])
    case = dict(op=op, heads=heads, kv_heads=kv_heads, d=d, page=page, even=rng.random() < 0.3)
    if op == "append":
        new = _log(rng, 1, 4000)
        return dict(case, batch=_log(rng, 1, max(2, min(48, 12000 // new))), keys=new + _log(rng, 1, 4000), new=new,
                    rot=rng.choice([d, d // 2, d // 4 + 8]), interleaved=rng.random() < 0.5, bounds=rng.random() < 0.7,
                    shift=rng.choice([0, 0, 1000, 200000]))
    if op == "prefix":
        groups = [rng.choice([0, _log(rng, 10, 16000), _log(rng, 10, 16000)]) for _ in range(rng.choice([1, 1, 2, 5]))]
        rows = max(1, 60000000 // (heads * (max(groups) + 1500)))      # queries: scores as in the largest listed case
        new = _log(rng, 1, min(300, max(1, rows // len(groups))))
        return dict(case, batch=_log(rng, len(groups), max(len(groups), min(64, rows // new))),
                    prefix=" ".join(map(str, groups)), keys=new + _log(rng, 1, 1500), new=new)
    new = rng.choice([1, 1, 1, 2, 3, 5])
    if op == "pages":
        keys = _log(rng, 8, 30000)
        return dict(case, batch=_log(rng, 1, max(1, min(48, 300000 // keys))), keys=keys, new=new,
                    count=_log(rng, 1, max(2, 3000 // page)))
    first, last = rng.choice([0, 1, 3]), rng.choice([1, 2, 5])
    keys = _log(rng, page * (first + last + 60), 30000)                # the longest sequence has pages to choose from
    spare = -(-keys // page) - first - last - 1
    return dict(case, batch=_log(rng, 1, max(1, min(48, 300000 // keys))), keys=keys, new=new, first=first, last=last,
                count=first + last + _log(rng, 1, min(200, spare)))


def _lengths(case):
    """Each sequence's keys after the call (prefix: its own ones), and how many of them are new."""
    b, keys, new = case["batch"], case["keys"], case["new"]
    if case["even"]:
        return [keys] * b, [new] * b
    rng = random.Random("%d %d %d %d" % (b, keys, new, case["page"]))
    total = [keys] + [rng.randint(max(1, keys // 64), keys) for _ in range(b - 1)]
    fresh = [new] + [rng.randint(1, new) for _ in range(b - 1)]
    return total, [min(n, t) for n, t in zip(fresh, total)]


def _shared(case):
    return [int(n) for n in case.get("prefix", "").split()]


def _members(case):
    """Sequences per prefix: as even as they go."""
    g, b = len(_shared(case)), case["batch"]
    return [(i + 1) * b // g - i * b // g for i in range(g)]


def work(case):
    total, fresh = _lengths(case)
    d, Hq, Hk, P, T = case["d"], case["heads"], case["kv_heads"], case["page"], sum(fresh)
    if case["op"] == "append":
        pages = sum(n // P + 1 for n in fresh)
        return {"bytes": T * (Hq * d * 4 + Hk * 2 * d * 3) + pages * Hk * (8 + (2 * d if case["bounds"] else 0)) + T * 4,
                "flops": T * ((Hq + Hk) * case["rot"] * 3 + Hk * d * 4)}
    if case["op"] == "select":
        rows = sum(-(-t // P) for t in total) * Hk
        return {"bytes": rows * (2 * d + 4) + T * (Hq * d * 2 + Hk * case["count"] * 4),
                "flops": sum(-(-t // P) * n for t, n in zip(total, fresh)) * Hq * d * 4}
    if case["op"] == "pages":
        # Lists of the same sequence may overlap: what they must read is at most the sequence itself.
        seen = [min(t, case["count"] * P) for t in total]
        read = sum(min(t, n * s) for t, n, s in zip(total, fresh, seen)) * Hk
        return {"bytes": read * (2 * d + 8 / P) + T * (Hq * (d * 4 + 4) + Hk * case["count"] * 4),
                "flops": 4 * sum(n * s for n, s in zip(fresh, seen)) * Hq * d}
    keys, pairs, at = sum(total) + sum(_shared(case)), 0, 0
    for p, m in zip(_shared(case), _members(case)):
        pairs += sum(n * (p + t) - n * (n - 1) // 2 for t, n in zip(total[at:at + m], fresh[at:at + m]))
        at += m
    return {"bytes": keys * Hk * (2 * d + 8 / P) + T * Hq * (d * 4 + 4), "flops": 4 * pairs * Hq * d}


# ------------------------------------------------------------------ inputs
def _power(amax):
    """The smallest power of two s with amax / s <= 448 (0 for 0)."""
    m, e = torch.frexp(amax)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e - torch.where(m <= 0.875, 9, 8)), 0.0)


def _code(x, scale):
    """e4m3 values (as such) of x / scale, scale a power of two or 0."""
    safe = torch.where(scale > 0, scale, 1.0)
    return (x / safe).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _cache(pages, Hk, P, d, gen, dev):
    """Codes and scales of unit normals with a gain for each page and head."""
    codes = torch.empty((pages, Hk, P, d), dtype=torch.uint8, device=dev)
    scale = torch.empty((pages, Hk), device=dev)
    for p in range(0, pages, 2048):
        x = torch.randn((min(2048, pages - p), Hk, P, d), generator=gen, device=dev)
        x *= torch.exp2(torch.randn(x.shape[:2], generator=gen, device=dev) * 0.5)[..., None, None]
        s = _power(x.abs().amax((-2, -1)))
        codes[p:p + 2048], scale[p:p + 2048] = _code(x, s[..., None, None]).view(torch.uint8), s
    return codes, scale


def _tables(need, gen, dev, start, order):
    width = max(need) + 1
    table = torch.full((len(need), width), -1, dtype=torch.int32, device=dev)
    for b, n in enumerate(need):
        table[b, :n] = order[start:start + n]
        start += n
    return table, start


def _offsets(ns, dev):
    return torch.tensor([sum(ns[:b]) for b in range(len(ns) + 1)], dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    op, d, P, Hq, Hk = case["op"], case["d"], case["page"], case["heads"], case["kv_heads"]
    total, fresh = _lengths(case)
    B, T = case["batch"], sum(fresh)
    need = [-(-t // P) for t in total]
    shared = [-(-t // P) for t in _shared(case)]
    pages = sum(need) + sum(shared) + 3
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    st = dict(op=op, page=P, new_max=max(fresh), kv_lens=torch.tensor(total, dtype=torch.int32, device=dev),
              cu=_offsets(fresh, dev), workspace=None, scale=d ** -0.5)
    st["table"], at = _tables(need, gen, dev, 0, order)
    rows = torch.randn((T, Hq + 2 * Hk, d), generator=gen, device=dev).to(torch.bfloat16)  # a fused projection's output
    if op == "append":
        st["q"], st["k"], st["v"] = (rows[:, lo:hi].transpose(0, 1) for lo, hi in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk)))
        j = torch.arange(0, case["rot"], 2, dtype=torch.float64, device=dev)
        st["inv_freq"] = 500000.0 ** (-j / case["rot"])
        st.update(rot=case["rot"], interleaved=case["interleaved"], mscale=1.0, positions=None, k_bounds=None)
        tok = torch.arange(T, device=dev)
        seq = torch.searchsorted(st["cu"][1:].long(), tok, right=True)
        start = st["kv_lens"].long() - st["cu"][1:] + st["cu"][:-1]
        st["q_out"] = torch.empty((Hq, T, d), dtype=torch.bfloat16, device=dev)
        if case["shift"]:
            st["positions"] = (start[seq] + tok - st["cu"].long()[seq] + case["shift"]).to(torch.int32)
        for n in ("k", "v"):
            st[n + "_cache"], st[n + "_scale"] = _cache(pages, Hk, P, d, gen, dev)
        if case["bounds"]:  # of the rows that earlier calls wrote
            st["k_bounds"] = torch.zeros((pages, Hk, 2, d), dtype=torch.uint8, device=dev)
            blocks = torch.arange(st["table"].shape[1], device=dev)
            had = (start[:, None] - blocks * P).clamp(0, P)
            used = torch.zeros(pages, dtype=torch.long, device=dev)
            used[st["table"].long().clamp(min=0)[had > 0]] = had[had > 0]
            _bound_pages(st, torch.nonzero(used)[:, 0], used)
        return st
    if op == "select":  # the extremes of P unit normals, around a mean of their own for each column, page and head
        u = torch.rand((pages, Hk, 2, d), generator=gen, device=dev, dtype=torch.float64).clamp_(1e-12)
        top = torch.special.ndtri(u ** (1.0 / P)).float()
        mean = torch.randn((1, Hk, 1, d), generator=gen, device=dev) + torch.randn((pages, Hk, 1, d), generator=gen, device=dev) * 0.5
        gain = torch.exp2(torch.randn((pages, Hk, 1, 1), generator=gen, device=dev) * 0.2)
        x = (torch.cat((torch.minimum(-top[:, :, :1], top[:, :, 1:]), torch.maximum(-top[:, :, :1], top[:, :, 1:])), 2) + mean) * gain
        s = _power(x.abs().amax((-2, -1)))
        st["k_bounds"], st["k_scale"] = _code(x, s[..., None, None]).view(torch.uint8), s
        st["q"] = rows[:, :Hq].transpose(0, 1).contiguous()
        st.update(count=case["count"], first=case["first"], last=case["last"],
                  pages=torch.empty((Hk, T, case["count"]), dtype=torch.int32, device=dev))
        return st
    for n in ("k", "v"):
        st[n + "_cache"], st[n + "_scale"] = _cache(pages, Hk, P, d, gen, dev)
    st["q"] = rows[:, :Hq].transpose(0, 1).contiguous()
    st["o"], st["lse"] = torch.empty_like(st["q"]), torch.empty((Hq, T), device=dev)
    if op == "pages":  # the first and the last page a query sees, and random ones between
        seq = torch.searchsorted(st["cu"][1:].long(), torch.arange(T, device=dev), right=True)
        visible = (_last_key(st)[seq, torch.arange(T, device=dev) - st["cu"].long()[seq]] // P + 1)[None, :, None]
        block = torch.arange(max(need), device=dev)
        luck = torch.rand((Hk, T, max(need)), generator=gen, device=dev)
        luck = torch.where((block == 0) | (block == visible - 1), 2.0, luck)
        luck = torch.where(block < visible, luck, -1.0)
        n = min(case["count"], max(need))
        best, at = luck.topk(n, -1)
        at = torch.where(best < 0, block.numel(), at).sort(-1)[0]
        st["pages"] = torch.full((Hk, T, case["count"]), -1, dtype=torch.int32, device=dev)
        st["pages"][..., :n] = torch.where(at < block.numel(), at, -1)
        return st
    st["prefix_table"], _ = _tables(shared, gen, dev, at, order)
    st["prefix_lens"] = torch.tensor(_shared(case), dtype=torch.int32, device=dev)
    ends = [sum(_members(case)[:i]) for i in range(len(shared) + 1)]
    st["cu_prefix"] = st["cu"][torch.tensor(ends, device=dev)].contiguous()
    st["prefix_q_max"] = max(sum(fresh[a:b]) for a, b in zip(ends, ends[1:]))
    st.update(prefix_max=max(_shared(case)), keys_max=max(total))
    return st


def _last_key(st):
    """[B, n]: the last key that each query of each sequence sees."""
    start = st["kv_lens"].long() - st["cu"][1:] + st["cu"][:-1]
    return torch.minimum(start[:, None] + torch.arange(st["new_max"], device=start.device), st["kv_lens"].long()[:, None] - 1)


# ------------------------------------------------------------------ one pass
def run(st):
    if own:
        return _own(st)
    return {"append": _append, "select": _select, "pages": _pages, "prefix": _prefix}[st["op"]](st)


def _own(st):
    import attention_attn_fwd_09_gb300 as A
    if st["op"] == "append":
        A.attn_rope_kv_append_fp8(st["q"], st["k"], st["v"], st["inv_freq"], st["k_cache"], st["v_cache"], st["k_scale"],
                                  st["v_scale"], st["table"], st["cu"], st["kv_lens"], positions=st["positions"],
                                  interleaved=st["interleaved"], mscale=st["mscale"], k_bounds=st["k_bounds"], q_out=st["q_out"])
        return _written(st)
    if st["op"] == "select":
        if st["workspace"] is None:  # a server keeps it from call to call
            n = A.attn_select_pages_fp8_workspace_size(st["k_bounds"].shape[1], st["q"].shape[1], st["table"].shape[1])
            st["workspace"] = torch.empty((max(n, 16),), dtype=torch.uint8, device=st["q"].device)
        return A.attn_select_pages_fp8(st["q"], st["k_bounds"], st["k_scale"], st["table"], st["cu"], st["kv_lens"], st["page"],
                                       st["count"], st["new_max"], first=st["first"], last=st["last"], pages=st["pages"],
                                       workspace=st["workspace"])
    T, Hq, Hk, d = st["q"].shape[1], st["q"].shape[0], st["k_cache"].shape[1], st["q"].shape[2]
    if st["op"] == "pages":
        if st["workspace"] is None:
            n = A.attn_fwd_kv_fp8_pages_workspace_size(Hq, Hk, T, d)
            st["workspace"] = torch.empty((max(n, 16),), dtype=torch.uint8, device=st["q"].device)
        return A.attn_fwd_kv_fp8_pages(st["q"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"], st["table"], st["cu"],
                                       st["kv_lens"], st["pages"], scale=st["scale"], o=st["o"], lse=st["lse"],
                                       workspace=st["workspace"])
    if st["workspace"] is None:
        n = A.attn_fwd_kv_fp8_prefix_workspace_size(Hq, Hk, T, st["prefix_q_max"], st["new_max"], d)
        st["workspace"] = torch.empty((max(n, 16),), dtype=torch.uint8, device=st["q"].device)
    return A.attn_fwd_kv_fp8_prefix(st["q"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"], st["prefix_table"],
                                    st["cu_prefix"], st["prefix_lens"], st["prefix_q_max"], st["table"], st["cu"], st["kv_lens"],
                                    st["new_max"], scale=st["scale"], o=st["o"], lse=st["lse"], workspace=st["workspace"])


def _written(st):
    """The rotated queries, and the cache and its bounds as the values the codes stand for (before
    their scales)."""
    out = {"q": st["q_out"], "k": st["k_cache"].view(torch.float8_e4m3fn), "v": st["v_cache"].view(torch.float8_e4m3fn),
           "k_scale": st["k_scale"], "v_scale": st["v_scale"]}
    if st["k_bounds"] is not None:
        out["k_bounds"] = st["k_bounds"].view(torch.float8_e4m3fn)
    return out


def _bound_pages(st, pages, used):
    """Smallest and largest code of each column over the first used[page] rows of these pages."""
    x = st["k_cache"].view(torch.float8_e4m3fn)[pages].float()
    hidden = torch.arange(st["page"], device=x.device)[:, None] >= used[pages][:, None, None, None]
    low, high = x.masked_fill(hidden, math.inf).amin(2), x.masked_fill(hidden, -math.inf).amax(2)
    st["k_bounds"][pages] = torch.stack((low, high), 2).to(torch.float8_e4m3fn).view(torch.uint8)


def _turn(x, cos, sin, rot, interleaved):
    x = x.float()
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    y, z = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((y, z), -1).flatten(-2) if interleaved else torch.cat((y, z), -1)
    return torch.cat((r, x[..., rot:]), -1)


def _append_one(xf, codes, scale, st, seq, pos, start):
    P = st["page"]
    xf = xf.transpose(0, 1)                                                 # [T, H, d]
    page = st["table"].long()[seq, pos // P]
    fresh = _power(torch.zeros_like(scale).index_reduce_(0, page, xf.abs().amax(-1), "amax"))
    # Only the first page a sequence writes to can hold earlier rows: their scale may only grow,
    # and the rows are rounded again when it does.
    head = st["table"].long().gather(1, (start // P)[:, None])[:, 0]
    slot = start % P
    was = torch.where((slot > 0)[:, None], scale[head], 0.0)
    wanted = fresh.index_reduce(0, head, was, "amax")                       # every page's scale, were it written to
    scale[page] = wanted[page]
    old = codes[head].view(torch.float8_e4m3fn).float() * was[..., None, None]
    again = _code(old, wanted[head][..., None, None]).view(torch.uint8)
    earlier = torch.arange(P, device=xf.device) < slot[:, None]
    codes[head] = torch.where(earlier[:, None, :, None], again, codes[head])
    codes[page, :, pos % P] = _code(xf, wanted[page][..., None]).view(torch.uint8)


def _append(st):
    cu, P = st["cu"].long(), st["page"]
    T = st["k"].shape[1]
    tok = torch.arange(T, device=cu.device)
    seq = torch.searchsorted(cu[1:], tok, right=True)
    start = st["kv_lens"].long() - (cu[1:] - cu[:-1])
    pos = start[seq] + tok - cu[seq]
    # Angles in 64 bits: a far position times a frequency near 1 keeps no fraction in 32.
    angle = (pos if st["positions"] is None else st["positions"]).double()[:, None] * st["inv_freq"]
    cos, sin = (angle.cos() * st["mscale"]).float(), (angle.sin() * st["mscale"]).float()
    st["q_out"].copy_(_turn(st["q"], cos, sin, st["rot"], st["interleaved"]))
    _append_one(_turn(st["k"], cos, sin, st["rot"], st["interleaved"]), st["k_cache"], st["k_scale"], st, seq, pos, start)
    _append_one(st["v"].float(), st["v_cache"], st["v_scale"], st, seq, pos, start)
    if st["k_bounds"] is not None:
        page = st["table"].long()[seq, pos // P]
        used = torch.zeros(st["k_cache"].shape[0], dtype=torch.long, device=cu.device)
        used[page] = (st["kv_lens"].long()[seq] - pos // P * P).clamp(max=P)
        _bound_pages(st, torch.unique(page), used)
    return _written(st)


def _select(st):
    """Scores in 64 bits: what decides is which of two pages near the border is ahead."""
    q, P, count, first, last = st["q"], st["page"], st["count"], st["first"], st["last"]
    Hq, T, d = q.shape
    Hk = st["k_scale"].shape[1]
    cu, blocks = st["cu"].long(), st["table"].shape[1]
    tok = torch.arange(T, device=q.device)
    seq = torch.searchsorted(cu[1:], tok, right=True)
    visible = _last_key(st)[seq, tok - cu[seq]] // P + 1                                    # pages each query sees
    x = q.double().view(Hk, Hq // Hk, T, d)
    score = torch.empty((Hk, T, blocks), dtype=torch.float64, device=q.device)
    pages = st["table"].long().clamp(min=0)
    bounds = st["k_bounds"].view(torch.float8_e4m3fn)
    for h in range(Hk):
        for t0 in range(0, T, 64):
            s = seq[t0:t0 + 64]
            low, high = (bounds[pages[s], h, i].double() for i in (0, 1))                   # [t, blocks, d]
            y = x[h, :, t0:t0 + 64].transpose(0, 1)                                         # [t, g, d]
            v = y.clamp(min=0) @ high.transpose(1, 2) + y.clamp(max=0) @ low.transpose(1, 2)
            score[h, t0:t0 + 64] = v.amax(1) * st["k_scale"][pages[s], h].double()
    block = torch.arange(blocks, device=q.device)
    kept = (block < first) | (block >= visible[:, None] - last)
    score = torch.where(kept, math.inf, score).masked_fill(block >= visible[:, None], -math.inf)
    n = min(count, blocks)
    at = torch.sort(score, dim=-1, descending=True, stable=True)[1][..., :n]                # equal ones by index
    at = torch.where(at < visible[:, None], at, blocks).sort(-1)[0]
    st["pages"].fill_(-1)
    st["pages"][..., :n] = torch.where(at < blocks, at, -1)
    return st["pages"]


def _softmax(s, v):
    """softmax(s) v and the log-sum-exp of rows that may be empty."""
    top = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    return (p @ v) / torch.where(total > 0, total, 1.0), (top + total.log())[..., 0]


def _pages(st):
    q, P, listed_pages = st["q"], st["page"], st["pages"]
    Hq, T, d = q.shape
    Hk = st["k_cache"].shape[1]
    g, cu = Hq // Hk, st["cu"].long()
    tok = torch.arange(T, device=q.device)
    seq = torch.searchsorted(cu[1:], tok, right=True)
    last = _last_key(st)[seq, tok - cu[seq]]
    o, lse = torch.empty((T, Hk, g, d), device=q.device), torch.empty((T, Hk, g), device=q.device)
    x = q.float().transpose(0, 1).reshape(T, Hk, g, d)
    head = torch.arange(Hk, device=q.device)[:, None]
    for t0 in range(0, T, 32):
        t1 = min(T, t0 + 32)
        block = listed_pages[:, t0:t1].long().transpose(0, 1)                               # [t, Hk, count]
        page = st["table"].long()[seq[t0:t1, None, None], block.clamp(min=0)].clamp(min=0)
        key = (block * P)[..., None] + torch.arange(P, device=q.device)
        hidden = ((key > last[t0:t1, None, None, None]) | (block < 0)[..., None]).flatten(2)  # [t, Hk, keys]
        k, v = ((st[n + "_cache"][page, head].view(torch.float8_e4m3fn).float()
                 * st[n + "_scale"][page, head][..., None, None]).flatten(2, 3) for n in ("k", "v"))
        s = (x[t0:t1] @ k.transpose(2, 3) * st["scale"]).masked_fill_(hidden[:, :, None], -math.inf)
        o[t0:t1], lse[t0:t1] = _softmax(s, v.masked_fill_(hidden[..., None], 0.0))
    return o.flatten(1, 2).transpose(0, 1).contiguous().to(torch.bfloat16), lse.flatten(1, 2).transpose(0, 1).contiguous()


def _gather(codes, scale, table, blocks):
    pages = table[:, :blocks].long().clamp(min=0)
    x = codes[pages].view(torch.float8_e4m3fn).float().mul_(scale[pages][..., None, None])   # [B, blocks, H, P, d]
    return x.transpose(1, 2).flatten(2, 3)                                                    # [B, H, keys, d]


def _part(st, cu, table, lens, keys, rows, last):
    """O and LSE of every query over one table's keys: the queries of a table's row padded to `rows`."""
    q, P, Hk = st["q"], st["page"], st["k_cache"].shape[1]
    Hq, T, d = q.shape
    g, B, n = Hq // Hk, lens.numel(), rows
    if keys == 0:
        return torch.zeros((T, Hq, d), device=q.device), torch.full((T, Hq), -math.inf, device=q.device)
    tok = torch.arange(T, device=q.device)
    seq = torch.searchsorted(cu[1:], tok, right=True)
    row = tok - cu[seq]
    padded = torch.zeros((B, n, Hq, d), device=q.device)
    padded[seq, row] = q.float().transpose(0, 1)
    padded = padded.view(B, n, Hk, g, d).permute(0, 2, 3, 1, 4).reshape(B, Hk, g * n, d)
    blocks = -(-keys // P)
    key = torch.arange(blocks * P, device=q.device)
    hidden = (key > last[..., None])[:, None, None].expand(B, 1, g, n, key.numel()).reshape(B, 1, g * n, key.numel())
    s = padded @ _gather(st["k_cache"], st["k_scale"], table, blocks).transpose(2, 3)
    s = s.mul_(st["scale"]).masked_fill_(hidden, -math.inf)
    v = _gather(st["v_cache"], st["v_scale"], table, blocks).masked_fill_((key >= lens[:, None])[:, None, :, None], 0.0)
    o, lse = _softmax(s, v)
    o = o.view(B, Hk, g, n, d).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, d)
    lse = lse.view(B, Hk, g, n).permute(0, 3, 1, 2).reshape(B, n, Hq)
    return o[seq, row], lse[seq, row]


def _prefix(st):
    lens, shared = st["kv_lens"].long(), st["prefix_lens"].long()
    rows = st["prefix_q_max"]
    o1, l1 = _part(st, st["cu_prefix"].long(), st["prefix_table"], shared, st["prefix_max"], rows,
                   (shared - 1)[:, None].expand(-1, rows))
    o2, l2 = _part(st, st["cu"].long(), st["table"], lens, st["keys_max"], st["new_max"], _last_key(st))
    lse = torch.logaddexp(l1, l2)
    o = o1 * (l1 - lse).exp()[..., None] + o2 * (l2 - lse).exp()[..., None]
    return o.transpose(0, 1).contiguous().to(torch.bfloat16), lse.transpose(0, 1).contiguous()


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_append(case, st):
    total, fresh = _lengths(case)
    P, rot, out = case["page"], case["rot"], {}
    grid = torch.arange(127, dtype=torch.uint8, device=st["k"].device).view(torch.float8_e4m3fn).double()
    where = torch.cat([torch.arange(t - n, t) for t, n in zip(total, fresh)]).to(grid.device).double() + case["shift"]
    turn = torch.polar(torch.ones((1, 1), dtype=torch.float64, device=grid.device), where[:, None] * st["inv_freq"])

    def rotated(x):
        y = x.double().contiguous()
        if case["interleaved"]:
            z = torch.view_as_complex(y[..., :rot].unflatten(-1, (rot // 2, 2)).contiguous()) * turn
            y[..., :rot] = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * turn
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        return y

    def nearest(y):  # the e4m3 value next to y; halfway, the one with the even code
        a = y.abs().clamp(max=E4M3_MAX)
        up = torch.searchsorted(grid, a.contiguous()).clamp(max=126)
        lo = (up - 1).clamp(min=0)
        near, far = grid[up] - a, a - grid[lo]
        pick = torch.where((near < far) | ((near == far) & (up % 2 == 0)), up, lo)
        return torch.copysign(grid[pick], y)

    out["q"] = rotated(st["q"])
    for name in ("k", "v"):
        codes = st[name + "_cache"].view(torch.float8_e4m3fn).double()
        bounds = None
        if name == "k" and st["k_bounds"] is not None:
            bounds = st["k_bounds"].view(torch.float8_e4m3fn).double()
        scale, x, at = st[name + "_scale"].double(), rotated(st["k"]) if name == "k" else st["v"].double(), 0
        for t, n, row in zip(total, fresh, st["table"].tolist()):
            begin = t - n
            for block in range(begin // P, (t - 1) // P + 1):
                lo, hi = max(begin, block * P), min(t, (block + 1) * P)
                new = x[:, at + lo - begin:at + hi - begin]
                page, kept = row[block], lo - block * P
                s = torch.exp2(torch.ceil(torch.log2(new.abs().amax((1, 2)) / E4M3_MAX)))
                if kept:
                    before = scale[page].clone()
                    s = torch.maximum(s, before)
                    codes[page, :, :kept] = nearest(codes[page, :, :kept] * (before / s)[:, None, None])
                scale[page] = s
                codes[page, :, kept:kept + hi - lo] = nearest(new / s[:, None, None])
                if bounds is not None:
                    mine = codes[page, :, :kept + hi - lo]
                    bounds[page, :, 0], bounds[page, :, 1] = mine.amin(1), mine.amax(1)
            at += n
        out[name], out[name + "_scale"] = codes, scale
        if bounds is not None:
            out["k_bounds"] = bounds
    return {n: out[n] for n in ("q", "k", "v", "k_scale", "v_scale", "k_bounds") if n in out}


def _exact_select(case, st):
    """By the definition: each column's larger product, page by page, and the ranks counted out."""
    total, fresh = _lengths(case)
    Hk, g, P, count = case["kv_heads"], case["heads"] // case["kv_heads"], case["page"], case["count"]
    out, at = torch.full_like(st["pages"], -1), 0
    for b, (t, n) in enumerate(zip(total, fresh)):
        for i in range(n):
            sees = (t - n + i) // P + 1
            if sees <= count:
                out[:, at + i, :sees] = torch.arange(sees, device=out.device)
                continue
            pages = st["table"][b, :sees].long()
            lo, hi = case["first"], sees - case["last"]
            pool = pages[lo:hi]
            ends = st["k_bounds"][pool].view(torch.float8_e4m3fn).double() * st["k_scale"][pool].double()[..., None, None]
            q = st["q"][:, at + i].double().view(Hk, g, -1)
            for h in range(Hk):
                s = torch.maximum(q[h, :, None] * ends[None, :, h, 0], q[h, :, None] * ends[None, :, h, 1]).sum(-1).amax(0)
                ahead = torch.argsort(s, descending=True, stable=True)[:count - case["first"] - case["last"]] + lo
                chosen = torch.cat((torch.arange(lo, device=out.device), ahead, torch.arange(hi, sees, device=out.device)))
                out[h, at + i] = chosen.sort()[0].to(torch.int32)
        at += n
    return out


def _attention(q, k, v, hidden, scale):
    s = (q @ k.T * scale).masked_fill(hidden, -math.inf)
    return torch.softmax(s, -1) @ v, torch.logsumexp(s, -1)


def _keys(st, pages, h, name):
    return (st[name + "_cache"][pages, h].view(torch.float8_e4m3fn).double()
            * st[name + "_scale"][pages, h].double()[:, None, None]).flatten(0, 1)


def _exact_pages(case, st):
    total, fresh = _lengths(case)
    Hk, g, P = case["kv_heads"], case["heads"] // case["kv_heads"], case["page"]
    o, lse, at = torch.empty_like(st["q"], dtype=torch.float64), torch.empty_like(st["lse"], dtype=torch.float64), 0
    for b, (t, n) in enumerate(zip(total, fresh)):
        for i in range(n):
            for h in range(Hk):
                block = st["pages"][h, at + i].long()
                block = block[block >= 0]
                pages, key = st["table"][b].long()[block], (block[:, None] * P + torch.arange(P, device=o.device)).flatten()
                rows = slice(h * g, (h + 1) * g)
                o[rows, at + i], lse[rows, at + i] = _attention(st["q"][rows, at + i].double(), _keys(st, pages, h, "k"),
                                                                _keys(st, pages, h, "v"), key > t - n + i, st["scale"])
        at += n
    return o, lse


def _exact_prefix(case, st):
    total, fresh = _lengths(case)
    Hk, g, P = case["kv_heads"], case["heads"] // case["kv_heads"], case["page"]
    o, lse, at, b = torch.empty_like(st["q"], dtype=torch.float64), torch.empty_like(st["lse"], dtype=torch.float64), 0, 0
    for j, (m, shared) in enumerate(zip(_members(case), _shared(case))):
        front = st["prefix_table"][j, :-(-shared // P)].long()
        head = [[_keys(st, front, h, c)[:shared] for c in ("k", "v")] for h in range(Hk)]
        for _ in range(m):
            t, n = total[b], fresh[b]
            mine = st["table"][b, :-(-t // P)].long()
            here = torch.arange(n, device=o.device)[:, None]
            hidden = torch.arange(shared + t, device=o.device) > shared + t - n + here
            for h in range(Hk):
                k, v = (torch.cat((x, _keys(st, mine, h, c)[:t])) for x, c in zip(head[h], ("k", "v")))
                for r in range(h * g, (h + 1) * g):
                    o[r, at:at + n], lse[r, at:at + n] = _attention(st["q"][r, at:at + n].double(), k, v, hidden, st["scale"])
            at, b = at + n, b + 1
    return o, lse


def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "select": _exact_select, "pages": _exact_pages, "prefix": _exact_prefix}[case["op"]](case, st)
