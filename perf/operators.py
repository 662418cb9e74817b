"""Operators around a decoder's attention call, with the cases they are timed and checked on.

Three operators, each in its plain form (elementary torch operations, 32 bits or more,
rounded once at the end) and as the package's own call:

  rope    rotary positions of Q and K as they come out of a projection ([tokens, heads, d]
          views), forward and backward, half-split and interleaved pairs, part of the head,
          frequencies scaled for long contexts
  append  new K, V rows written into a paged e4m3 cache that has one fp32 scale per page and
          head (the smallest power of two that keeps the page within +-448)
  attend  attention of packed queries over such a cache: softmax(scale Q K^T [causal]) V and
          the row's log-sum-exp, the queries standing at the end of each sequence
"""
import math
import random

import torch

own = False  # True: run() makes the package's calls; False: the plain forms

E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One decoding step of a batch of 8 (32 query and 8 K/V heads), far into a context
        # stretched to four times the trained length: latency is everything.
        dict(name="rope_step_b8", op="rope", batch=1, tokens=8, heads=32, kv_heads=8, d=128, rot=128, interleaved=False,
             scaling="yarn", factor=4.0, trained=8192, first=30011, backward=False),
        # The training batch of the benchmark (4 sequences of 2048, 16 heads), forward.
        dict(name="rope_train_2k", op="rope", batch=4, tokens=2048, heads=16, kv_heads=16, d=128, rot=128,
             interleaved=False, scaling="none", factor=1.0, trained=2048, first=0, backward=False),
        # Gradients of two long sequences with grouped heads; half of each head rotates, pairs
        # interleaved, positions compressed; written into the projection's own layout.
        dict(name="rope_grad_8k_part", op="rope", batch=2, tokens=8192, heads=32, kv_heads=8, d=128, rot=64,
             interleaved=True, scaling="linear", factor=2.0, trained=4096, first=0, backward=True),
        # One decoding step of 64 sequences: a token each, most pages partly filled.
        dict(name="append_step_b64", op="append", batch=64, heads=8, d=128, page=64, keys=8192, new=1, even=False),
        # Ragged pieces of prompts, small pages, 64-wide heads.
        dict(name="append_ragged_d64", op="append", batch=16, heads=4, d=64, page=16, keys=4000, new=300, even=False),
        # Two whole prompts of 8192 tokens.
        dict(name="append_prompt_8k", op="append", batch=2, heads=8, d=128, page=128, keys=8192, new=8192, even=True),
        # One short conversation, one token: nothing to hide the latency behind.
        dict(name="attend_one_1k", op="attend", batch=1, heads=32, kv_heads=8, d=128, page=16, keys=1000, new=1, even=True,
             causal=True),
        # The benchmark's decoding batch: 8 sequences of 8192 cached keys.
        dict(name="attend_step_b8_8k", op="attend", batch=8, heads=32, kv_heads=8, d=128, page=128, keys=8192, new=1,
             even=True, causal=True),
        # A busy server: 64 sequences of very different lengths up to 32768.
        dict(name="attend_step_ragged_32k", op="attend", batch=64, heads=32, kv_heads=8, d=128, page=64, keys=32768,
             new=1, even=False, causal=True),
        # Four drafted tokens verified at once, one K/V head shared by 32 query heads.
        dict(name="attend_draft_mqa", op="attend", batch=8, heads=32, kv_heads=1, d=128, page=32, keys=8191, new=4,
             even=True, causal=True),
        # Pieces of prompts (chunked prefill) after contexts of different lengths.
        dict(name="attend_chunk_512", op="attend", batch=4, heads=32, kv_heads=8, d=128, page=128, keys=16000, new=512,
             even=False, causal=True),
        # The second half of two long prompts.
        dict(name="attend_prompt_4k", op="attend", batch=2, heads=32, kv_heads=8, d=128, page=128, keys=8192, new=4096,
             even=True, causal=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend"])
    d = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "rope":
        d = rng.choice([64, 128, 192, 256])
        tokens = _log(rng, 1, 6000)
        batch = rng.choice([1, 2, 3]) if tokens < 2500 else 1
        return dict(op="rope", batch=batch, tokens=tokens, heads=kv_heads * min(group, 4), kv_heads=kv_heads, d=d,
                    rot=rng.choice([d, d // 2, d // 4 + 8]), interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]), factor=rng.choice([2.0, 3.5, 8.0]),
                    trained=rng.choice([2048, 4096, 8192]), first=_log(rng, 1, 400000), backward=rng.random() < 0.5)
    if op == "append":
        new = _log(rng, 1, 4000)
        return dict(op="append", batch=_log(rng, 1, max(2, min(48, 12000 // new))), heads=kv_heads, d=d, page=page,
                    keys=new + _log(rng, 1, 4000), new=new, even=rng.random() < 0.3)
    if rng.random() < 0.6:  # decoding, or a few drafted tokens
        new, keys = rng.choice([1, 1, 1, 2, 3, 5]), _log(rng, 8, 30000)
        batch = _log(rng, 1, max(1, min(48, 400000 // keys)))
    else:  # pieces of prompts
        new = _log(rng, 9, 2000)
        keys, batch = new + _log(rng, 1, 8000), rng.choice([1, 2, 3])
    return dict(op="attend", batch=batch, heads=kv_heads * group, kv_heads=kv_heads, d=d, page=page, keys=keys, new=new,
                even=rng.random() < 0.3, causal=rng.random() < 0.8)


def _lengths(case):
    """Each sequence's keys after the call, and how many of them are new."""
    b, keys, new = case["batch"], case["keys"], case["new"]
    if case["even"]:
        return [keys] * b, [new] * b
    rng = random.Random("%d %d %d %d" % (b, keys, new, case["page"]))
    total = [keys] + [rng.randint(max(1, keys // 64), keys) for _ in range(b - 1)]
    fresh = [new] + [rng.randint(1, new) for _ in range(b - 1)]
    return total, [min(n, t) for n, t in zip(fresh, total)]


def work(case):
    if case["op"] == "rope":
        rows = case["batch"] * case["tokens"] * (case["heads"] + case["kv_heads"])
        return {"bytes": rows * case["d"] * 4 + case["batch"] * case["tokens"] * 4 + case["rot"] * 4,
                "flops": rows * case["rot"] * 3}
    total, fresh = _lengths(case)
    if case["op"] == "append":
        rows, pages = sum(fresh) * case["heads"] * 2, sum(n // case["page"] + 1 for n in fresh)
        return {"bytes": rows * case["d"] * 3 + pages * case["heads"] * 8, "flops": rows * case["d"] * 2}
    cache = sum(2 * case["kv_heads"] * (t * case["d"] + 4 * -(-t // case["page"])) for t in total)
    seen = sum(n * t - (n * (n - 1) // 2 if case["causal"] else 0) for t, n in zip(total, fresh))
    return {"bytes": cache + sum(fresh) * case["heads"] * (case["d"] * 4 + 4), "flops": 4 * seen * case["heads"] * case["d"]}


# ------------------------------------------------------------------ inputs
def _inverse_frequencies(case):
    """Radians a position turns each pair by (64 bits), and the factor on the rotated part."""
    rot, base, s = case["rot"], 10000.0, case["factor"]
    j = torch.arange(0, rot, 2, dtype=torch.float64)
    if case["scaling"] == "ntk":
        base *= s ** (rot / max(rot - 2, 1))
    f = base ** (-j / rot)
    if case["scaling"] == "linear":
        return f / s, 1.0
    if case["scaling"] == "yarn":
        turns = case["trained"] * f / (2 * math.pi)          # turns over the trained length
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)    # 1: fast pairs, left alone; 0: slow ones, compressed
        return f * keep + f / s * (1 - keep), 0.1 * math.log(s) + 1.0
    return f, 1.0


def _quantise(x):
    """fp32 [..., rows, d] -> e4m3 codes (uint8) and one power-of-two scale per leading index."""
    amax = x.abs().amax((-2, -1))
    m, e = torch.frexp(amax)
    scale = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e - torch.where(m <= 0.875, 9, 8)), 0.0)
    safe = torch.where(scale > 0, scale, 1.0)
    return (x / safe[..., None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8), scale


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    d = case["d"]
    if case["op"] == "rope":
        B, N, Hq, Hk = case["batch"], case["tokens"], case["heads"], case["kv_heads"]
        rows = torch.randn((B, N, Hq + 2 * Hk, d), generator=gen, device=dev).to(torch.bfloat16)  # a fused projection's output
        first = torch.randint(0, 64, (B, 1), generator=gen, device=dev) + case["first"]
        st = dict(op="rope", positions=(first + torch.arange(N, device=dev)).to(torch.int32).contiguous(),
                  interleaved=case["interleaved"], rot=case["rot"], backward=case["backward"])
        f, st["mscale"] = _inverse_frequencies(case)
        st["inv_freq"] = f.to(dev)
        split = (rows[:, :, :Hq].transpose(1, 2), rows[:, :, Hq:Hq + Hk].transpose(1, 2))
        if case["backward"]:  # gradients from the attention, [B, H, N, d]; out into the projection's layout
            st["q"], st["k"] = (t.contiguous() for t in split)
            st["q_out"], st["k_out"] = split
        else:
            st["q"], st["k"] = split
            st["q_out"], st["k_out"] = (torch.empty((B, h, N, d), dtype=torch.bfloat16, device=dev) for h in (Hq, Hk))
        return st
    total, fresh = _lengths(case)
    B, P = case["batch"], case["page"]
    Hk = case["heads"] if case["op"] == "append" else case["kv_heads"]
    need = [-(-t // P) for t in total]
    pages, width = sum(need) + 3, max(need) + 1
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    st = dict(op=case["op"], table=table, page=P, new=case["new"], new_max=max(fresh),
              kv_lens=torch.tensor(total, dtype=torch.int32, device=dev),
              cu=torch.tensor([sum(fresh[:b]) for b in range(B + 1)], dtype=torch.int32, device=dev))
    for name in ("k", "v"):  # what earlier calls left in the cache: unit normals with a gain for each page and head
        codes = torch.empty((pages, Hk, P, d), dtype=torch.uint8, device=dev)
        scale = torch.empty((pages, Hk), device=dev)
        for p in range(0, pages, 4096):
            x = torch.randn((min(4096, pages - p), Hk, P, d), generator=gen, device=dev)
            x *= torch.exp2(torch.randn(x.shape[:2], generator=gen, device=dev) * 0.5)[..., None, None]
            codes[p:p + 4096], scale[p:p + 4096] = _quantise(x)
        st[name + "_cache"], st[name + "_scale"] = codes, scale
    T = sum(fresh)
    if case["op"] == "append":
        rows = torch.randn((T, 2 * Hk, d), generator=gen, device=dev).to(torch.bfloat16)
        st["k"], st["v"] = rows[:, :Hk].transpose(0, 1), rows[:, Hk:].transpose(0, 1)
        return st
    Hq = case["heads"]
    st["q"] = torch.randn((Hq, T, d), generator=gen, device=dev).to(torch.bfloat16)
    st["o"] = torch.empty_like(st["q"])
    st["lse"] = torch.empty((Hq, T), device=dev)
    st.update(causal=case["causal"], scale=d ** -0.5, keys=max(total), workspace=None)
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    if own:
        return _own(st)
    return {"rope": _rope, "append": _append, "attend": _attend}[st["op"]](st)


def _own(st):
    import attention_attn_fwd_09_gb300 as A
    if st["op"] == "rope":
        call = A.attn_rope_bwd if st["backward"] else A.attn_rope
        return call(st["q"], st["k"], st["inv_freq"], st["positions"], interleaved=st["interleaved"],
                    mscale=st["mscale"], q_out=st["q_out"], k_out=st["k_out"])
    if st["op"] == "append":
        A.attn_kv_append_fp8(st["k"], st["v"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"], st["table"],
                             st["cu"], st["kv_lens"])
        return _cache(st)
    if st["workspace"] is None:  # a server keeps it from call to call
        n = A.attn_fwd_kv_fp8_workspace_size(st["kv_lens"].numel(), st["q"].shape[0], st["k_cache"].shape[1],
                                             st["q"].shape[1], st["new_max"], st["q"].shape[2])
        st["workspace"] = torch.empty((max(n, 16),), dtype=torch.uint8, device=st["q"].device)
    return A.attn_fwd_kv_fp8(st["q"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"], st["table"], st["cu"],
                             st["kv_lens"], st["new_max"], causal=st["causal"], scale=st["scale"], o=st["o"],
                             lse=st["lse"], workspace=st["workspace"])


def _cache(st):
    """The cache as the values its codes stand for (before their scales), and the scales."""
    return {"k": st["k_cache"].view(torch.float8_e4m3fn), "v": st["v_cache"].view(torch.float8_e4m3fn),
            "k_scale": st["k_scale"], "v_scale": st["v_scale"]}


def _turn(x, cos, sin, rot, interleaved):
    x = x.float()
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    y, z = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((y, z), -1).flatten(-2) if interleaved else torch.cat((y, z), -1)
    return torch.cat((r, x[..., rot:]), -1).to(torch.bfloat16)


def _rope(st):
    # Angles in 64 bits: a far position times a frequency near 1 keeps no fraction in 32.
    angle = st["positions"].double()[:, None, :, None] * st["inv_freq"]
    cos, sin = (angle.cos() * st["mscale"]).float(), (angle.sin() * st["mscale"]).float()
    if st["backward"]:
        sin = -sin  # the transposed rotation
    return tuple(_turn(st[n], cos, sin, st["rot"], st["interleaved"]) for n in ("q", "k"))


def _append_one(x, codes, scale, st, seq, pos, start):
    P = st["page"]
    xf = x.float().transpose(0, 1)                                          # [T, H, d]
    page = st["table"].long()[seq, pos // P]
    finite = torch.where(torch.isfinite(xf), xf.abs(), 0.0).amax(-1)        # [T, H]
    m, e = torch.frexp(torch.zeros_like(scale).index_reduce_(0, page, finite, "amax"))
    fresh = torch.where(m > 0, torch.ldexp(torch.ones_like(m), e - torch.where(m <= 0.875, 9, 8)), 0.0)
    # Only the first page a sequence writes to can hold earlier rows: their scale may only grow,
    # and the rows are rounded again when it does.
    head = st["table"].long().gather(1, (start // P)[:, None])[:, 0]
    slot = start % P
    was = torch.where((slot > 0)[:, None], scale[head], 0.0)
    wanted = fresh.index_reduce(0, head, was, "amax")                       # every page's scale, were it written to
    scale[page] = wanted[page]
    safe = torch.where(wanted > 0, wanted, 1.0)
    old = codes[head].view(torch.float8_e4m3fn).float() * was[..., None, None]
    again = (old / safe[head][..., None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    earlier = torch.arange(P, device=x.device) < slot[:, None]
    codes[head] = torch.where(earlier[:, None, :, None], again, codes[head])
    y = (xf / safe[page][..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    codes[page, :, pos % P] = y


def _append(st):
    T = st["k"].shape[1]
    tok = torch.arange(T, device=st["cu"].device)
    cu = st["cu"].long()
    seq = torch.searchsorted(cu[1:], tok, right=True)
    start = st["kv_lens"].long() - (cu[1:] - cu[:-1])
    pos = start[seq] + tok - cu[seq]
    _append_one(st["k"], st["k_cache"], st["k_scale"], st, seq, pos, start)
    _append_one(st["v"], st["v_cache"], st["v_scale"], st, seq, pos, start)
    return _cache(st)


def _gather(codes, scale, table, blocks):
    pages = table[:, :blocks].long().clamp(min=0)
    x = codes[pages].view(torch.float8_e4m3fn).float().mul_(scale[pages][..., None, None])   # [B, blocks, H, P, d]
    return x.transpose(1, 2).flatten(2, 3)                                                    # [B, H, keys, d]


def _attend(st):
    q, P = st["q"], st["page"]
    Hq, T, d = q.shape
    blocks = -(-st["keys"] // P)
    Hk = st["k_cache"].shape[1]
    g, n = Hq // Hk, st["new_max"]
    cu, lens = st["cu"].long(), st["kv_lens"].long()
    B = lens.numel()
    tok = torch.arange(T, device=q.device)
    seq = torch.searchsorted(cu[1:], tok, right=True)
    row = tok - cu[seq]
    padded = torch.zeros((B, n, Hq, d), device=q.device)
    padded[seq, row] = q.float().transpose(0, 1)
    padded = padded.view(B, n, Hk, g, d).permute(0, 2, 3, 1, 4).reshape(B, Hk, g * n, d)
    key = torch.arange(blocks * P, device=q.device)
    last = lens[:, None].expand(B, n) - 1
    if st["causal"]:
        last = (lens - (cu[1:] - cu[:-1]))[:, None] + torch.arange(n, device=q.device)
        last = torch.minimum(last, lens[:, None] - 1)
    hidden = (key > last[..., None])[:, None, None].expand(B, 1, g, n, key.numel()).reshape(B, 1, g * n, key.numel())
    s = padded @ _gather(st["k_cache"], st["k_scale"], st["table"], blocks).transpose(2, 3)
    s = s.mul_(st["scale"]).masked_fill_(hidden, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = _gather(st["v_cache"], st["v_scale"], st["table"], blocks)
    v = v.masked_fill_((key >= lens[:, None])[:, None, :, None], 0.0)      # what lies behind the last key is not data
    o = ((p @ v) / total).view(B, Hk, g, n, d).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, d)
    lse = (top + total.log())[..., 0].view(B, Hk, g, n).permute(0, 3, 1, 2).reshape(B, n, Hq)
    return o[seq, row].transpose(0, 1).contiguous().to(torch.bfloat16), lse[seq, row].transpose(0, 1).contiguous()


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_rope(case, st):
    turn = torch.polar(torch.full((1,), st["mscale"], dtype=torch.float64, device=st["q"].device),
                       st["positions"].double()[..., None] * st["inv_freq"])[:, None]
    turn = turn.conj() if case["backward"] else turn
    out = []
    for x in (st["q"], st["k"]):
        y, r = x.double().contiguous(), case["rot"]
        if case["interleaved"]:
            z = torch.view_as_complex(y[..., :r].unflatten(-1, (r // 2, 2)).contiguous()) * turn
            y[..., :r] = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(y[..., :r // 2], y[..., r // 2:r]) * turn
            y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
        out.append(y)
    return tuple(out)


def _exact_append(case, st):
    total, fresh = _lengths(case)
    P, out = case["page"], {}
    grid = torch.arange(127, dtype=torch.uint8, device=st["k"].device).view(torch.float8_e4m3fn).double()
    for name in ("k", "v"):
        codes = st[name + "_cache"].view(torch.float8_e4m3fn).double()
        scale, x, at = st[name + "_scale"].double(), st[name].double(), 0

        def nearest(y):  # the e4m3 value next to y; halfway, the one with the even code
            a = y.abs().clamp(max=E4M3_MAX)
            up = torch.searchsorted(grid, a.contiguous()).clamp(max=126)
            lo = (up - 1).clamp(min=0)
            near, far = grid[up] - a, a - grid[lo]
            pick = torch.where((near < far) | ((near == far) & (up % 2 == 0)), up, lo)
            return torch.copysign(grid[pick], y)

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
            at += n
        out[name], out[name + "_scale"] = codes, scale
    return out


def _exact_attend(case, st):
    total, fresh = _lengths(case)
    Hk, g, P = case["kv_heads"], case["heads"] // case["kv_heads"], case["page"]
    o, lse, at = torch.empty_like(st["q"], dtype=torch.float64), torch.empty_like(st["lse"], dtype=torch.float64), 0
    for b, (t, n) in enumerate(zip(total, fresh)):
        pages = st["table"][b, :-(-t // P)].long()
        for h in range(Hk):
            k, v = ((st[c + "_cache"][pages, h].view(torch.float8_e4m3fn).double()
                     * st[c + "_scale"][pages, h].double()[:, None, None]).flatten(0, 1)[:t] for c in ("k", "v"))
            for i in range(0, n, 1024):
                m = min(1024, n - i)
                s = st["q"][h * g:(h + 1) * g, at + i:at + i + m].double() @ k.T * st["scale"]
                if case["causal"]:
                    here = t - n + i + torch.arange(m, device=s.device)
                    s = s.masked_fill(torch.arange(t, device=s.device) > here[:, None], -math.inf)
                lse[h * g:(h + 1) * g, at + i:at + i + m] = torch.logsumexp(s, -1)
                o[h * g:(h + 1) * g, at + i:at + i + m] = torch.softmax(s, -1) @ v
        at += n
    return o, lse


def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "attend": _exact_attend}[case["op"]](case, st)
