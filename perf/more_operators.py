"""The 8-bit paged cache and the attention over the paged cache, as they are measured.

Five operators:

  append8  new tokens' K and V quantised into 8-bit pages (a scale for each
           token and head) with the means of the touched blocks, and read back;
  read     cached tokens' K and V out of their pages as bf16 rows;
  decode8  single tokens that select blocks by their means and attend to
           their keys in 8-bit pages;
  window   new tokens (one each, or a prompt's chunk) attending to the last W
           keys and to the first few (sinks), over bf16 or 8-bit pages;
  tree     a tree of drafted tokens for each sequence attending to the whole
           prefix and to their ancestors, over bf16 or 8-bit pages.

``run`` computes them in plain torch operations, or through the library's
entry points where ``own`` is true; ``exact`` gives their values in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding step into 8-bit pages: a token for each of 64 sequences; latency counts
        dict(name="append8_decode", op="append8", seqs=64, tokens=64, heads=8, d=128, page=64, past=16384,
             ragged=False),
        # prefill of new prompts of odd lengths behind cached prefixes, read back as they will be attended to
        dict(name="append8_prefill", op="append8", seqs=7, tokens=65521, heads=8, d=128, page=64, past=3001,
             ragged=True),
        # short ragged prefixes out of small bf16 pages
        dict(name="read_short", op="read", seqs=5, tokens=1237, heads=4, d=64, page=16, past=300, ragged=True,
             bits=16, heads_first=False),
        # a long 8-bit prefix in the [heads][n][d] layout that the sparse forward takes
        dict(name="read_n131072", op="read", seqs=1, tokens=131072, heads=8, d=128, page=64, past=0, ragged=False,
             bits=8, heads_first=True),
        # one sequence at 131072 tokens, top-32, 8-bit pages (interactive use)
        dict(name="decode8_n131072", op="decode8", seqs=1, per_seq=1, q_heads=64, heads=8, d=128, page=64,
             longest=131072, topk=32, share=False, local=True),
        # serving batch over 8-bit pages, grouped heads share one selection, ragged lengths to 32768
        dict(name="decode8_shared", op="decode8", seqs=48, per_seq=1, q_heads=64, heads=8, d=128, page=64,
             longest=32768, topk=32, share=True, local=True),
        # one short sequence, ungrouped heads, a small window over 8-bit pages: latency
        dict(name="window_n1000", op="window", seqs=1, tokens=1, ragged=False, q_heads=2, heads=2, d=64, page=64,
             longest=1000, window=256, sinks=4, bits=8),
        # serving batch: the last 4096 keys and four sinks of long sequences
        dict(name="window_decode", op="window", seqs=64, tokens=64, ragged=False, q_heads=32, heads=8, d=128, page=64,
             longest=32768, window=4096, sinks=4, bits=16),
        # prompts in chunks behind cached prefixes, ragged, each token with its own window
        dict(name="window_prompt", op="window", seqs=3, tokens=8191, ragged=True, q_heads=32, heads=8, d=128, page=64,
             longest=8192, window=4096, sinks=4, bits=16),
        # one sequence's tree of 16 drafted tokens behind 8192 keys: latency
        dict(name="tree_n8192", op="tree", seqs=1, per_seq=16, q_heads=32, heads=8, d=128, page=64, longest=8192,
             window=0, sinks=0, bits=16),
        # serving batch: trees of 64 drafted tokens behind ragged prefixes to 32768 keys
        dict(name="tree_batch", op="tree", seqs=16, per_seq=64, q_heads=32, heads=8, d=128, page=64, longest=32768,
             window=0, sinks=0, bits=16),
        # smaller trees of an odd size over small 8-bit pages, grouped by six
        dict(name="tree_batch8", op="tree", seqs=24, per_seq=13, q_heads=24, heads=4, d=64, page=32, longest=32768,
             window=0, sinks=0, bits=8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["append8", "read", "decode8", "window", "window", "tree", "tree"])
    d, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    if op in ("append8", "read"):
        seqs = _log_int(rng, 1, 128)
        ragged = rng.random() < 0.6
        tokens = _log_int(rng, seqs, 65536) if ragged else seqs * rng.choice([1, 1, 2, 5])
        case = dict(op=op, seqs=seqs, tokens=tokens, heads=rng.randint(1, 8), d=d, page=page,
                    past=_log_int(rng, 1, 16384), ragged=ragged)
        if op == "read":
            case.update(bits=rng.choice([8, 16]), heads_first=rng.random() < 0.5)
        return case
    heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 7, 8, 16])
    if op == "decode8":
        seqs, per_seq, share = _log_int(rng, 1, 48), rng.choice([1, 1, 2, 5]), rng.random() < 0.4
        longest = _log_int(rng, rng.choice([1, 1000]), min(131072, 48 * 32768 // seqs))
        lists = seqs * per_seq * heads * (1 if share else group)
        most = max(1, min(32, 48 * 8 * 32 * 64 * 128 // (lists * page * d)))
        return dict(op=op, seqs=seqs, per_seq=per_seq, q_heads=heads * group, heads=heads, d=d, page=page,
                    longest=longest, topk=rng.randint(1, most), share=share, local=rng.random() < 0.7)
    bits = rng.choice([8, 16])
    window = rng.choice([0, _log_int(rng, 1, 8192)]) if op == "tree" else _log_int(rng, 1, 8192)
    sinks = rng.choice([0, 1, 4, 130]) if window else 0
    seqs = _log_int(rng, 1, 64)
    # keys of all sequences, and pairs of query rows and keys, below those of the largest listed cases
    longest = _log_int(rng, rng.choice([1, 500]), min(65536, 16 * 32768 * 8 // (seqs * heads)))
    if op == "tree":
        room = 16 * 64 * 32 * 32768 // (seqs * heads * group * longest)
        return dict(op=op, seqs=seqs, per_seq=rng.randint(1, max(1, min(64, room))), q_heads=heads * group,
                    heads=heads, d=d, page=page, longest=longest, window=window, sinks=sinks, bits=bits)
    ragged = rng.random() < 0.5
    room = 8191 * 32 * 4096 // (heads * group * min(window + sinks, longest + 1))
    tokens = _log_int(rng, seqs, max(seqs, min(8192, room))) if ragged else seqs
    return dict(op=op, seqs=seqs, tokens=tokens, ragged=ragged, q_heads=heads * group, heads=heads, d=d, page=page,
                longest=longest, window=window, sinks=sinks, bits=bits)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed * 2654435761 % (1 << 31) + 29)


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _cut(g, total, parts):
    """`total` cut at random into `parts` numbers of at least one."""
    if parts == 1:
        return torch.tensor([total], device=DEV)
    at = torch.randperm(total - 1, generator=g, device=DEV)[:parts - 1].sort().values + 1
    ends = torch.cat([at, torch.tensor([total], device=DEV)])
    return torch.diff(ends, prepend=torch.zeros(1, dtype=ends.dtype, device=DEV))


def _tables(g, lens, page, first=None, pool=None):
    """(table, pool): random pages for blocks [first, ceil(lens / page)) of each sequence."""
    per = (lens + page - 1) // page
    first = torch.zeros_like(per) if first is None else first
    held = per - first
    base = torch.cumsum(held, 0) - held
    pool = int(held.sum()) + 1 if pool is None else pool
    ids = torch.randperm(pool - 1, generator=g, device=DEV) if pool > 1 else torch.zeros(1, dtype=torch.long, device=DEV)
    col = torch.arange(max(1, int(per.max())), device=DEV)[None]
    inside = (col >= first[:, None]) & (col < per[:, None])
    at = (base[:, None] + col - first[:, None]).clamp(0, max(0, pool - 2))
    return torch.where(inside, ids[at], pool - 1).int().contiguous(), pool


def _pages8(g, pool, heads, page, d):
    """8-bit pages as appends leave them: codes to +-127, a scale for each row."""
    codes = torch.empty(pool, heads, page, d, dtype=torch.int8, device=DEV)
    for a in range(0, pool, 4096):
        x = _randn(g, min(4096, pool - a), heads, page, d)
        codes[a:a + 4096] = (x * 44.0).clamp_(-127, 127).round_()
    scale = 0.015 + 0.02 * torch.rand(pool, heads, page, generator=g, device=DEV)
    return codes, scale


def _pages(st, g, pool, heads, page, d, bits):
    if bits == 8:
        st["k"], st["ks"] = _pages8(g, pool, heads, page, d)
        st["v"], st["vs"] = _pages8(g, pool, heads, page, d)
    else:
        st["k"] = _randn(g, pool, heads, page, d)
        st["v"] = _randn(g, pool, heads, page, d)


def _starts_and_new(case, g):
    s, t = case["seqs"], case["tokens"]
    new = _cut(g, t, s) if case["ragged"] else torch.full((s,), t // s, device=DEV)
    return new, torch.cat([torch.zeros(1, dtype=torch.int32, device=DEV), new.cumsum(0).int()])


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    op, heads, d, page, s = case["op"], case["heads"], case["d"], case["page"], case["seqs"]
    bits = 8 if op in ("append8", "decode8") else case["bits"]
    if op in ("append8", "read"):
        start = torch.randint(0, case["past"] + 1, (s,), generator=g, device=DEV)
        new, st["cu"] = _starts_and_new(case, g)
        st["start"] = start.int()
        # only the pages of the tokens in question are there, at most as many as the pool has
        st["table"], pool = _tables(g, start + new, page, start // page, case["tokens"] // page + 2 * s + 1)
        _pages(st, g, pool, heads, page, d, bits)
        if op == "append8":
            qkv = _randn(g, case["tokens"], 2 * heads, d)
            st["new_k"], st["new_v"] = qkv[:, :heads], qkv[:, heads:]
    elif op == "decode8":
        lens = torch.randint(max(1, case["longest"] // 8), case["longest"] + 1, (s,), generator=g, device=DEV)
        lens[0] = case["longest"]
        st["table"], pool = _tables(g, lens, page)
        _pages(st, g, pool, heads, page, d, 8)
        t = s * case["per_seq"]
        st["q"] = _randn(g, t, case["q_heads"], d)
        back = torch.arange(case["per_seq"] - 1, -1, -1, device=DEV)
        st["lens"] = (lens[:, None] - back[None]).clamp(min=0).reshape(-1).int().contiguous()
        st["seq"] = torch.arange(s, device=DEV).repeat_interleave(case["per_seq"]).int()
        kbar = torch.empty(pool, heads, d, device=DEV)
        for a in range(0, pool, 4096):
            kbar[a:a + 4096] = (st["k"][a:a + 4096].float() * st["ks"][a:a + 4096, ..., None]).mean(2)
        st["kbar"] = kbar
    else:
        start = torch.randint(case["longest"] // 8, case["longest"] + 1, (s,), generator=g, device=DEV)
        start[0] = case["longest"]
        if op == "tree":
            new = torch.full((s,), case["per_seq"], device=DEV)
            r, masks = random.Random(seed), []
            for _ in range(s):
                tree = []
                for i in range(case["per_seq"]):
                    parent = r.randint(max(-1, i - 8), i - 1)
                    tree.append((tree[parent] if parent >= 0 else 0) | 1 << i)
                masks += [m - (1 << 64) if m >> 63 else m for m in tree]
            st["tree"] = torch.tensor(masks, dtype=torch.int64, device=DEV)
            st["cu"] = torch.cat([torch.zeros(1, dtype=torch.int32, device=DEV), new.cumsum(0).int()])
        else:
            new, st["cu"] = _starts_and_new(case, g)
        st["start"] = start.int()
        st["table"], pool = _tables(g, start + new, page)
        _pages(st, g, pool, heads, page, d, bits)
        st["q"] = _randn(g, int(new.sum()), case["q_heads"], d)
        # a serving program holds these on the host too
        st["start_host"], st["cu_host"] = st["start"].tolist(), st["cu"].tolist()
    if "kbar" not in st:
        st["kbar"] = torch.zeros(pool, heads, d, device=DEV)
    if own:
        from content_dependent_block_gb300 import bsa
        st["cache"] = bsa.PagedCache8(st["k"], st["v"], st["ks"], st["vs"], st["kbar"]) if bits == 8 else \
            bsa.PagedCache(st["k"], st["v"], st["kbar"])
    return st


# ------------------------------------------------------------------ passes
def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    if case["op"] in ("window", "tree"):
        return _plain_attention(case, state)
    return {"append8": _plain_append8, "read": _plain_read, "decode8": _plain_decode8}[case["op"]](case, state)


def _run_own(case, st):
    from content_dependent_block_gb300 import bsa
    cache, op = st["cache"], case["op"]
    if op in ("append8", "read"):
        cu = st["cu"] if case["ragged"] else None
        if op == "append8":
            bsa.cache_append(cache, st["new_k"], st["new_v"], st["table"], st["start"], cu_tokens=cu)
        k, v = bsa.cache_read(cache, st["table"], st["start"], case["tokens"], cu_tokens=cu,
                              heads_first=op == "read" and case["heads_first"])
        return (k, v, cache.kbar) if op == "append8" else (k, v)
    if op == "decode8":
        return bsa.paged_decode(cache, st["q"], st["table"], st["lens"], case["topk"],
                                token_seq=st["seq"] if case["per_seq"] > 1 else None,
                                local_block=case["local"], share_group=case["share"])
    cu = st["cu"] if op == "window" and case["ragged"] else None
    return bsa.paged_attention(cache, st["q"], st["table"], st["start"], cu_tokens=cu, tree=st.get("tree"),
                               window=case["window"], sinks=case["sinks"])


def _where(case, st):
    """Page and slot of every token in question."""
    page, cu = case["page"], st["cu"].long()
    tok = torch.arange(case["tokens"], device=DEV)
    seq = torch.searchsorted(cu, tok, right=True) - 1
    pos = st["start"].long()[seq] + tok - cu[seq]
    return seq, tok, st["table"][seq, pos // page].long(), pos % page


def _plain_quantise(x):
    x = x.float()
    a = x.abs().amax(-1, keepdim=True)
    codes = torch.where(a > 0, torch.round(x * 127.0 / a), 0.0)
    return codes.to(torch.int8), (a / 127.0).squeeze(-1)


def _plain_append8(case, st):
    page = case["page"]
    seq, tok, where, slot = _where(case, st)
    for pages, scales, new in (("k", "ks", "new_k"), ("v", "vs", "new_v")):
        st[pages][where, :, slot], st[scales][where, :, slot] = _plain_quantise(st[new])
    # one token for each touched page: the last of it that is there
    ends = (slot == page - 1) | (tok == st["cu"].long()[seq + 1] - 1)
    pages, filled = where[ends], slot[ends] + 1
    rows = torch.arange(page, device=DEV)[None, None, :, None] < filled[:, None, None, None]
    keys = st["k"][pages].float() * st["ks"][pages][..., None]
    st["kbar"][pages] = torch.where(rows, keys, 0.0).sum(2) / filled[:, None, None].float()
    k, v = (st[p][where, :, slot].float() * st[c][where, :, slot][..., None] for p, c in (("k", "ks"), ("v", "vs")))
    return k.to(torch.bfloat16), v.to(torch.bfloat16), st["kbar"]


def _plain_read(case, st):
    _, _, where, slot = _where(case, st)
    out = []
    for p, c in (("k", "ks"), ("v", "vs")):
        x = st[p][where, :, slot]
        if case["bits"] == 8:
            x = (x.float() * st[c][where, :, slot][..., None]).to(torch.bfloat16)
        out.append(x.transpose(0, 1).contiguous() if case["heads_first"] else x)
    return tuple(out)


def _plain_decode8(case, st):
    """Scores in 64 bits (which block is the k-th best must not hang on rounding), the softmax in 32."""
    hq, hkv, d, page, topk = case["q_heads"], case["heads"], case["d"], case["page"], case["topk"]
    group = hq // hkv
    t, width = st["q"].shape[0], st["table"].shape[1]
    rows = 1 if case["share"] else group
    out = torch.empty(t, hq, d, dtype=torch.bfloat16, device=DEV)
    idx = torch.full((t, hkv * rows, topk), -1, dtype=torch.int32, device=DEV)
    step = max(1, (1 << 30) // max(hkv * width * d * 8, hq * min(topk, width) * page * d * 8))
    head = torch.arange(hkv, device=DEV)[None, :, None, None]
    block = torch.arange(width, device=DEV)
    for a in range(0, t, step):
        q, lens = st["q"][a:a + step], st["lens"][a:a + step].long()
        c = q.shape[0]
        table = st["table"][st["seq"][a:a + step].long()].long()
        nb = (lens + page - 1) // page
        means = st["kbar"][table].double()                                 # [c, width, hkv, d]
        qs = q.view(c, hkv, group, d).double()
        if case["share"]:
            qs = qs.sum(2, keepdim=True)
        score = torch.einsum("chgd,cbhd->chgb", qs, means)
        score = torch.where((block[None] < nb[:, None])[:, None, None], score, -math.inf)
        if case["local"]:
            score = torch.where((block[None] == nb[:, None] - 1)[:, None, None], math.inf, score)
        kk = min(topk, width)
        best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :kk]
        chosen = torch.arange(kk, device=DEV) < nb.clamp(max=kk)[:, None, None, None]
        best = torch.where(chosen, best, width).sort(-1).values
        chosen = best < width
        idx[a:a + step, :, :kk] = torch.where(chosen, best, -1).view(c, hkv * rows, kk).int()
        best = best.clamp(max=width - 1)
        pages = torch.gather(table[:, None, None].expand(c, hkv, rows, width), 3, best)
        key = best[..., None] * page + torch.arange(page, device=DEV)
        admit = (chosen[..., None] & (key < lens[:, None, None, None, None]))     # [c, hkv, rows, kk, page]
        kk_ = (st["k"][pages, head].float() * st["ks"][pages, head][..., None]).flatten(3, 4)
        vv = (st["v"][pages, head].float() * st["vs"][pages, head][..., None]).flatten(3, 4)
        admit = admit.flatten(3, 4)[:, :, :, None]
        qq = q.view(c, hkv, rows, group // rows, d).float()
        s = torch.einsum("chrgd,chrjd->chrgj", qq, kk_) / math.sqrt(d)
        s = torch.where(admit, s, -math.inf)
        m = s.amax(-1, keepdim=True).clamp(min=-1e30)
        p = torch.exp(s - m)
        o = torch.einsum("chrgj,chrjd->chrgd", p, vv) / p.sum(-1, keepdim=True).clamp(min=1e-30)
        out[a:a + step] = o.reshape(c, hq, d).to(torch.bfloat16)
    return out, idx


def _plain_attention(case, st):
    """Sequence by sequence: the keys that some new token may see, the mask, the softmax in 32 bits."""
    hq, hkv, d, page = case["q_heads"], case["heads"], case["d"], case["page"]
    group, window, sinks = hq // hkv, case["window"], case["sinks"]
    out = torch.empty(st["q"].shape, dtype=torch.bfloat16, device=DEV)
    bit = torch.arange(64, device=DEV)
    for s in range(case["seqs"]):
        start, lo, hi = st["start_host"][s], st["cu_host"][s], st["cu_host"][s + 1]
        n = hi - lo
        if "tree" in st:
            sees = (st["tree"][lo:hi, None] >> bit[None, :n] & 1).bool()          # [n, n]
            depth = (sees & ~torch.eye(n, dtype=torch.bool, device=DEV)).sum(1)
        else:
            sees, depth = None, torch.arange(n, device=DEV)
        place = torch.cat([torch.arange(start, device=DEV), start + depth])       # of every key
        for a in range(0, n, max(1, (1 << 28) // (hq * (start + n)))):
            b = min(n, a + max(1, (1 << 28) // (hq * (start + n))))
            end = start + (b if sees is None else n)
            first = max(0, start + (a if sees is None else 0) - window + 1) if window else 0
            keys = torch.arange(first, end, device=DEV)
            if min(sinks, first):
                keys = torch.cat([torch.arange(min(sinks, first), device=DEV), keys])
            pages, slot = st["table"][s, keys // page].long(), keys % page
            k, v = st["k"][pages, :, slot].float(), st["v"][pages, :, slot].float()   # [keys, hkv, d]
            if case["bits"] == 8:
                k = k * st["ks"][pages, :, slot][..., None]
                v = v * st["vs"][pages, :, slot][..., None]
            at = start + depth[a:b, None]
            seen = torch.where(keys[None] < start, True, keys[None] <= start + torch.arange(a, b, device=DEV)[:, None]) \
                if sees is None else torch.where(keys[None] < start, True, sees[a:b][:, (keys - start).clamp(min=0)])
            if window:
                seen = seen & ((place[keys][None] > at - window) | (place[keys][None] < sinks))
            q = st["q"][lo + a:lo + b].view(b - a, hkv, group, d).float()
            x = torch.einsum("thgd,jhd->htgj", q, k) / math.sqrt(d)
            x = torch.where(seen[None, :, None], x, -math.inf)
            m = x.amax(-1, keepdim=True).clamp(min=-1e30)
            p = torch.exp(x - m)
            o = torch.einsum("htgj,jhd->htgd", p, v) / p.sum(-1, keepdim=True).clamp(min=1e-30)
            out[lo + a:lo + b] = o.transpose(0, 1).reshape(b - a, hq, d).to(torch.bfloat16)
    return out


# ------------------------------------------------------------------ work
def work(case):
    op, heads, d, page, s = case["op"], case["heads"], case["d"], case["page"], case["seqs"]
    if op in ("append8", "read"):
        n = case["tokens"] * heads
        if op == "read":
            e = 2 * d + 8 if case["bits"] == 8 else 4 * d
            return dict(bytes=n * (e + 4 * d), flops=2 * n * d)
        touched = case["tokens"] / page + s
        # new rows in, codes and scales out and in again, values out, means
        return dict(bytes=n * (4 * d + 2 * (2 * d + 8) + 4 * d) + 4 * touched * heads * d, flops=8 * n * d)
    hq = case["q_heads"]
    group = hq // heads
    mean = case["longest"] * (9 / 16 if s > 1 else 1)
    if op == "decode8":
        topk = case["topk"]
        nb = max(1.0, mean / page)
        lists = (1 if case["share"] else group) * case["per_seq"]
        k = min(topk, nb)
        union = nb * (1 - (1 - k / nb) ** lists)
        keys = min(page, case["longest"])
        t = s * case["per_seq"]
        return dict(bytes=s * heads * (nb * d * 4 * (1 if nb > topk else 0) + union * keys * (2 * d + 8)) + 4 * t * hq * d,
                    flops=2 * t * hq * d * (nb / (group if case["share"] else 1) + 2 * k * keys))
    t = s * case["per_seq"] if op == "tree" else case["tokens"]
    window = case["window"]
    each = t / s
    own_keys = (each + 1) / 2 if op == "window" else min(each, 9)
    seen = min(mean + own_keys, window + case["sinks"]) if window else mean + own_keys
    union = min(mean + each, window + each + case["sinks"]) if window else mean + each
    return dict(bytes=s * union * heads * (2 * d + 8 if case["bits"] == 8 else 4 * d) + 4 * t * hq * d,
                flops=4 * t * hq * d * seen)


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"append8": _exact_append8, "read": _exact_read, "decode8": _exact_decode8,
            "window": _exact_attention, "tree": _exact_attention}[case["op"]](case, st)


def _values(st, name):
    """The pages' values in 64 bits."""
    x = st[name].double()
    return x * st[name + "s"].double().unsqueeze(-1) if st[name].dtype is torch.int8 else x


def _spans(case, st):
    """(sequence, first and last token, page, slots) of every run of tokens within one page."""
    cu, start, table, page = st["cu"].tolist(), st["start"].tolist(), st["table"].tolist(), case["page"]
    for s in range(case["seqs"]):
        at = cu[s]
        while at < cu[s + 1]:
            p = start[s] + at - cu[s]
            n = min(page - p % page, cu[s + 1] - at)
            yield at, at + n, table[s][p // page], p % page, p % page + n
            at += n


def _exact_append8(case, st):
    vals, news, kbar = {}, {}, st["kbar"].double()
    for name in ("k", "v"):
        x = st["new_" + name].double()
        top = x.abs().max(-1, keepdim=True).values
        step = top / 127
        # the nearest multiple of the step, ties to the even one
        ratio = torch.where(top > 0, 127 * x / top, torch.zeros_like(x))
        news[name] = torch.round(ratio) * step
        vals[name] = _values(st, name)
    for lo, hi, where, r0, r1 in _spans(case, st):
        for name in ("k", "v"):
            vals[name][where, :, r0:r1] = news[name][lo:hi].transpose(0, 1)
        kbar[where] = vals["k"][where, :, :r1].mean(1)
    return news["k"], news["v"], kbar


def _exact_read(case, st):
    out = []
    for name in ("k", "v"):
        x, y = _values(st, name), torch.empty(case["tokens"], case["heads"], case["d"], dtype=torch.float64, device=DEV)
        for lo, hi, where, r0, r1 in _spans(case, st):
            y[lo:hi] = x[where, :, r0:r1].permute(1, 0, 2)
        out.append(y.permute(1, 0, 2).contiguous() if case["heads_first"] else y)
    return tuple(out)


def _exact_decode8(case, st):
    hq, hkv, d, page, topk = case["q_heads"], case["heads"], case["d"], case["page"], case["topk"]
    t, group = st["q"].shape[0], hq // hkv
    rows = 1 if case["share"] else group
    if t * hkv > 2048:
        return None
    out = torch.zeros(t, hq, d, dtype=torch.float64, device=DEV)
    idx = torch.full((t, hkv * rows, topk), -1, dtype=torch.int64)
    lens, seq, table = st["lens"].tolist(), st["seq"].tolist(), st["table"].long()
    flat = {name: (st[name].view(-1, d), st[name + "s"].view(-1)) for name in ("k", "v")}
    for i in range(t):
        if lens[i] == 0:
            continue
        nb = -(-lens[i] // page)
        pages = table[seq[i], :nb]
        q = st["q"][i].double().view(hkv, group, d)
        means = st["kbar"][pages].double().permute(1, 2, 0)               # [hkv, d, nb]
        score = torch.matmul(q.sum(1, keepdim=True) if case["share"] else q, means)
        if case["local"]:
            score[..., nb - 1] = math.inf
        pick = torch.zeros(hkv, rows, nb, dtype=torch.bool, device=DEV)
        if nb <= topk:
            pick[:] = True
        else:
            for _ in range(topk):        # the first of the largest, k times
                b = score.max(-1, keepdim=True).values
                first = (score == b).to(torch.uint8).argmax(-1, keepdim=True)
                pick.scatter_(2, first, True)
                score.scatter_(2, first, -math.inf)
        hit = pick.nonzero()[:, 2].view(hkv, rows, -1)
        idx[i, :, :hit.shape[2]] = hit.view(hkv * rows, -1).cpu()
        pos = (hit[..., None] * page + torch.arange(page, device=DEV)).flatten(2)  # [hkv, rows, j]
        ok = pos < lens[i]
        phys = pages[hit].repeat_interleave(page, 2) * hkv + torch.arange(hkv, device=DEV)[:, None, None]
        at = phys * page + pos % page
        kk, vv = (torch.where(ok[..., None], flat[n][0][at].double() * flat[n][1][at].double()[..., None], 0.0)
                  for n in ("k", "v"))
        qq = q.view(hkv, rows, group // rows, d)
        s = torch.matmul(qq, kk.transpose(2, 3)) * d ** -0.5
        w = torch.softmax(s.masked_fill(~ok[:, :, None], -math.inf), -1)
        out[i] = torch.matmul(w, vv).view(hq, d)
    return out, idx.to(device=DEV, dtype=torch.int32)


def _exact_attention(case, st):
    """Head by head over all keys of a sequence, with the mask as the set of keys that each token sees."""
    hq, hkv, d, page = case["q_heads"], case["heads"], case["d"], case["page"]
    window, sinks = case["window"], case["sinks"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    masks = st["tree"].tolist() if "tree" in st else None
    total = sum((st["start_host"][s] + case.get("per_seq", 1)) * (st["cu_host"][s + 1] - st["cu_host"][s])
                for s in range(case["seqs"]))
    if total * hq * d > 1.5e12:
        return None
    for s in range(case["seqs"]):
        start, lo, hi = st["start_host"][s], st["cu_host"][s], st["cu_host"][s + 1]
        n, keys = hi - lo, start + hi - lo
        if masks is None:
            at = torch.arange(start, keys, device=DEV)
            gap = at[:, None] - torch.arange(keys, device=DEV)[None]
            hidden = gap < 0
            if window:
                hidden |= (gap >= window) & (torch.arange(keys, device=DEV)[None] >= sinks)
        else:
            kin = [[j for j in range(n) if masks[lo + i] >> j & 1] for i in range(n)]
            deep = [len([j for j in kin[i] if j != i]) for i in range(n)]
            rows = torch.ones(n, keys, dtype=torch.bool)
            for i in range(n):
                p = start + deep[i]
                rows[i, (max(0, p - window + 1) if window else 0):start] = False
                rows[i, :min(sinks, start) if window else 0] = False
                for j in kin[i]:
                    if not window or deep[i] - deep[j] < window or start + deep[j] < sinks:
                        rows[i, start + j] = False
            hidden = rows.to(DEV)
        pages = st["table"][s, :-(-keys // page)].long()
        for h in range(hkv):
            k, v = ((st[x][pages, h].double() * (st[x + "s"][pages, h].double()[..., None] if case["bits"] == 8 else 1.0))
                    .reshape(-1, d)[:keys] for x in ("k", "v"))
            for r in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                for a in range(0, n, 2048):
                    x = st["q"][lo + a:lo + min(n, a + 2048), r].double() @ k.T * d ** -0.5
                    w = torch.softmax(x.masked_fill(hidden[a:a + 2048], -math.inf), -1)
                    out[lo + a:lo + min(n, a + 2048), r] = w @ v
    return out
