"""The serving and position operators of the library, as they are measured.

Four operators over a paged key/value cache whose pages are the key blocks of
the two-stage selection (page = block of B tokens):

  rope     rotary positions on q or k, forward and backward;
  append   new tokens' K and V into their pages, and the means of the touched
           blocks;
  decode   single tokens: score every block mean, keep the best blocks,
           attend to their keys (heads grouped over the cache's heads);
  pages    page copies of a fork (copy on write) or of a compaction.

``run`` computes them in plain torch operations, or through the library's
entry points where ``own`` is true; ``exact`` gives their values in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding step of 64 sequences far into long contexts: 32 query heads rotated
        # by part-wise stretched frequencies; launch latency counts
        dict(name="rope_decode", op="rope", batch=1, heads=32, n=64, d=128, rot=128, dtype="bf16",
             interleaved=False, layout="bnhd", far=131072, scaling="parts", factor=4.0, backward=False),
        # q of a training or prefill pass as the projection leaves it ([n][heads][d]), brought
        # into the [heads][n][d] layout the sparse forward takes
        dict(name="rope_n32768", op="rope", batch=2, heads=32, n=32768, d=128, rot=128, dtype="bf16",
             interleaved=False, layout="bnhd", far=0, scaling="none", factor=1.0, backward=False),
        # gradient through partly rotated, interleaved heads in fp32, ragged length
        dict(name="rope_backward_n4100", op="rope", batch=3, heads=8, n=4100, d=64, rot=32, dtype="fp32",
             interleaved=True, layout="bhnd", far=0, scaling="linear", factor=2.0, backward=True),
        # one decoding step: a token for each of 64 sequences
        dict(name="append_decode", op="append", seqs=64, tokens=64, heads=8, d=128, page=64, past=16384,
             ragged=False),
        # prefill of new prompts of odd lengths behind cached prefixes
        dict(name="append_prefill", op="append", seqs=7, tokens=65521, heads=8, d=128, page=64, past=3001,
             ragged=True),
        # beams forked: the partly filled last page of each is copied
        dict(name="pages_fork", op="pages", pool=512, pairs=37, heads=8, d=128, page=64),
        # compaction of a pool after sequences ended
        dict(name="pages_compact", op="pages", pool=6144, pairs=2500, heads=8, d=64, page=64),
        # the smallest: one short sequence, ungrouped heads, top-4
        dict(name="decode_n1024", op="decode", seqs=1, per_seq=1, q_heads=2, heads=2, d=64, page=64,
             longest=1024, topk=4, share=False, local=True),
        # one sequence at 131072 tokens, top-32 (interactive use: latency over a long context)
        dict(name="decode_n131072", op="decode", seqs=1, per_seq=1, q_heads=64, heads=8, d=128, page=64,
             longest=131072, topk=32, share=False, local=True),
        # serving batch, every query head selects for itself, top-16, ragged lengths to 32768
        dict(name="decode_batch", op="decode", seqs=32, per_seq=1, q_heads=32, heads=8, d=64, page=64,
             longest=32768, topk=16, share=False, local=True),
        # a larger serving batch whose grouped heads share one selection
        dict(name="decode_shared", op="decode", seqs=96, per_seq=1, q_heads=64, heads=8, d=128, page=64,
             longest=32768, topk=32, share=True, local=True),
        # four drafted tokens for each of 13 sequences, small pages, no forced block
        dict(name="decode_draft", op="decode", seqs=13, per_seq=4, q_heads=24, heads=4, d=128, page=32,
             longest=8191, topk=24, share=False, local=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "pages", "decode", "decode"])
    if op == "rope":
        d = rng.choice([64, 128])
        heads, batch = rng.randint(1, 40), rng.randint(1, 3)
        n = _log_int(rng, 1, max(1, 2 * 32 * 32768 // (heads * batch)))
        return dict(op=op, batch=batch, heads=heads, n=min(n, 65536), d=d, rot=2 * rng.randint(4, d // 2),
                    dtype=rng.choice(["bf16", "fp32"] if heads * batch * n * d < 1 << 27 else ["bf16"]),
                    interleaved=rng.random() < 0.5,
                    layout=rng.choice(["bhnd", "bnhd"]), far=rng.choice([0, 4096, 1 << 20]),
                    scaling=rng.choice(["none", "linear", "base", "parts"]), factor=rng.choice([1.0, 2.0, 8.0]),
                    backward=rng.random() < 0.5)
    d, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    if op == "append":
        seqs = _log_int(rng, 1, 128)
        ragged = rng.random() < 0.6
        tokens = _log_int(rng, seqs, 65536) if ragged else seqs * rng.choice([1, 1, 2, 5])
        return dict(op=op, seqs=seqs, tokens=tokens, heads=rng.randint(1, 8), d=d, page=page,
                    past=_log_int(rng, 1, 16384), ragged=ragged)
    if op == "pages":
        pool = _log_int(rng, 32, 6144 * 64 // page * 64 // d)
        return dict(op=op, pool=pool, pairs=rng.randint(1, pool * 2 // 5), heads=rng.randint(1, 8), d=d, page=page)
    heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 7, 8, 16])
    seqs, per_seq, share = _log_int(rng, 1, 96), rng.choice([1, 1, 2, 5]), rng.random() < 0.4
    longest = _log_int(rng, rng.choice([1, 1000]), min(131072, 96 * 32768 // seqs))
    # no more blocks in all than the largest listed case selects
    lists = seqs * per_seq * heads * (1 if share else group)
    most = max(1, min(32, 96 * 8 * 32 * 64 * 128 // (lists * page * d)))
    return dict(op=op, seqs=seqs, per_seq=per_seq, q_heads=heads * group, heads=heads, d=d, page=page,
                longest=longest, topk=rng.randint(1, most), share=share, local=rng.random() < 0.7)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed * 2654435761 % (1 << 31) + 17)


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _dtype(case):
    return torch.bfloat16 if case.get("dtype", "bf16") == "bf16" else torch.float32


def _inv_freq(case):
    """The frequencies in 64 bits, on the device."""
    rot, s = case["rot"], case["factor"]
    theta = 10000.0
    if case["scaling"] == "base":
        theta = theta * s ** (rot / (rot - 2))
    f = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    if case["scaling"] == "linear":
        f = f / s
    if case["scaling"] == "parts":
        turns = 8192.0 * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        f = f * keep + (1 - keep) * f / s
    return f


def _attention_factor(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "parts" else 1.0


def _plan(case):
    """The rotation's plan, which a program makes once."""
    from content_dependent_block_gb300 import bsa
    return bsa.Rope(case["rot"], 10000.0, interleaved=case["interleaved"], scaling=case["scaling"],
                    factor=case["factor"], original=8192, low=1.0, high=32.0,
                    attention_factor=_attention_factor(case), device=DEV)


def _cut(g, total, parts):
    """`total` cut at random into `parts` numbers of at least one."""
    if parts == 1:
        return torch.tensor([total], device=DEV)
    at = torch.randperm(total - 1, generator=g, device=DEV)[:parts - 1].sort().values + 1
    ends = torch.cat([at, torch.tensor([total], device=DEV)])
    return torch.diff(ends, prepend=torch.zeros(1, dtype=ends.dtype, device=DEV))


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    if case["op"] == "rope":
        b, h, n, d = case["batch"], case["heads"], case["n"], case["d"]
        if case["layout"] == "bnhd":
            st["x"] = _randn(g, b, n, h, d, dtype=_dtype(case)).transpose(1, 2)
        else:
            st["x"] = _randn(g, b, h, n, d, dtype=_dtype(case))
        if case["far"]:
            st["positions"] = torch.randint(0, case["far"], (b, n), generator=g, device=DEV, dtype=torch.int32)
        else:
            st["positions"] = torch.arange(n, dtype=torch.int32, device=DEV).expand(b, n).contiguous()
        st["inv_freq"] = _inv_freq(case)
        if own:
            st["plan"] = _plan(case)
        return st

    heads, d, page = case["heads"], case["d"], case["page"]
    if case["op"] == "pages":
        pool = case["pool"]
        order = torch.randperm(pool, generator=g, device=DEV)
        n = case["pairs"]
        st["pairs"] = torch.stack([order[:n], order[n:2 * n]], 1).int().contiguous()
        st["k"] = _randn(g, pool, heads, page, d)
        st["v"] = _randn(g, pool, heads, page, d)
        st["kbar"] = _randn(g, pool, heads, d, dtype=torch.float32)
    elif case["op"] == "append":
        s, t = case["seqs"], case["tokens"]
        start = torch.randint(0, case["past"] + 1, (s,), generator=g, device=DEV)
        new = _cut(g, t, s) if case["ragged"] else torch.full((s,), t // s, device=DEV)
        st["start"] = start.int()
        st["cu"] = torch.cat([torch.zeros(1, dtype=torch.int32, device=DEV), new.cumsum(0).int()])
        per = (start + new + page - 1) // page
        width = int(per.max())
        # the pool holds the pages that are written; the cached prefix's pages before them are
        # not touched, and their table entries name pages of the pool all the same
        first = start // page
        touched = per - first
        base = torch.cumsum(touched, 0) - touched
        pool = t // page + 2 * s + 3          # at least as many as are touched
        ids = torch.randperm(pool, generator=g, device=DEV)
        col = torch.arange(width, device=DEV)[None]
        at = base[:, None] + col - first[:, None]
        inside = (col >= first[:, None]) & (col < per[:, None])
        st["table"] = torch.where(inside, ids[at.clamp(0, pool - 1)], ids[pool - 1]).int().contiguous()
        # k and v are slices of the projection's output, k rotated by then
        qkv = _randn(g, t, 2 * heads, d)
        st["new_k"], st["new_v"] = qkv[:, :heads], qkv[:, heads:]
        st["k"] = _randn(g, pool, heads, page, d)
        st["v"] = _randn(g, pool, heads, page, d)
        st["kbar"] = torch.zeros(pool, heads, d, device=DEV)
    else:
        s, per_seq, longest = case["seqs"], case["per_seq"], case["longest"]
        lens = torch.randint(max(1, longest // 8), longest + 1, (s,), generator=g, device=DEV)
        lens[0] = longest
        per = (lens + page - 1) // page
        width, pool = (longest + page - 1) // page, int(per.sum()) + 1
        base = torch.cumsum(per, 0) - per
        ids = torch.randperm(pool - 1, generator=g, device=DEV)
        col = torch.arange(width, device=DEV)[None]
        inside = col < per[:, None]
        st["table"] = torch.where(inside, ids[(base[:, None] + col).clamp(0, pool - 2)], -1).int().contiguous()
        # keys as the selection meets them: a centre for each block and noise around it
        k = _randn(g, pool, heads, page, d)
        k += 0.5 * _randn(g, pool, heads, 1, d)
        st["v"] = _randn(g, pool, heads, page, d)
        kbar = torch.empty(pool, heads, d, device=DEV)
        for a in range(0, pool, 4096):
            kbar[a:a + 4096] = k[a:a + 4096].float().mean(2)
        # the last page of each sequence is partly filled: its mean is that of the filled rows, and
        # the rows behind them hold whatever was there
        last = ids[base + per - 1]
        fill = lens - (per - 1) * page
        rows = torch.arange(page, device=DEV)[None, None, :, None] < fill[:, None, None, None]
        tail = k[last]
        kbar[last] = torch.where(rows, tail.float(), 0.0).sum(2) / fill[:, None, None]
        k[last] = torch.where(rows, tail, float("nan"))
        st["v"][last] = torch.where(rows, st["v"][last], float("inf"))
        st["k"], st["kbar"] = k, kbar
        t = s * per_seq
        st["q"] = _randn(g, t, case["q_heads"], d)
        back = torch.arange(per_seq - 1, -1, -1, device=DEV)
        st["lens"] = (lens[:, None] - back[None]).clamp(min=0).reshape(-1).int().contiguous()
        st["seq"] = torch.arange(s, device=DEV).repeat_interleave(per_seq).int()
    if own:
        from content_dependent_block_gb300 import bsa
        st["cache"] = bsa.PagedCache(st["k"], st["v"], st["kbar"])
    return st


# ------------------------------------------------------------------ passes
def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    if case["op"] == "rope":
        return _plain_rope(state["x"], state["positions"], state["inv_freq"], case)
    return {"append": _plain_append, "pages": _plain_pages, "decode": _plain_decode}[case["op"]](case, state)


def _run_own(case, st):
    from content_dependent_block_gb300 import bsa
    if case["op"] == "rope":
        call = bsa.rope_backward if case["backward"] else bsa.rope
        return call(st["x"], st["plan"], st["positions"])
    cache = st["cache"]
    if case["op"] == "append":
        bsa.cache_append(cache, st["new_k"], st["new_v"], st["table"], st["start"],
                         cu_tokens=st["cu"] if case["ragged"] else None)
        return cache.k, cache.v, cache.kbar
    if case["op"] == "pages":
        bsa.copy_pages(cache, st["pairs"])
        return cache.k, cache.v, cache.kbar
    return bsa.paged_decode(cache, st["q"], st["table"], st["lens"], case["topk"],
                            token_seq=st["seq"] if case["per_seq"] > 1 else None,
                            local_block=case["local"], share_group=case["share"])


def _plain_rope(x, positions, inv_freq, case):
    """x [b, h, n, d]; angles in 64 bits, the rotation in 32."""
    rot = case["rot"]
    angle = positions.double()[:, None, :, None] * inv_freq
    m = _attention_factor(case)
    cos, sin = (m * torch.cos(angle)).float(), (m * torch.sin(angle)).float()
    if case.get("backward"):
        sin = -sin
    if case["interleaved"]:
        a, b = x[..., 0:rot:2].float(), x[..., 1:rot:2].float()
    else:
        a, b = x[..., :rot // 2].float(), x[..., rot // 2:rot].float()
    ra, rb = a * cos - b * sin, b * cos + a * sin
    out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    if case["interleaved"]:
        out[..., 0:rot:2], out[..., 1:rot:2] = ra.to(x.dtype), rb.to(x.dtype)
    else:
        out[..., :rot // 2], out[..., rot // 2:rot] = ra.to(x.dtype), rb.to(x.dtype)
    out[..., rot:] = x[..., rot:]
    return out


def _plain_append(case, st):
    page, cu, start = case["page"], st["cu"], st["start"].long()
    t = case["tokens"]
    tok = torch.arange(t, device=DEV)
    seq = torch.searchsorted(cu.long(), tok, right=True) - 1
    pos = start[seq] + tok - cu.long()[seq]
    where, slot = st["table"][seq, pos // page].long(), pos % page
    st["k"][where, :, slot] = st["new_k"]
    st["v"][where, :, slot] = st["new_v"]
    # one token for each touched page: the last of it that is there
    ends = (slot == page - 1) | (tok == cu.long()[seq + 1] - 1)
    pages, filled = where[ends], slot[ends] + 1
    rows = torch.arange(page, device=DEV)[None, None, :, None] < filled[:, None, None, None]
    st["kbar"][pages] = torch.where(rows, st["k"][pages].float(), 0.0).sum(2) / filled[:, None, None].float()
    return st["k"], st["v"], st["kbar"]


def _plain_pages(case, st):
    src, dst = st["pairs"][:, 0].long(), st["pairs"][:, 1].long()
    k, v, kbar = st["k"], st["v"], st["kbar"]
    k[dst], v[dst], kbar[dst] = k[src], v[src], kbar[src]
    return k, v, kbar


def _plain_decode(case, st):
    """Scores in 64 bits (which block is the k-th best must not hang on rounding), the softmax in 32."""
    hq, hkv, d, page, topk = case["q_heads"], case["heads"], case["d"], case["page"], case["topk"]
    group = hq // hkv
    t, width = st["q"].shape[0], st["table"].shape[1]
    rows = 1 if case["share"] else group
    out = torch.empty(t, hq, d, dtype=torch.bfloat16, device=DEV)
    idx = torch.full((t, hkv * rows, topk), -1, dtype=torch.int32, device=DEV)
    step = max(1, (1 << 30) // max(hkv * width * d * 8, hq * min(topk, width) * page * d * 8))
    head = torch.arange(hkv, device=DEV)[None, :, None, None]
    for a in range(0, t, step):
        q, lens = st["q"][a:a + step], st["lens"][a:a + step].long()
        c = q.shape[0]
        table = st["table"][st["seq"][a:a + step].long()].long()
        nb = (lens + page - 1) // page
        block = torch.arange(width, device=DEV)
        there = block[None] < nb[:, None]
        means = st["kbar"][table.clamp(min=0)].double()                  # [c, width, hkv, d]
        qs = q.view(c, hkv, group, d).double()
        if case["share"]:
            qs = qs.sum(2, keepdim=True)
        score = torch.einsum("chgd,cbhd->chgb", qs, means)
        score = torch.where(there[:, None, None], score, -math.inf)
        if case["local"]:
            score = torch.where((block[None] == nb[:, None] - 1)[:, None, None], math.inf, score)
        kk = min(topk, width)
        best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :kk]
        count = nb.clamp(max=kk)[:, None, None, None]
        chosen = torch.arange(kk, device=DEV) < count
        best = torch.where(chosen, best, width).sort(-1).values
        chosen = best < width
        idx[a:a + step, :, :kk] = torch.where(chosen, best, -1).view(c, hkv * rows, kk).int()
        best = best.clamp(max=width - 1)
        pages = torch.gather(table[:, None, None].expand(c, hkv, rows, width), 3, best).clamp(min=0)
        key = best[..., None] * page + torch.arange(page, device=DEV)
        admit = (chosen[..., None] & (key < lens[:, None, None, None, None]))     # [c, hkv, rows, kk, page]
        kk_, vv = st["k"][pages, head].float(), st["v"][pages, head].float()       # [c, hkv, rows, kk, page, d]
        kk_ = torch.where(admit[..., None], kk_, 0.0).flatten(3, 4)
        vv = torch.where(admit[..., None], vv, 0.0).flatten(3, 4)
        admit = admit.flatten(3, 4)[:, :, :, None]
        qq = q.view(c, hkv, rows, group // rows, d).float()
        s = torch.einsum("chrgd,chrjd->chrgj", qq, kk_) / math.sqrt(d)
        s = torch.where(admit, s, -math.inf)
        m = s.amax(-1, keepdim=True).clamp(min=-1e30)
        p = torch.exp(s - m)
        o = torch.einsum("chrgj,chrjd->chrgd", p, vv) / p.sum(-1, keepdim=True).clamp(min=1e-30)
        out[a:a + step] = o.reshape(c, hq, d).to(torch.bfloat16)
    return out, idx


# ------------------------------------------------------------------ work
def work(case):
    if case["op"] == "rope":
        e = 2 if case["dtype"] == "bf16" else 4
        n = case["batch"] * case["heads"] * case["n"]
        # x once in, y once out; 6 operations a pair
        return dict(bytes=2 * n * case["d"] * e + 4 * case["batch"] * case["n"], flops=3 * n * case["rot"])
    heads, d, page = case["heads"], case["d"], case["page"]
    if case["op"] == "pages":
        return dict(bytes=2 * case["pairs"] * heads * d * (4 * page + 4), flops=0)
    if case["op"] == "append":
        touched = case["tokens"] / page + case["seqs"]
        return dict(bytes=8 * case["tokens"] * heads * d + 4 * touched * heads * d,
                    flops=case["tokens"] * heads * d)
    # the means of a sequence's blocks once for all its tokens; the pages that the heads of a group
    # (and a sequence's tokens) choose, counted once where they meet by chance
    s, hq, topk = case["seqs"], case["q_heads"], case["topk"]
    group = hq // heads
    mean_len = case["longest"] * (9 / 16 if s > 1 else 1)
    nb = max(1.0, math.ceil(case["longest"] / page) * (mean_len / case["longest"]))
    lists = (1 if case["share"] else group) * case["per_seq"]
    k = min(topk, nb)
    union = nb * (1 - (1 - k / nb) ** lists)
    keys = min(page, case["longest"])
    t = s * case["per_seq"]
    return dict(bytes=s * heads * (nb * d * 4 * (1 if nb > topk else 0) + union * keys * d * 4) + 4 * t * hq * d,
                flops=2 * t * hq * d * (nb / (group if case["share"] else 1) + 2 * k * keys))


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "rope":
        return _exact_rotate(st["x"].double(), st["positions"].long(), case,
                             -1.0 if case["backward"] else 1.0)
    if case["op"] == "pages":
        out = []
        for x in (st["k"], st["v"], st["kbar"]):
            y = x.clone()
            y.index_copy_(0, st["pairs"][:, 1].long(), x.index_select(0, st["pairs"][:, 0].long()))
            out.append(y)
        return tuple(out)
    return _exact_append(case, st) if case["op"] == "append" else _exact_decode(case, st)


def _exact_rotate(x, positions, case, sign):
    """Each pair as a complex number times m e^(i p f)."""
    rot = case["rot"]
    f = _inv_freq(case)
    turn = torch.polar(torch.full((), _attention_factor(case), dtype=torch.float64, device=DEV).expand(
        positions.shape + f.shape), sign * positions.double().unsqueeze(-1) * f).unsqueeze(1)
    y = x.clone()
    if case["interleaved"]:
        z = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) * turn
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * turn
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def _exact_append(case, st):
    k, v, kbar = st["k"].double(), st["v"].double(), st["kbar"].double()
    page = case["page"]
    cu, start, table = st["cu"].tolist(), st["start"].tolist(), st["table"].tolist()
    for s in range(case["seqs"]):
        lo, hi = cu[s], cu[s + 1]
        nk = st["new_k"][lo:hi].double().transpose(0, 1)
        nv = st["new_v"][lo:hi].double().transpose(0, 1)
        at = 0
        while at < hi - lo:
            p = start[s] + at
            n = min(page - p % page, hi - lo - at)
            where = table[s][p // page]
            k[where, :, p % page:p % page + n] = nk[:, at:at + n]
            v[where, :, p % page:p % page + n] = nv[:, at:at + n]
            kbar[where] = k[where, :, :p % page + n].mean(1)
            at += n
    return k, v, kbar


def _exact_decode(case, st):
    hq, hkv, d, page, topk = case["q_heads"], case["heads"], case["d"], case["page"], case["topk"]
    t, group = st["q"].shape[0], hq // hkv
    rows = 1 if case["share"] else group
    if t * hkv > 4096:
        return None
    out = torch.zeros(t, hq, d, dtype=torch.float64, device=DEV)
    idx = torch.full((t, hkv * rows, topk), -1, dtype=torch.int64)
    lens, seq, table = st["lens"].tolist(), st["seq"].tolist(), st["table"].long()
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
        flat = phys * page + pos % page
        kk = torch.where(ok[..., None], st["k"].view(-1, d)[flat].double(), 0.0)
        vv = torch.where(ok[..., None], st["v"].view(-1, d)[flat].double(), 0.0)
        qq = q.view(hkv, rows, group // rows, d)
        s = torch.matmul(qq, kk.transpose(2, 3)) * d ** -0.5
        w = torch.softmax(s.masked_fill(~ok[:, :, None], -math.inf), -1)
        out[i] = torch.matmul(w, vv).view(hq, d)
    return out, idx.to(device=DEV, dtype=torch.int32)
