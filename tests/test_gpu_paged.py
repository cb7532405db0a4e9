"""The paged cache on the GPU: append, page copies and decoding against plain
64-bit references, their run together, refusals and reported errors."""
import numpy as np
import pytest
import torch

from content_dependent_block_gb300 import _build, bsa
from tests import paged_reference as ref

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    _build.build()


@pytest.fixture(autouse=True)
def _clean_status():
    bsa.device_status()
    yield
    torch.cuda.synchronize()


def _randn(g, *shape, dtype=BF16):
    return torch.randn(*shape, generator=g).to(dtype)


def _cache(k, v, kbar):
    return bsa.PagedCache(k.cuda(), v.cuda(), kbar.cuda())


def _i32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


# ------------------------------------------------------------------- append
@pytest.mark.parametrize("d,page,heads", [(64, 64, 2), (128, 64, 3), (64, 16, 1), (128, 128, 2),
                                          (64, 128, 1), (128, 16, 5), (128, 32, 1), (64, 32, 9)])
@pytest.mark.parametrize("ragged", [True, False])
def test_append(d, page, heads, ragged):
    g = torch.Generator().manual_seed(d + page + heads)
    if ragged:
        new = [1, 0, page - 1, 2 * page + 3, page, 0, 1, 7]
        start = [0, 5, 1, page - 2, 3 * page, 0, page - 1, page]
    else:
        new, start = [3] * 5, [0, page - 1, page - 3, page, 2 * page + 1]
    seqs, width = len(new), 6
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    spare = 4                                    # tokens behind the last sequence
    table = torch.randperm(seqs * width, generator=g).view(seqs, width)
    pool = seqs * width + 2
    k, v = _randn(g, pool, heads, page, d), _randn(g, pool, heads, page, d)
    kbar = _randn(g, pool, heads, d, dtype=torch.float32)
    rows = _randn(g, cu[-1] + (spare if ragged else 0), 2 * heads + 1, d)
    nk, nv = rows[:, :heads], rows[:, heads + 1:]
    c = _cache(k, v, kbar)
    on = rows.cuda()
    for _ in range(2):                           # a call may be repeated
        bsa.cache_append(c, on[:, :heads], on[:, heads + 1:], _i32(table), _i32(start),
                         cu_tokens=_i32(cu) if ragged else None)
        wk, wv, wm, tol = ref.append(k, v, kbar, nk, nv, cu, start, table.tolist())
        assert torch.equal(c.k.cpu(), wk) and torch.equal(c.v.cpu(), wv)
        ref.assert_within(c.kbar, wm, tol, "means")
    assert bsa.device_status() == 0


def test_append_many_sequences_and_none():
    """More sequences than one search step covers, most of them empty."""
    g = torch.Generator().manual_seed(3)
    seqs, width, page, d = 1500, 2, 16, 64
    new = [int(x) for x in torch.randint(0, 9, (seqs,), generator=g) // 5]
    cu = [0] + torch.tensor(new).cumsum(0).tolist()
    start = torch.randint(0, 20, (seqs,), generator=g).tolist()
    table = torch.arange(seqs * width).view(seqs, width)
    k, v = _randn(g, seqs * width, 1, page, d), _randn(g, seqs * width, 1, page, d)
    kbar = torch.zeros(seqs * width, 1, d)
    rows = _randn(g, cu[-1], 2, d)
    c = _cache(k, v, kbar)
    on = rows.cuda()
    bsa.cache_append(c, on[:, :1], on[:, 1:], _i32(table), _i32(start), cu_tokens=_i32(cu))
    wk, wv, wm, tol = ref.append(k, v, kbar, rows[:, :1], rows[:, 1:], cu, start, table.tolist())
    assert torch.equal(c.k.cpu(), wk) and torch.equal(c.v.cpu(), wv)
    ref.assert_within(c.kbar, wm, tol, "means")
    bsa.cache_append(c, on[:0, :1], on[:0, 1:], _i32(table), _i32(start), cu_tokens=_i32([0] * (seqs + 1)))
    assert torch.equal(c.k.cpu(), wk) and bsa.device_status() == 0


def test_append_tokens_before_the_first_sequence():
    """cu_tokens need not start at 0: a step's tokens of other sequences lie
    before and behind."""
    g = torch.Generator().manual_seed(6)
    k, v = _randn(g, 12, 2, 16, 64), _randn(g, 12, 2, 16, 64)
    kbar = _randn(g, 12, 2, 64, dtype=torch.float32)
    rows = _randn(g, 150, 2, 64)
    table, start, cu = torch.arange(12).view(3, 4), [0, 15, 3], [83, 100, 101, 140]
    c = _cache(k, v, kbar)
    bsa.cache_append(c, rows.cuda(), rows.cuda(), _i32(table), _i32(start), cu_tokens=_i32(cu))
    wk, wv, wm, tol = ref.append(k, v, kbar, rows, rows, cu, start, table.tolist())
    assert torch.equal(c.k.cpu(), wk) and torch.equal(c.v.cpu(), wv) and bsa.device_status() == 0
    ref.assert_within(c.kbar, wm, tol, "means")


def test_append_reads_no_row_past_the_filled_ones():
    """Rows behind a sequence's end hold anything; a shorter sequence's means
    are those of its own rows."""
    g = torch.Generator().manual_seed(4)
    k = torch.full((1, 1, 64, 64), float("nan"), dtype=BF16)
    v = k.clone()
    old = _randn(g, 9, 1, 64)
    k[0, :, :9] = old.transpose(0, 1)
    c = _cache(k, v, torch.full((1, 1, 64), float("inf")))
    new = _randn(g, 2, 1, 64)
    bsa.cache_append(c, new.cuda(), new.cuda(), _i32([[0]]), _i32([9]))
    want = torch.cat([old, new]).double().mean(0)
    ref.assert_within(c.kbar[0], want, torch.full_like(want, 12 * 2.0 ** -24 * 4), "mean")
    assert c.k[0, 0, 11:].isnan().all()
    bsa.cache_append(c, new.cuda(), new.cuda(), _i32([[0]]), _i32([4]))     # cut to 4, appended to
    want = torch.cat([old[:4], new]).double().mean(0)
    ref.assert_within(c.kbar[0], want, torch.full_like(want, 7 * 2.0 ** -24 * 4), "mean")


@pytest.mark.parametrize("what", ["page", "unused page", "start", "room", "cu"])
def test_append_reports_bad_arguments_and_skips(what):
    g = torch.Generator().manual_seed(5)
    k, v, kbar = _randn(g, 6, 1, 16, 64), _randn(g, 6, 1, 16, 64), torch.zeros(6, 1, 64)
    rows = _randn(g, 6, 1, 64)
    table, start, cu = [[0, 1], [2, 3], [4, 5]], [0, 14, 3], [0, 2, 4, 6]
    if what == "page":
        table[1] = [6, 3]
    if what == "unused page":                    # its tokens end with the first page
        table[1] = [2, 6]
    if what == "start":
        start[1] = -1
    if what == "room":
        start[1] = 31
    if what == "cu":
        cu = [0, 2, 1, 6]
    c = _cache(k, v, kbar)
    bsa.cache_append(c, rows.cuda(), rows.cuda(), _i32(table), _i32(start), cu_tokens=_i32(cu))
    assert bsa.device_status() == {"page": 3, "unused page": 0}.get(what, 1)
    got = c.k.cpu()
    assert torch.equal(got[0, 0, :2], rows[:2, 0])                  # the others were served
    if what != "cu":
        assert torch.equal(got[4, 0, 3:5], rows[4:, 0])
    assert torch.equal(got[3], k[3])
    assert torch.equal(got[2, 0, :14], k[2, 0, :14])


# -------------------------------------------------------------------- copies
@pytest.mark.parametrize("d,page,heads,pool,count", [(64, 16, 1, 5, 1), (128, 128, 7, 31, 11),
                                                     (64, 64, 2, 200, 90), (128, 32, 1, 9, 0)])
def test_copy_pages(d, page, heads, pool, count):
    g = torch.Generator().manual_seed(pool)
    k, v = _randn(g, pool, heads, page, d), _randn(g, pool, heads, page, d)
    kbar = _randn(g, pool, heads, d, dtype=torch.float32)
    order = torch.randperm(pool, generator=g)
    pairs = torch.stack([order[:count], order[count:2 * count]], 1).int()
    c = _cache(k, v, kbar)
    bsa.copy_pages(c, pairs.cuda() if count % 2 else pairs.numpy())
    for got, was in ((c.k, k), (c.v, v), (c.kbar, kbar)):
        was[pairs[:, 1].long()] = was[pairs[:, 0].long()]
        assert torch.equal(got.cpu(), was)
    assert bsa.device_status() == 0


def test_copy_pages_from_one_to_many_and_bad_ids():
    g = torch.Generator().manual_seed(1)
    k, v, kbar = _randn(g, 4, 1, 16, 64), _randn(g, 4, 1, 16, 64), _randn(g, 4, 1, 64, dtype=torch.float32)
    c = _cache(k, v, kbar)
    bsa.copy_pages(c, np.array([[0, 1], [0, 2], [4, 3], [0, -1]], dtype=np.int32))
    assert bsa.device_status() == 3
    for got, was in ((c.k, k), (c.v, v), (c.kbar, kbar)):
        assert torch.equal(got.cpu()[:3], was[:1].expand_as(was[:3])) and torch.equal(got.cpu()[3], was[3])


# -------------------------------------------------------------------- decode
def _problem(g, lens, hq, hkv, d, page, width=None, q_cols=0):
    """A cache of sequences of these lengths, the rows behind each end NaN or
    inf, and one query row per sequence."""
    seqs = len(lens)
    per = [-(-n // page) for n in lens]
    width = width or max(1, max(per))
    pool = sum(per) + 1
    ids = torch.randperm(pool - 1, generator=g).tolist()
    table = torch.full((seqs, width), -1, dtype=torch.int32)
    k, v = _randn(g, pool, hkv, page, d), _randn(g, pool, hkv, page, d)
    k = (k.float() + 0.5 * torch.randn(pool, hkv, 1, d, generator=g)).to(BF16)
    kbar = k.float().mean(2)
    at = 0
    for s in range(seqs):
        table[s, :per[s]] = torch.tensor(ids[at:at + per[s]], dtype=torch.int32)
        at += per[s]
        if lens[s] % page:
            p, fill = table[s, per[s] - 1], lens[s] % page
            kbar[p] = k[p, :, :fill].float().mean(1)
            k[p, :, fill:] = float("nan")
            v[p, :, fill:] = float("inf")
    q = _randn(g, seqs, hq + q_cols, d)
    return k, v, kbar, q, table


def _check(k, v, kbar, q, table, lens, topk, q_dev=None, **kw):
    c = _cache(k, v, kbar)
    ts = kw.pop("token_seq", None)
    out, idx = bsa.paged_decode(c, q.cuda() if q_dev is None else q_dev, table.cuda(), _i32(lens), topk,
                                token_seq=None if ts is None else _i32(ts), local_block=kw.get("local", True),
                                share_group=kw.get("share", False), scale=kw.get("scale") or 0.0)
    want, tol, widx = ref.decode(k, v, kbar, q, table, lens, topk, ts, **kw)
    assert torch.equal(idx.cpu(), widx), (idx.cpu() != widx).nonzero()[:4]
    ref.assert_within(out, want, tol, "decode")
    assert bsa.device_status() == 0
    return out, idx


SHAPES = [  # q heads, cache heads, d, page, topk
    (1, 1, 64, 64, 4), (2, 2, 64, 64, 1), (6, 2, 128, 16, 3), (8, 1, 128, 64, 16), (20, 4, 64, 32, 7),
    (7, 1, 128, 128, 2), (16, 1, 64, 16, 32), (24, 2, 128, 32, 5), (17, 1, 64, 64, 3), (66, 2, 128, 16, 2),
    (128, 1, 64, 16, 4), (4, 4, 128, 64, 32),
]


@pytest.mark.parametrize("hq,hkv,d,page,topk", SHAPES)
@pytest.mark.parametrize("share", [False, True])
@pytest.mark.parametrize("local", [False, True])
def test_decode_shapes(hq, hkv, d, page, topk, share, local):
    g = torch.Generator().manual_seed(hq * 1000 + d + page + topk)
    lens = [0, 1, page - 1, page, page + 1, 5 * page + 3, 40 * page - 1, 12 * page]
    k, v, kbar, q, table = _problem(g, lens, hq, hkv, d, page, width=43)
    _check(k, v, kbar, q, table, lens, topk, share=share, local=local)


@pytest.mark.parametrize("seqs,hkv", [(1, 1), (3, 2), (40, 1), (90, 2), (160, 2)])
@pytest.mark.parametrize("share", [False, True])
def test_decode_at_every_cluster_size(seqs, hkv, share):
    """Few tokens take clusters of eight CTAs, many take single ones."""
    g = torch.Generator().manual_seed(seqs)
    lens = torch.randint(1, 700, (seqs,), generator=g).tolist()
    k, v, kbar, q, table = _problem(g, lens, 3 * hkv, hkv, 64, 16)
    _check(k, v, kbar, q, table, lens, 6, share=share)


def test_decode_long_sequence():
    g = torch.Generator().manual_seed(8)
    lens = [65537]
    k, v, kbar, q, table = _problem(g, lens, 8, 1, 64, 16)
    _check(k, v, kbar, q, table, lens, 32)
    _check(k, v, kbar, q, table, lens, 32, share=True, local=False)


@pytest.mark.parametrize("hq", [1, 16])
def test_decode_widest_table(hq):
    """All 16384 blocks, and a table that is mostly behind the sequence."""
    g = torch.Generator().manual_seed(9)
    lens = [16384 * 16 - 5]
    k, v, kbar, q, table = _problem(g, lens, hq, 1, 64, 16)
    assert table.shape[1] == 16384
    _check(k, v, kbar, q, table, lens, 5)
    _check(k, v, kbar, q, table, [100], 5)


def test_decode_several_tokens_of_a_sequence_and_strided_rows():
    g = torch.Generator().manual_seed(10)
    lens = [130, 64, 300]
    k, v, kbar, _, table = _problem(g, lens, 4, 2, 128, 32)
    rows = _randn(g, 7, 9, 128)
    dev = rows.cuda()
    _check(k, v, kbar, rows[:, 2:6], table, [128, 129, 130, 64, 0, 299, 300], 3,
           q_dev=dev[:, 2:6], token_seq=[0, 0, 0, 1, 1, 2, 2])


@pytest.mark.parametrize("scale", [1.0, 0.01, 4.0])
def test_decode_scale(scale):
    g = torch.Generator().manual_seed(11)
    k, v, kbar, q, table = _problem(g, [500, 77], 4, 1, 64, 16)
    _check(k, v, kbar, q, table, [500, 77], 4, scale=scale)


@pytest.mark.parametrize("share", [False, True])
@pytest.mark.parametrize("seqs", [1, 60])
def test_decode_ties_go_to_the_lower_block(share, seqs):
    """Equal means everywhere, equal means in runs, means of zero."""
    g = torch.Generator().manual_seed(12)
    lens = [40 * 16] * seqs
    k, v, kbar, q, table = _problem(g, lens, 5, 1, 64, 16)
    kbar[:] = kbar[0]
    _check(k, v, kbar, q, table, lens, 7, share=share, local=False)
    kbar[:] = 0
    _check(k, v, kbar, q, table, lens, 7, share=share)
    some = torch.randn(6, 1, 64, generator=g)
    for s in range(seqs):
        for b in range(40):
            kbar[table[s, b]] = some[b % 6]
    _check(k, v, kbar, q, table, lens, 9, share=share, local=False)


@pytest.mark.parametrize("topk", [3, 16])
def test_decode_settles_close_scores(topk):
    """Means that differ in their last bits: the order of the fp32 sums would
    decide, the exact values do."""
    g = torch.Generator().manual_seed(13)
    lens = [300 * 16, 120 * 16 + 3]
    k, v, kbar, q, table = _problem(g, lens, 8, 1, 128, 16)
    base = torch.randn(1, 1, 128, generator=g)
    step = torch.randint(-2, 3, kbar.shape, generator=g).float() * 2.0 ** -23
    kbar[:] = base * (1 + step)
    _check(k, v, kbar, q, table, lens, topk, local=False)
    _check(k, v, kbar, q, table, lens, topk, share=True)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 3.0e38])
def test_decode_means_that_are_not_finite(value):
    """Scores that are NaN rank as -inf, infinite ones by their sign; finite
    means whose fp32 score overflows rank by their exact one."""
    g = torch.Generator().manual_seed(14)
    lens = [50 * 16]
    k, v, kbar, q, table = _problem(g, lens, 3, 1, 64, 16)
    for b in (3, 17, 18, 40):
        kbar[table[0, b]] = value if value == 3.0e38 else torch.where(
            torch.arange(64) == b, value, kbar[table[0, b]])
    _check(k, v, kbar, q, table, lens, 4, local=False)
    _check(k, v, kbar, q, table, lens, 4)


@pytest.mark.parametrize("seqs", [1, 2, 70])
def test_decode_keeps_other_rows_from_values_that_are_not_finite(seqs):
    """Heads of a group share the tiles of their blocks; an infinite or NaN
    value counts for the heads that selected its block, and for no other."""
    g = torch.Generator().manual_seed(30)
    lens = [60 * 16 + 5] * seqs
    k, v, kbar, q, table = _problem(g, lens, 6, 1, 64, 16)
    _, _, sel = ref.decode(k, v, kbar, q, table, lens, 4)
    v = torch.where(torch.isfinite(v), v, 0)               # the rows behind the end, too
    bad = []
    for s in range(seqs):
        only = [b for b in sel[s, 0].tolist() if b not in sel[s, 1:].flatten().tolist()]
        bad.append(bool(only))
        if only:
            v[table[s, only[0]], 0, 3, 7] = float("inf") if s % 2 else float("nan")
    assert any(bad)
    want, tol, widx = ref.decode(k, v, kbar, q, table, lens, 4)
    out, idx = bsa.paged_decode(_cache(k, v, kbar), q.cuda(), table.cuda(), _i32(lens), 4)
    out = out.cpu()
    assert torch.equal(idx.cpu(), widx)
    ref.assert_within(out[:, 1:], want[:, 1:], tol[:, 1:], "the other heads")
    for s in range(seqs):
        rest = [c for c in range(64) if c != 7]
        ref.assert_within(out[s, 0, rest], want[s, 0, rest], tol[s, 0, rest], "the head's other channels")
        assert torch.isfinite(out[s, 0, 7]) == torch.tensor(not bad[s])


@pytest.mark.parametrize("what", ["q zero", "q nan", "q inf", "means zero", "a page missing"])
@pytest.mark.parametrize("width", [80, 3000])
def test_decode_scores_that_decide_nothing(what, width):
    """No score differs (or none is a number): the lowest ids, and in time."""
    g = torch.Generator().manual_seed(31)
    n = width * 16 - 3
    k, v, kbar, q, table = _problem(g, [n], 3, 1, 64, 16)
    fill = {"q zero": 0.0, "q nan": float("nan"), "q inf": float("inf")}.get(what)
    if fill is not None:
        q[:, 1] = fill
    if what in ("means zero", "a page missing"):
        kbar[:] = 0
    bad = table.clone()
    if what == "a page missing":
        bad[0, 2] = -5
    c = _cache(k, v, kbar)
    out, idx = bsa.paged_decode(c, q.cuda(), bad.cuda(), _i32([n]), 4, local_block=False)
    torch.cuda.synchronize()
    assert bsa.device_status() == (3 if what == "a page missing" else 0)
    if what in ("q zero", "means zero"):
        assert idx[0, 1].tolist() == [0, 1, 2, 3]
    if what == "a page missing":
        assert idx[0].tolist() == [[0, 1, 3, 4]] * 3
    if what == "q nan":
        assert idx[0, 1].tolist() == [0, 1, 2, 3] and out[0, 1].isnan().all()
    if what == "q inf":              # every score is NaN or infinite
        assert (idx[0, 1].diff() > 0).all() and not torch.isfinite(out[0, 1]).any()
    others = [0, 2] if fill is not None else [0, 1, 2] if what == "means zero" else []
    want, tol, widx = ref.decode(k, v, kbar, q, table, [n], 4, local=False)
    for h in others:
        assert torch.equal(idx[0, h].cpu(), widx[0, h])
        ref.assert_within(out[0, h], want[0, h], tol[0, h], "the other heads")


def test_pages_past_32_bit_offsets():
    """A cache of more than 2^32 elements: pages at its end are appended to,
    copied and read at their own places."""
    g = torch.Generator().manual_seed(32)
    heads, page, d = 8, 128, 128
    pool = (1 << 32) // (heads * page * d) + 40
    k, v = (torch.empty((pool, heads, page, d), dtype=BF16, device="cuda") for _ in range(2))
    kbar = torch.zeros((pool, heads, d), device="cuda")
    c = bsa.PagedCache(k, v, kbar)
    ids = [pool - 1, 3, pool - 2, pool - 7, 5]
    n = 5 * page - 11
    nk, nv = _randn(g, n, heads, d), _randn(g, n, heads, d)
    bsa.cache_append(c, nk.cuda(), nv.cuda(), _i32([ids]), _i32([0]))
    moved = [pool - 20, 3, pool - 2, pool - 21, 5]
    bsa.copy_pages(c, np.array([[pool - 1, pool - 20], [pool - 7, pool - 21]], dtype=np.int32))
    q = _randn(g, 1, 2 * heads, d)
    out, idx = bsa.paged_decode(c, q.cuda(), _i32([moved]), _i32([n]), 3)
    small = [torch.stack([t[i] for i in moved]).cpu() for t in (k, v, kbar)]
    rows = torch.cat([nk, torch.zeros(11, heads, d, dtype=BF16)]).view(5, page, heads, d).transpose(1, 2)
    assert torch.equal(small[0][:4], rows[:4]) and torch.equal(small[0][4, :, :page - 11], rows[4, :, :page - 11])
    want, tol, widx = ref.decode(*small, q, torch.arange(5)[None], [n], 3)
    assert torch.equal(idx.cpu(), widx)
    ref.assert_within(out, want, tol, "decode")
    assert bsa.device_status() == 0


def test_two_calls_at_once():
    """Calls on two streams share nothing but the status word."""
    g = torch.Generator().manual_seed(33)
    calls = []
    for i in range(2):
        lens = torch.randint(1, 3000, (20,), generator=g).tolist()
        k, v, kbar, q, table = _problem(g, lens, 8, 2, 64, 16)
        calls.append((_cache(k, v, kbar), q.cuda(), table.cuda(), _i32(lens)))
    want = [bsa.paged_decode(*c, 8)[0] for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(bsa.paged_decode(*calls[i], 8)[0])
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        assert all(torch.equal(w, x) for x in runs)


def test_decode_selects_alike_in_any_batch():
    """The blocks a token sees do not hang on what it is decoded with: all
    tokens at once (single CTAs), some, and one (clusters)."""
    g = torch.Generator().manual_seed(34)
    lens = torch.randint(1, 9000, (400,), generator=g).tolist()
    k, v, kbar, _, table = _problem(g, [9000], 8, 2, 64, 16)
    q = _randn(g, 400, 8, 64)
    c, seq = _cache(k, v, kbar), _i32([0] * 400)
    for share in (False, True):
        call = lambda a, b: bsa.paged_decode(c, q[a:b].cuda(), table.cuda(), _i32(lens[a:b]), 9,
                                             token_seq=seq[a:b], share_group=share, local_block=False)
        out, idx = call(0, 400)
        for a, b in ((0, 1), (17, 18), (100, 120), (200, 333)):
            some, ids = call(a, b)
            assert torch.equal(ids, idx[a:b])
            # other clusters merge in another order: one bf16 step at most
            assert float((some.float() - out[a:b].float()).abs().max()) <= 2.0 ** -7 * float(out.abs().max())


def test_c_call_without_options_or_selection():
    """idx_out NULL: no selection is written; options NULL: no forced block,
    every head for itself."""
    g = torch.Generator().manual_seed(35)
    lens = [700, 31]
    k, v, kbar, q, table = _problem(g, lens, 4, 2, 64, 16)
    c, dev, tab, n = _cache(k, v, kbar), q.cuda(), table.cuda(), _i32(lens)
    out = torch.full((2, 4, 64), 9.0, dtype=BF16, device="cuda")
    L = bsa.lib()
    assert L.bsa_paged_decode(c.struct, dev.data_ptr(), 256, 2, 4, tab.data_ptr(), table.shape[1], 2, None,
                              n.data_ptr(), 3, None, 0.0, out.data_ptr(), None,
                              torch.cuda.current_stream().cuda_stream) == 0
    want, tol, _ = ref.decode(k, v, kbar, q, table, lens, 3, local=False)
    ref.assert_within(out, want, tol, "decode")
    same, _ = bsa.paged_decode(c, dev, tab, n, 3, local_block=False)
    assert torch.equal(out, same)


def test_no_tokens():
    c = bsa.PagedCache.empty(4, 2, 16, 64)
    q = torch.zeros(0, 4, 64, dtype=BF16, device="cuda")
    out, idx = bsa.paged_decode(c, q, _i32([[0]]), _i32([]), 2)
    assert out.shape == (0, 4, 64) and idx.shape == (0, 4, 2)


def test_decode_reads_no_page_behind_the_end():
    g = torch.Generator().manual_seed(15)
    lens = [33, 1]
    k, v, kbar, q, table = _problem(g, lens, 2, 1, 64, 16, width=50)
    table[:, 4:] = 2 ** 31 - 1
    _check(k, v, kbar, q, table, lens, 2)


@pytest.mark.parametrize("what", ["page", "all pages", "long", "negative", "seq"])
def test_decode_reports_bad_arguments(what):
    g = torch.Generator().manual_seed(16)
    lens = [20 * 16, 3 * 16, 50]
    k, v, kbar, q, table = _problem(g, lens, 2, 1, 64, 16)
    bad, ts = table.clone(), None
    if what == "page":
        bad[0, 5] = k.shape[0]
        bad[1, 1] = -7
    if what == "all pages":
        bad[1, :] = -1
    if what == "long":
        lens[1] = 20 * 16 + 1
    if what == "negative":
        lens[1] = -1
    if what == "seq":
        ts = [0, 3, 2]
    c = _cache(k, v, kbar)
    out, idx = bsa.paged_decode(c, q.cuda(), bad.cuda(), _i32(lens), 3, local_block=False,
                                token_seq=None if ts is None else _i32(ts))
    torch.cuda.synchronize()
    assert bsa.device_status() in ((1, 3) if what == "long" else (1,) if what == "negative" else (3,))
    want, tol, widx = ref.decode(k, v, kbar, q[2:], table[2:], [50], 3, local=False)
    assert torch.equal(idx[2:].cpu(), widx)
    ref.assert_within(out[2:], want, tol, "the good token")
    if what in ("negative", "seq"):
        assert not out[1].any() and (idx[1] == -1).all()
    if what == "all pages":
        assert not out[1].any()
    if what == "page":
        assert 5 not in idx[0].tolist() and idx[1].tolist() == [[0, 1, 2]] * 2
        # the bad page's keys are left out of the softmax
        kk = torch.cat([k[table[1, 0], 0], k[table[1, 2], 0]]).double()
        vv = torch.cat([v[table[1, 0], 0], v[table[1, 2], 0]]).double()
        w = torch.softmax(kk @ q[1, 0].double() / 8, 0) @ vv
        ref.assert_within(out[1, 0], w, torch.full_like(w, 2.0 ** -6), "without the bad page")


def test_decode_is_deterministic_and_writes_its_rows_only():
    g = torch.Generator().manual_seed(17)
    lens = torch.randint(1, 4000, (24,), generator=g).tolist()
    k, v, kbar, q, table = _problem(g, lens, 8, 2, 128, 32)
    c = _cache(k, v, kbar)
    dev = q.cuda()
    frame = torch.full((26, 8, 128), 7.0, dtype=BF16, device="cuda")
    a, ia = bsa.paged_decode(c, dev, table.cuda(), _i32(lens), 8, out=frame[1:25])
    b, ib = bsa.paged_decode(c, dev, table.cuda(), _i32(lens), 8)
    assert torch.equal(a, b) and torch.equal(ia, ib)
    assert (frame[0] == 7).all() and (frame[25] == 7).all()
    assert torch.equal(c.k.cpu().view(torch.int16), k.view(torch.int16)) and torch.equal(c.kbar.cpu(), kbar)


def test_python_refusals():
    c = bsa.PagedCache.empty(4, 2, 16, 64)
    q = torch.zeros(3, 4, 64, dtype=BF16, device="cuda")
    table, lens = _i32([[0], [1], [2]]), _i32([1, 1, 1])
    for err, call in [
        (TypeError, lambda: bsa.paged_decode(c, q, table.long(), lens, 1)),
        (TypeError, lambda: bsa.paged_decode(c, q, table, lens[:2], 1)),
        (ValueError, lambda: bsa.paged_decode(c, q.half(), table, lens, 1)),
        (ValueError, lambda: bsa.paged_decode(c, q.transpose(0, 1), table, lens, 1)),
        (ValueError, lambda: bsa.paged_decode(c, q.cpu(), table, lens, 1)),
        (bsa.BsaError, lambda: bsa.paged_decode(c, q[:, :3], table, lens, 1)),
        (bsa.BsaError, lambda: bsa.paged_decode(c, q, table, lens, 33)),
        (ValueError, lambda: bsa.cache_append(c, q, q, table, lens)),
        (TypeError, lambda: bsa.cache_append(c, q[:, :2], q[:, :2], table, lens, cu_tokens=lens)),
        (TypeError, lambda: bsa.copy_pages(c, _i32([0, 1]))),
        (ValueError, lambda: bsa.PagedCache(c.k, c.v[:2], c.kbar)),
        (ValueError, lambda: bsa.PagedCache(c.k, c.v, c.kbar.double())),
    ]:
        with pytest.raises((err, IndexError)):
            call()


# ----------------------------------------------------------------- together
def test_prefill_decode_fork_and_compaction():
    """Prompts rotated, appended, decoded; two of the sequences forked and cut
    short; the pool compacted; each step against the logical sequences."""
    g = torch.Generator().manual_seed(20)
    hq, hkv, d, page, topk = 8, 2, 64, 16, 5
    pt = bsa.PageTable(96, page, 5, 24)
    cache = bsa.PagedCache.empty(96, hkv, page, d)
    plan = bsa.Rope(d, scaling="parts", factor=4.0, original=64.0, attention_factor=1.1)
    freq = ref.inv_freq(d, scaling="parts", factor=4.0, original=64.0)
    logical = [(torch.zeros(0, hkv, d, dtype=BF16), torch.zeros(0, hkv, d, dtype=BF16)) for _ in range(5)]

    def step(new):
        """new: tokens for each sequence; returns nothing, checks all."""
        _, before = pt.tables()
        for s, n in enumerate(new):
            pt.reserve(s, n)
        bsa.copy_pages(cache, pt.take_copies())
        table, lens = pt.tables()
        t = sum(new)
        pos = torch.cat([torch.arange(before[s], before[s] + n) for s, n in enumerate(new)]).int()
        qkv = _randn(g, t, hq + 2 * hkv, d)
        dev = qkv.cuda()
        qk = dev[:, :hq + hkv].transpose(0, 1)
        bsa.rope(qk, plan, pos.cuda(), out=qk)                       # q and k where they are
        want, tol = ref.rope(qkv[:, :hq + hkv].transpose(0, 1)[None], pos[None], freq, False, 1.1)
        ref.assert_within(qk[None], want, tol, "rotated")
        cu = _i32(np.concatenate([[0], np.cumsum(new)]))
        bsa.cache_append(cache, dev[:, hq:hq + hkv], dev[:, hq + hkv:], _i32(table), _i32(before),
                         cu_tokens=cu)
        host = dev.cpu()
        at = 0
        for s, n in enumerate(new):
            logical[s] = tuple(torch.cat([old, part]) for old, part in
                               zip(logical[s], (host[at:at + n, hq:hq + hkv], host[at:at + n, hq + hkv:])))
            at += n
        # every new token sees the sequence up to itself, its own block forced
        ts = torch.cat([torch.full((n,), s) for s, n in enumerate(new)]).int()
        out, idx = bsa.paged_decode(cache, dev[:, :hq], _i32(table), _i32(pos + 1), topk,
                                    token_seq=ts.cuda())
        # the reference's own pages: sequence s's block b is page s * 24 + b
        k, v = torch.zeros(120, hkv, page, d, dtype=BF16), torch.zeros(120, hkv, page, d, dtype=BF16)
        for s in range(5):
            for i in range(logical[s][0].shape[0]):
                k[s * 24 + i // page, :, i % page] = logical[s][0][i]
                v[s * 24 + i // page, :, i % page] = logical[s][1][i]
        kbar = torch.zeros(120, hkv, d)
        for s in range(5):
            for b in range(-(-int(lens[s]) // page)):
                kbar[s * 24 + b] = cache.kbar[int(table[s, b])].cpu()
                rows = min(page, int(lens[s]) - b * page)
                mean = k[s * 24 + b, :, :rows].double().mean(1)
                ref.assert_within(kbar[s * 24 + b], mean, torch.full_like(mean, 2.0 ** -18), "mean")
        ids = torch.arange(120).view(5, 24)
        want, tol, widx = ref.decode(k, v, kbar, host[:, :hq], ids, (pos + 1).tolist(), topk, ts.tolist())
        assert torch.equal(idx.cpu(), widx)
        ref.assert_within(out, want, tol, "decode")
        assert bsa.device_status() == 0

    step([150, 33, 0, 0, 1])
    step([1, 1, 0, 0, 1])
    pt.fork(0, 2)
    logical[2] = logical[0]
    pt.fork(0, 3)
    logical[3] = logical[0]
    step([1, 1, 1, 2, 1])
    pt.truncate(3, 100)
    logical[3] = tuple(x[:100] for x in logical[3])
    step([1, 0, 1, 3, 1])
    pt.free(0)
    logical[0] = tuple(x[:0] for x in logical[0])
    bsa.copy_pages(cache, pt.compact())
    assert pt.tables()[0].max() < 96 - pt.free_pages
    step([0, 1, 1, 1, 16])
    step([5, 1, 1, 1, 1])


def test_decode_agrees_with_the_forward():
    """The last token of the causal forward with the own block forced, and the
    same token decoded from a cache of its keys: same blocks, same attention
    (each off the exact value by its own roundings)."""
    g = torch.Generator().manual_seed(21)
    bh, n, d, page, topk = 4, 2048 + 37, 64, 64, 8
    q, k, v = (_randn(g, bh, n, d).cuda() for _ in range(3))
    k = (k.float() + 0.5 * torch.randn(bh, -(-n // page), 1, d, generator=g).cuda().expand(
        -1, -1, page, -1).reshape(bh, -1, d)[:, :n]).to(BF16)
    full, fidx = bsa.forward(q, k, v, page, topk, causal=True, local_block=True)
    cache = bsa.PagedCache.empty(40, bh, page, d)
    table = torch.randperm(40, generator=g)[None, :-(-n // page)]
    bsa.cache_append(cache, k.transpose(0, 1).contiguous(), v.transpose(0, 1).contiguous(), _i32(table),
                     _i32([0]))
    means = bsa.pool_blocks(k, page)
    back = cache.kbar[table[0].cuda()].transpose(0, 1)
    assert float((back - means).abs().max()) <= 2 * 65 * 2.0 ** -24 * 4
    out, idx = bsa.paged_decode(cache, q[:, -1][None].contiguous(), _i32(table), _i32([n]), topk)
    assert torch.equal(idx[0], fidx[:, -1])
    err = (out[0].float() - full[:, -1].float()).abs().max()
    assert float(err) <= 2e-2


def test_streams_and_graph_replay():
    """A captured step (rotate, append, decode) replayed with new inputs and
    longer sequences equals the eager one; another stream gives the same."""
    g = torch.Generator().manual_seed(22)
    hq, hkv, d, page, seqs, width = 8, 2, 128, 64, 6, 8
    lens = [1, 63, 64, 200, 301, 129]
    k, v, kbar, _, table = _problem(g, [n + 2 for n in lens], hq, hkv, d, page, width=width)
    qkv = _randn(g, seqs, hq + 2 * hkv, d).cuda()
    plan = bsa.Rope(d)
    start, after, table = _i32(lens), _i32(lens) + 1, table.cuda()

    def one(cache, out):
        x = qkv.clone()
        qk = x[:, :hq + hkv].transpose(0, 1)
        bsa.rope(qk, plan, start, out=qk)
        bsa.cache_append(cache, x[:, hq:hq + hkv], x[:, hq + hkv:], table, start)
        return bsa.paged_decode(cache, x[:, :hq], table, after, 3, out=out)[0]

    eager, captured = _cache(k, v, kbar), _cache(k, v, kbar)
    out = torch.zeros(seqs, hq, d, dtype=BF16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm = one(captured, None)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one(captured, out)
    want = one(eager, None)
    assert torch.equal(warm, want)
    graph.replay()
    assert torch.equal(out, want)
    start += 1
    after += 1
    qkv.copy_(_randn(g, seqs, hq + 2 * hkv, d).cuda())
    graph.replay()
    assert torch.equal(out, one(eager, None))
    assert torch.equal(captured.kbar, eager.kbar) and bsa.device_status() == 0
