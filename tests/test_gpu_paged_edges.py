"""The paged cache's operators on the GPU where the other tests do not go: the
precision of the weights, infinite values under one selection, forks."""
import pytest
import torch

from content_dependent_block_gb300 import _build, bsa
from tests import paged_reference as ref
from tests.test_gpu_paged import _cache, _i32, _problem, _randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    _build.build()


@pytest.fixture(autouse=True)
def _clean_status():
    bsa.device_status()
    yield
    torch.cuda.synchronize()


# ------------------------------------------------------- decode: precision
def half_step(y):
    """Half of the distance between the bf16 numbers around |y| (normal range)."""
    return torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -120))) - 8)


def narrow_bounds(k, v, q, table, lens, share, scale):
    """(out, tol) in fp64 of tokens that see all their blocks.  The weights'
    rounding is not among what tol allows but for 2^-17 (a bf16 value and the
    bf16 remainder of it leave 2^-18): the scores' roundings, exponentials and
    sums as in the decode reference, and the output's to the nearest bf16."""
    hkv, page, d = k.shape[1:]
    g = q.shape[1] // hkv
    out = torch.zeros(q.shape, dtype=torch.float64)
    tol = torch.zeros_like(out)
    for t, n in enumerate(lens):
        for h in range(hkv):
            pages = table[t, :-(-n // page)].long()
            kk, vv = (x[pages, h].reshape(-1, d)[:n].double() for x in (k, v))
            for r in range(h * g, (h + 1) * g):
                qd = q[t, r].double()
                w = torch.softmax(kk @ qd * scale, 0)
                out[t, r] = w @ vv
                slip = float((kk.abs() @ qd.abs()).max()) * scale * (d + 2) * 2.0 ** -24
                rel = 2.0 ** -17 + 2 * slip + 2.0 ** -20 + 2 * n * 2.0 ** -24
                off = rel * (w @ vv.abs())
                tol[t, r] = off + half_step(out[t, r].abs() + off)
    return out, tol


@pytest.mark.parametrize("hq,hkv,d,page", [(1, 1, 64, 16), (8, 2, 128, 16), (16, 1, 64, 64), (6, 1, 128, 128),
                                           (48, 4, 128, 32)])
@pytest.mark.parametrize("share", [False, True])
def test_decode_weights_keep_more_than_bf16(hq, hkv, d, page, share):
    """One rounding, to the output's type, is what the result is off by."""
    g = torch.Generator().manual_seed(hq + d + page)
    lens = [2, 3, 7, 15, page + 1, 3 * page - 1] * 4
    k, v, kbar, q, table = _problem(g, lens, hq, hkv, d, page)
    want, tol = narrow_bounds(k, v, q, table, lens, share, d ** -0.5)
    out, _ = bsa.paged_decode(_cache(k, v, kbar), q.cuda(), table.cuda(), _i32(lens), 32, share_group=share)
    ref.assert_within(out, want, tol, "decode")


@pytest.mark.parametrize("hq,share", [(1, False), (1, True), (4, True), (16, True), (3, False)])
@pytest.mark.parametrize("seqs", [1, 40])
@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
def test_decode_infinite_values_of_selected_blocks(hq, share, seqs, value):
    """An infinite value of the block that every head selects: its channel is
    that infinity, the other channels and tokens are finite."""
    g = torch.Generator().manual_seed(hq + seqs)
    lens = [30 * 16 + 9] * seqs
    k, v, kbar, q, table = _problem(g, lens, hq, 1, 64, 16)
    v = torch.where(torch.isfinite(v), v, 0)
    clean = v.clone()
    hit = [s for s in range(seqs) if s % 3 == 0]
    for s in hit:
        v[table[s, 30], 0, 4, 11] = value                   # the last block, always selected
    want, tol, widx = ref.decode(k, clean, kbar, q, table, lens, 4, share=share)
    out, idx = bsa.paged_decode(_cache(k, v, kbar), q.cuda(), table.cuda(), _i32(lens), 4, share_group=share)
    out = out.cpu()
    assert torch.equal(idx.cpu(), widx)
    rest = [c for c in range(64) if c != 11]
    ref.assert_within(out[..., rest], want[..., rest], tol[..., rest], "the other channels")
    for s in range(seqs):
        if s in hit:
            assert (out[s, :, 11] == value).all()
        else:
            ref.assert_within(out[s, :, 11], want[s, :, 11], tol[s, :, 11], "the other tokens")
    assert bsa.device_status() == 0


# --------------------------------------------------------- append: cu_tokens
@pytest.mark.parametrize("cu,start", [
    ([0, 64, 0, 64], [5, 0, 0]), ([0, 1000, 10, 20], [0, 64, 4]), ([0, 2, 1, 6], [0, 14, 3]),
    ([0, 500, 499, 1000], [3, 0, 16]), ([-1, 2, 4, 6], [0, 0, 0]), ([0, 2, 4, 1001], [0, 0, 0]),
    ([0, 2000, 2005, 1000], [0, 0, 0]), ([0, 1 << 30, -(1 << 30), 1000], [0, 0, 0]),
    ([1000, 0, 1000, 0], [0, 0, 0]), ([0, 3, 3, -1], [1, 2, 3]),
])
def test_append_reports_cu_tokens_that_make_no_sense(cu, start):
    """Reported wherever they are; a row that is written is its sequence's own,
    and a sequence with impossible bounds writes none."""
    g = torch.Generator().manual_seed(50)
    seqs, width, page, tokens = 3, 70, 16, 1000
    k, v = (_randn(g, seqs * width, 1, page, 64) for _ in range(2))
    rows = _randn(g, tokens, 2, 64)
    table = torch.arange(seqs * width).view(seqs, width)
    c, on = _cache(k, v, torch.zeros(seqs * width, 1, 64)), rows.cuda()
    bsa.cache_append(c, on[:, :1], on[:, 1:], table.int().cuda(), _i32(start), cu_tokens=_i32(cu))
    assert bsa.device_status() == 1
    for s in range(seqs):
        lo, hi = cu[s], cu[s + 1]
        for got, was, new in ((c.k, k, rows[:, 0]), (c.v, v, rows[:, 1])):
            a = got.cpu()[s * width:(s + 1) * width, 0].reshape(-1, 64)
            b = was[s * width:(s + 1) * width, 0].reshape(-1, 64).clone()
            moved = (a != b).any(1)
            if 0 <= lo <= hi <= tokens:
                at = slice(start[s], start[s] + hi - lo)
                b[at] = torch.where(moved[at, None], new[lo:hi], b[at])
            assert torch.equal(a, b)


def test_append_many_sequences_report_one_bad_bound():
    """One fall among thousands of sequences that get a token each or none."""
    g = torch.Generator().manual_seed(51)
    seqs = 5000
    for at in (0, 1, 127, 128, 2500, seqs - 1):
        cu = (torch.arange(seqs + 1) // 3).int()
        cu[at + 1:] -= 1
        if at == seqs - 1:
            cu[seqs] = cu[seqs - 1] - 1
        cu = torch.where(torch.arange(seqs + 1) == 0, 0, cu).int()
        falls = bool((cu.diff() < 0).any()) or bool((cu < 0).any())
        rows = _randn(g, int(seqs // 3) + 1, 1, 64).cuda()
        c = bsa.PagedCache.empty(seqs, 1, 16, 64)
        bsa.cache_append(c, rows, rows, torch.arange(seqs, dtype=torch.int32, device="cuda")[:, None],
                         _i32([0] * seqs), cu_tokens=cu.cuda())
        assert (bsa.device_status() == 1) == falls, at


# ----------------------------------------------------- decode: cluster sizes
def _tokens_of_one_sequence(g, width, rows, tokens, least, d=64):
    """One sequence over a table of `width` pages of 16, read by several tokens."""
    k, v, kbar, _, table = _problem(g, [width * 16], rows, 1, d, 16)
    lens = torch.randint(least, width * 16 + 1, (tokens,), generator=g).tolist()
    return k, v, kbar, _randn(g, tokens, rows, d), table, lens, [0] * tokens


def _check_tokens(k, v, kbar, q, table, lens, seq, topk, share):
    out, idx = bsa.paged_decode(_cache(k, v, kbar), q.cuda(), table.cuda(), _i32(lens), topk,
                                token_seq=_i32(seq), share_group=share)
    want, tol, widx = ref.decode(k, v, kbar, q, table, lens, topk, seq, share=share)
    assert torch.equal(idx.cpu(), widx)
    ref.assert_within(out, want, tol, "decode")
    assert bsa.device_status() == 0


@pytest.mark.parametrize("cluster", range(1, 17))
@pytest.mark.parametrize("rows,share", [(3, False), (3, True), (12, False), (12, True)])
def test_decode_in_clusters_of_every_size(cluster, rows, share):
    """One token takes a CTA for every 192 blocks (128 where a group has more
    than eight heads, and three at least for the blocks these select), up to
    sixteen."""
    g = torch.Generator().manual_seed(cluster + rows)
    width = (192 if rows <= 8 else 128) * cluster - 40
    _check_tokens(*_tokens_of_one_sequence(g, width, rows, 1, width * 15), 3, share)


@pytest.mark.parametrize("tokens", [7, 8, 13, 15, 23, 28, 29, 76, 100, 152, 200, 400])
@pytest.mark.parametrize("rows,share", [(2, False), (2, True), (9, False)])
def test_decode_in_the_clusters_of_every_batch(tokens, rows, share):
    """As the tokens grow, two heads take clusters of 13, 12, 10, 9, 6 and 5,
    then of 8, 8, 4, 4, 2 and 1 small CTAs; nine heads start at 16."""
    g = torch.Generator().manual_seed(tokens + rows)
    _check_tokens(*_tokens_of_one_sequence(g, 2500 if tokens <= 28 else 620, rows, tokens, 1), 4, share)


@pytest.mark.parametrize("tokens", [17, 28, 160])
def test_decode_in_clusters_that_grow_to_hold_the_scores(tokens):
    """Sixteen rows of 16384 scores are more than the cluster of that batch
    holds: it is doubled until they fit."""
    g = torch.Generator().manual_seed(tokens)
    k, v, kbar, _, table = _problem(g, [500], 16, 1, 64, 16, width=16384)
    lens = torch.randint(1, 501, (tokens,), generator=g).tolist()
    _check_tokens(k, v, kbar, _randn(g, tokens, 16, 64), table, lens, [0] * tokens, 3, False)
