"""New tokens over the paged cache on the GPU, against plain 64-bit
references: single tokens, chunks, trees, windows with sinks, both kinds of
pages."""
import numpy as np
import pytest
import torch

from content_dependent_block_gb300 import _build, bsa
from tests import attention_reference as att
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


def _i32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def _trees(g, new):
    words = []
    for n in new:
        parents = [int(torch.randint(-1, i, (1,), generator=g)) if i else -1 for i in range(n)]
        words += att.tree_masks(parents)
    return words


class Step:
    """A step over random pages: rows past each sequence's end, and pages that
    no sequence has, hold what must not be read."""

    def __init__(self, seed, d, page, heads, group, bits, start, new, poison=True, width=None):
        g = self.g = torch.Generator().manual_seed(seed)
        self.start, self.new, self.bits = start, new, bits
        self.cu = np.cumsum([0] + new).tolist()
        width = width or max(1, max(-(-(s + n) // page) for s, n in zip(start, new)))
        seqs = len(new)
        pool = seqs * width + 1
        self.table = torch.randperm(seqs * width, generator=g).view(seqs, width).tolist()
        if bits == 8:
            self.k, self.v = (torch.randint(-127, 128, (pool, heads, page, d), generator=g).to(torch.int8)
                              for _ in range(2))
            self.ks, self.vs = (0.01 + 0.02 * torch.rand(pool, heads, page, generator=g) for _ in range(2))
        else:
            self.k, self.v = _randn(g, pool, heads, page, d), _randn(g, pool, heads, page, d)
        if poison:
            for s in range(seqs):
                end = start[s] + new[s]
                for b in range(width):
                    rows = min(max(end - b * page, 0), page)
                    at = self.table[s][b]
                    if bits == 8:
                        self.ks[at, :, rows:], self.vs[at, :, rows:] = float("nan"), float("inf")
                    else:
                        self.k[at, :, rows:], self.v[at, :, rows:] = float("inf"), float("nan")
        self.q = _randn(g, self.cu[-1], heads * group, d)

    def cache(self):
        kbar = torch.zeros(self.k.shape[0], self.k.shape[1], self.k.shape[3], device="cuda")
        if self.bits == 8:
            return bsa.PagedCache8(self.k.cuda(), self.v.cuda(), self.ks.cuda(), self.vs.cuda(), kbar)
        return bsa.PagedCache(self.k.cuda(), self.v.cuda(), kbar)

    def values(self):
        if self.bits == 8:
            return att.values(self.k, self.ks), att.values(self.v, self.vs)
        return self.k, self.v

    def check(self, words=None, window=0, sinks=0, bounds=True, scale=0.0, what="", skipped=()):
        tree = None if words is None else torch.tensor(words, dtype=torch.int64, device="cuda")
        got = bsa.paged_attention(self.cache(), self.q.cuda(), _i32(self.table), _i32(self.start),
                                  cu_tokens=_i32(self.cu) if bounds else None, tree=tree, window=window,
                                  sinks=sinks, scale=scale)
        k, v = self.values()
        want, tol = att.attention(k, v, self.q, self.table, self.cu, self.start, words, window, sinks,
                                  scale or None, self.bits, skipped)
        ref.assert_within(got, want, tol, f"attention {what}")
        return got


SHAPES = [(64, 64, 2, 1), (128, 64, 2, 4), (64, 16, 1, 8), (128, 128, 1, 3), (128, 16, 2, 7), (64, 32, 1, 16),
          (128, 32, 1, 20), (64, 128, 1, 128)]


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("d,page,heads,group", SHAPES)
def test_single_tokens(d, page, heads, group, bits):
    """The last token of each sequence, the first of all among them."""
    start = [0, 1, 15, 16, page - 1, page, 3 * page + 5, 200]
    step = Step(1, d, page, heads, group, bits, start, [1] * len(start))
    step.check(bounds=False)
    for window, sinks in ((1, 0), (1, 3), (17, 0), (40, 4), (33, 130), (1000, 2)):
        step.check(window=window, sinks=sinks, bounds=False, what=f"window {window}, sinks {sinks}")
    assert bsa.device_status() == 0


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("d,page,heads,group", SHAPES)
def test_chunks(d, page, heads, group, bits):
    """Prompts in chunks of unlike lengths, none for one sequence."""
    start, new = [0, 7, page, 0, 130], [33, 0, 5, 150, 64]
    step = Step(2, d, page, heads, group, bits, start, new)
    step.check()
    for window, sinks in ((1, 0), (20, 4), (64, 0), (100, 70)):
        step.check(window=window, sinks=sinks, what=f"window {window}, sinks {sinks}")
    assert bsa.device_status() == 0


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("d,page,heads,group", SHAPES)
def test_trees(d, page, heads, group, bits):
    start, new = [0, 63, page, 250, 31], [5, 64, 1, 17, 33]
    step = Step(3, d, page, heads, group, bits, start, new)
    words = _trees(step.g, new)
    step.check(words)
    for window, sinks in ((3, 0), (2, 66), (70, 4), (1, 0)):
        step.check(words, window=window, sinks=sinks, what=f"window {window}, sinks {sinks}")
    # a chain of drafted tokens is the same as no tree
    chain = [w for n in new for w in att.tree_masks(range(-1, n - 1))]
    a, b = step.check(chain, what="chain"), step.check(what="no tree")
    assert torch.equal(a, b)
    assert bsa.device_status() == 0


@pytest.mark.parametrize("bits", [16, 8])
def test_trees_that_are_not_trees(bits):
    """Any words: no token seen (zeros without a prefix), tokens that come
    later, oneself not among them, bits past the last token."""
    start, new = [0, 40], [6, 64]
    step = Step(4, 64, 16, 1, 2, bits, start, new)
    words = [0, 1, 63, -1, 0b101000, 1 << 5] + torch.randint(-2 ** 62, 2 ** 62, (64,), generator=step.g).tolist()
    got = step.check(words)
    assert not got[0].any()
    step.check(words, window=5, sinks=2)
    step.check(words, window=30, sinks=0)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("group,new", [(1, 1), (8, 1), (4, 4), (4, 40)])
def test_one_long_sequence(bits, group, new):
    """Work split over many CTAs and joined; a ragged end."""
    step = Step(5, 128, 64, 1, group, bits, [5003], [new])
    step.check(bounds=False)
    step.check(window=2500, sinks=5, bounds=False)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("d,group", [(64, 4), (128, 4), (64, 12), (128, 12)])
@pytest.mark.parametrize("seqs,longest", [(300, 150), (100, 300), (40, 1000), (16, 4000)])
def test_many_sequences(seqs, longest, d, group, bits):
    """Small CTAs, alone and in clusters of two to eight."""
    g = torch.Generator().manual_seed(20)
    start = torch.randint(0, longest // 8, (seqs,), generator=g).tolist()
    start[seqs // 2] = longest
    step = Step(20, d, 16, 2, group, bits, start, [1] * seqs)
    step.check(bounds=False)
    step.check(window=longest // 3, sinks=3, bounds=False)
    assert bsa.device_status() == 0


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("d,group,new", [(64, 8, [20, 40]), (128, 8, [20, 40]), (64, 2, [1, 64]), (128, 5, [64, 64])])
def test_long_prefixes(d, group, new, bits):
    """The keys of a tile of rows dealt to clusters of CTAs, some of which see
    none of them in the shorter sequence; drafted trees and chains."""
    step = Step(21, d, 64, 1, group, bits, [6011, 90], new)
    step.check()
    step.check(_trees(step.g, new))
    step.check(window=3000, sinks=200)
    assert bsa.device_status() == 0


@pytest.mark.parametrize("new", [1, 40])
def test_masked_values_that_are_not_finite_in_clusters(new):
    step = Step(22, 64, 16, 1, 4, 16, [6000], [new])
    for j, bad in ((3, float("inf")), (4000, float("nan"))):
        step.v[step.table[0][j // 16], 0, j % 16, 5] = bad
    step.check(window=1500, sinks=2, bounds=False)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("new", [1, 24])
def test_positions_and_offsets_past_31_bits(bits, new):
    """The last pages of a pool of more than 2^32 elements, and of a table of
    2^24 pages; one more key than a sequence may have is reported."""
    page, d, heads = 128, 128, 2
    pool = (1 << 32) // (heads * page * d) + 7
    g = torch.Generator().manual_seed(23)
    if bits == 8:
        cache = bsa.PagedCache8.empty(pool, heads, page, d)
    else:
        cache = bsa.PagedCache.empty(pool, heads, page, d)
    most = (1 << 31) - 256
    width = -(-most // page) + 1
    table = torch.full((1, width), -7, dtype=torch.int32, device="cuda")
    start = most - new
    b0 = (start - 300) // page
    table[0, b0:most // page + 1] = torch.arange(pool - (most // page + 1 - b0), pool, dtype=torch.int32, device="cuda")
    rows = _randn(g, 300 + new, 2 * heads, d)
    at = _i32([start - 300])
    bsa.cache_append(cache, rows[:, :heads].cuda(), rows[:, heads:].cuda(), table, at)
    k, v = bsa.cache_read(cache, table, at, 300 + new)
    q = _randn(g, new, 4, d)
    out = bsa.paged_attention(cache, q.cuda(), table, _i32([start]), window=280)
    assert bsa.device_status() == 0
    if bits == 8:
        kv = [att.values(*att.quantise(x)) for x in (rows[:, :heads], rows[:, heads:])]
        for got, x in zip((k, v), (rows[:, :heads], rows[:, heads:])):
            c, s = att.quantise(x)
            assert torch.equal(got.cpu(), (c.float() * s[..., None]).bfloat16())
    else:
        kv = [rows[:, :heads], rows[:, heads:]]
        assert torch.equal(k.cpu(), kv[0]) and torch.equal(v.cpu(), kv[1])
    # the same step at the front of a small cache
    kk, vv = (torch.cat([x, x[:(-len(x)) % 16]]).view(-1, 16, heads, d).transpose(1, 2) for x in kv)
    want, tol = att.attention(kk, vv, q, [list(range(kk.shape[0]))], [0, new], [300], None, 280, 0, bits=bits)
    ref.assert_within(out, want, tol, "far")
    out.fill_(5.0)
    bsa.paged_attention(cache, q.cuda(), table, _i32([start + 1]), window=280, out=out)
    assert bsa.device_status() == 1 and (out == 5).all()


@pytest.mark.parametrize("bits", [16, 8])
def test_a_serving_run(bits):
    """Prompts in chunks, a fork with copy on write, drafted trees that are
    verified and cut back, decoding with and without selection, compaction: each
    result against plain references over the tokens that were appended."""
    g = torch.Generator().manual_seed(24)
    heads, group, d, page, pool = 2, 4, 64, 16, 40
    kind = bsa.PagedCache8 if bits == 8 else bsa.PagedCache
    cache, pages = kind.empty(pool, heads, page, d), bsa.PageTable(pool, page, 3, 12)
    said = [[], [], []]                          # every sequence's rows [k and v heads, d]

    def stand(rows):
        return att.values(*att.quantise(rows)) if bits == 8 else rows.double()

    def step(news, words=None, window=0, sinks=0):
        """Appends news[s] tokens and attends; returns their rows."""
        start = [len(x) for x in said]
        for s, n in enumerate(news):
            if n:
                pages.reserve(s, n)
        copies = pages.take_copies()
        if len(copies):
            bsa.copy_pages(cache, copies)
        table = _i32(pages.tables()[0])
        cu = np.cumsum([0] + news).tolist()
        qkv = _randn(g, cu[-1], (group + 2) * heads, d)
        on = qkv.cuda()
        hq = group * heads
        bsa.cache_append(cache, on[:, hq:hq + heads], on[:, hq + heads:], table, _i32(start), cu_tokens=_i32(cu))
        tree = None if words is None else torch.tensor(words, dtype=torch.int64, device="cuda")
        out = bsa.paged_attention(cache, on[:, :hq], table, _i32(start), cu_tokens=_i32(cu), tree=tree,
                                  window=window, sinks=sinks)
        for s in range(3):
            said[s] += list(qkv[cu[s]:cu[s + 1], hq:])
        # the same over caches of one page a sequence
        longest = max(map(len, said))
        k, v = torch.zeros(3, heads, longest, d, dtype=torch.float64), torch.zeros(3, heads, longest, d, dtype=torch.float64)
        for s, rows in enumerate(said):
            if rows:
                x = torch.stack(rows)
                k[s, :, :len(rows)] = stand(x[:, :heads]).transpose(0, 1)
                v[s, :, :len(rows)] = stand(x[:, heads:]).transpose(0, 1)
        want, tol = att.attention(k, v, qkv[:, :hq], [[0], [1], [2]], cu, start, words, window, sinks, bits=bits)
        ref.assert_within(out, want, tol, f"step of {news}")
        kk, vv = bsa.cache_read(cache, table, _i32([0, 0, 0]), sum(map(len, said)),
                                cu_tokens=_i32(np.cumsum([0] + [len(x) for x in said])))
        rows = torch.stack([r for x in said for r in x])
        assert torch.equal(kk.cpu(), stand(rows[:, :heads]).float().bfloat16())
        assert torch.equal(vv.cpu(), stand(rows[:, heads:]).float().bfloat16())
        return table

    step([37, 20, 0])
    step([5, 0, 0], window=16, sinks=2)
    pages.fork(0, 2)
    said[2] = list(said[0])
    step([1, 1, 1])                              # the forked page is copied before it grows
    words = att.tree_masks([-1, 0, 0, 1]) + att.tree_masks([-1, -1]) + att.tree_masks([-1, 0, 1, 1, 3, 0])
    step([4, 2, 6], words, window=30, sinks=4)
    for s, keep in enumerate((2, 0, 3)):         # drafts that were not taken
        n = len(said[s]) - (4, 2, 6)[s] + keep
        pages.truncate(s, n)
        said[s] = said[s][:n]
    step([1, 3, 1])
    pages.free(1)
    said[1] = []
    bsa.copy_pages(cache, pages.compact())
    table = step([2, 18, 1])
    lens = [len(x) for x in said]
    q = _randn(g, 3, group * heads, d)
    out, idx = bsa.paged_decode(cache, q.cuda(), table, _i32(lens), 2)
    k, v = (stand_cache(cache, x) for x in "kv")
    # the last blocks' means are those of their filled rows
    want, tol, ids = ref.decode(k, v, cache.kbar.cpu(), q, table.cpu(), lens, 2)
    assert torch.equal(idx.cpu(), ids)
    ref.assert_within(out, want, tol, "decode")
    assert bsa.device_status() == 0


def stand_cache(cache, name):
    """The values that a cache's pages hold, on the host."""
    x = getattr(cache, name).cpu()
    return att.values(x, getattr(cache, name + "_scale").cpu()) if x.dtype is torch.int8 else x


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("new", [1, 30])
def test_two_steps_at_once(bits, new):
    """Two streams with their own caches share nothing."""
    steps = [Step(25 + i, 64, 16, 2, 4, bits, [200 + 300 * i, 50], [new, new]) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in steps]
    held = [(s.cache(), s.q.cuda(), _i32(s.table), _i32(s.start)) for s in steps]
    want = [bsa.paged_attention(c, q, t, st).clone() for c, q, t, st in held]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for stream, (c, q, t, st) in zip(streams, held):
            with torch.cuda.stream(stream):
                got.append(bsa.paged_attention(c, q, t, st))
    torch.cuda.synchronize()
    for i, x in enumerate(got):
        assert torch.equal(x, want[i % 2])


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("d,page,heads,group", [(128, 64, 8, 2), (64, 16, 8, 3), (128, 128, 4, 5), (64, 32, 3, 16)])
def test_many_rows(d, page, heads, group, bits):
    """Enough rows that two tiles of them share their keys; the second may be
    short or missing."""
    start, new = [0, 100, 37, 513], [700, 128 // group * 3, 2 * (128 // group) * 3, 400]
    step = Step(17, d, page, heads, group, bits, start, new)
    step.check()
    for window, sinks in ((150, 0), (90, 4), (300, 140)):
        step.check(window=window, sinks=sinks, what=f"window {window}, sinks {sinks}")
    assert bsa.device_status() == 0


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("d,group,seqs", [(128, 4, 24), (64, 7, 20)])
def test_many_trees(d, group, seqs, bits):
    g = torch.Generator().manual_seed(18)
    start = torch.randint(0, 500, (seqs,), generator=g).tolist()
    new = [64] * (seqs - 3) + [1, 40, 64]
    step = Step(18, d, 32, 6, group, bits, start, new)
    step.check(_trees(step.g, new))
    step.check(_trees(step.g, new), window=70, sinks=5)
    assert bsa.device_status() == 0


def test_masked_values_that_are_not_finite_among_many_rows():
    step = Step(19, 64, 16, 8, 4, 16, [70], [900])
    for j, bad in ((3, float("inf")), (70, float("nan")), (500, float("-inf"))):
        step.v[step.table[0][j // 16], :, j % 16, 5] = bad
    got = bsa.paged_attention(step.cache(), step.q.cuda(), _i32(step.table), _i32([70]), window=101, sinks=3).cpu()
    seen = att.sight(70, 900, None, 101, 3)
    clean = step.v.clone()
    clean[~torch.isfinite(clean)] = 0.0
    want, tol = att.attention(step.k, clean, step.q, step.table, [0, 900], [70], None, 101, 3)
    hit = seen[:, 3] | seen[:, 70] | seen[:, 500]
    assert 100 < int(hit.sum()) < 800
    assert bool(torch.isfinite(got[~hit]).all()) and not bool(torch.isfinite(got[hit][..., 5]).any())
    ref.assert_within(got[~hit], want[~hit], tol[~hit], "rows that see none")
    ref.assert_within(got[hit][..., 6:], want[hit][..., 6:], tol[hit][..., 6:], "other channels")


@pytest.mark.parametrize("bits", [16, 8])
def test_mixed_batch(bits):
    """Single tokens, drafts and a prompt in one call, tokens before the first
    sequence and behind the last, which stay as they were."""
    start, new = [300, 0, 90, 511, 17], [1, 260, 4, 1, 16]
    step = Step(6, 64, 32, 2, 4, bits, start, new)
    lead = 3
    q = torch.cat([_randn(step.g, lead, 8, 64), step.q, _randn(step.g, 2, 8, 64)])
    out = torch.full(q.shape, 5.0, dtype=BF16, device="cuda")
    bsa.paged_attention(step.cache(), q.cuda(), _i32(step.table), _i32(start),
                        cu_tokens=_i32([c + lead for c in step.cu]), out=out)
    k, v = step.values()
    want, tol = att.attention(k, v, step.q, step.table, step.cu, start, bits=bits)
    ref.assert_within(out[lead:-2], want, tol, "mixed")
    assert (out[:lead] == 5).all() and (out[-2:] == 5).all() and bsa.device_status() == 0


@pytest.mark.parametrize("new", [2, 40, 100])
def test_masked_values_that_are_not_finite(new):
    """A key that some rows of a tile see and others do not: infinite or NaN
    values reach only those that see it."""
    step = Step(7, 64, 16, 1, 4, 16, [70], [new])
    page = 16
    for j, bad in ((3, float("inf")), (70, float("nan")), (70 + new // 2, float("-inf"))):
        step.v[step.table[0][j // page], 0, j % page, 5] = bad
    for window, sinks in ((60, 0), (1, 4), (new // 3 + 1, 0)):
        got = bsa.paged_attention(step.cache(), step.q.cuda(), _i32(step.table), _i32([70]), window=window,
                                  sinks=sinks).cpu()
        seen = att.sight(70, new, None, window, sinks)
        clean = step.v.clone()
        clean[~torch.isfinite(clean)] = 0.0
        want, tol = att.attention(step.k, clean, step.q, step.table, [0, new], [70], None, window, sinks)
        hit = seen[:, 3] | seen[:, 70] | seen[:, 70 + new // 2]
        assert bool(torch.isfinite(got[~hit]).all()) and not bool(torch.isfinite(got[hit][..., 5]).any())
        fine = torch.ones(64, dtype=torch.bool)
        fine[5] = False
        ref.assert_within(got[~hit], want[~hit], tol[~hit], "rows that see none")
        ref.assert_within(got[hit][..., fine], want[hit][..., fine], tol[hit][..., fine], "other channels")


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("new", [1, 50])
def test_masked_keys_that_are_not_finite(bits, new):
    """Keys before the window are never seen, whatever they hold."""
    step = Step(8, 64, 16, 1, 4, bits, [200], [new])
    for j in range(0, 100):
        at = (step.table[0][j // 16], 0, j % 16)
        if bits == 8:
            step.ks[at], step.vs[at] = float("nan"), float("nan")
        else:
            step.k[at], step.v[at] = float("nan"), float("inf")
    step.check(window=101 - new if new > 1 else 100, sinks=0, bounds=False)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("new", [1, 30])
def test_bad_pages(bits, new):
    step = Step(9, 64, 16, 2, 4, bits, [100, 33], [new, new], poison=False)
    step.table[0][2] = 10 ** 6
    step.table[1][0] = -1
    step.check(bounds=False, skipped=(10 ** 6, -1))
    assert bsa.device_status() == 3
    # pages that the window does not reach are not looked up
    step.check(window=16, bounds=False, skipped=(10 ** 6, -1))
    assert bsa.device_status() == 0


@pytest.mark.parametrize("new", [1, 64])
def test_sequences_that_make_no_sense(new):
    step = Step(10, 64, 16, 1, 2, 16, [10, 20, 30], [new] * 3)
    out = torch.full(step.q.shape, 5.0, dtype=BF16, device="cuda")
    for start, cu in (([10, -1, 30], None), ([10, 10 ** 6, 30], None)):
        bsa.paged_attention(step.cache(), step.q.cuda(), _i32(step.table), _i32(start), out=out)
        assert bsa.device_status() == 1
        assert (out[new:2 * new] == 5).all()
        k, v = step.values()
        want, tol = att.attention(k, v, step.q, step.table, step.cu, [10, 20, 30])
        for s in (0, 2):
            rows = slice(s * new, (s + 1) * new)
            ref.assert_within(out[rows], want[rows], tol[rows], "the others")
    for cu in ([0, 3 * new, new, 3 * new], [-1, 1, 2, 3], [0, 1, 2, 3 * new + 1]):
        bsa.paged_attention(step.cache(), step.q.cuda(), _i32(step.table), _i32([10, 20, 30]),
                            cu_tokens=_i32(cu))
        assert bsa.device_status() == 1


def test_a_tree_of_more_than_64_tokens_is_reported():
    step = Step(11, 64, 16, 1, 1, 16, [5], [65])
    out = torch.full(step.q.shape, 5.0, dtype=BF16, device="cuda")
    tree = torch.ones(65, dtype=torch.int64, device="cuda")
    bsa.paged_attention(step.cache(), step.q.cuda(), _i32(step.table), _i32([5]), tree=tree, out=out)
    assert bsa.device_status() == 1 and (out == 5).all()


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("new", [1, 48])
def test_strides_scale_and_growing_scores(bits, new):
    """Rows of a projection's output; scores that grow along the keys, so that
    the running maximum moves in every tile; a scale of one's own."""
    step = Step(12, 128, 64, 2, 3, bits, [700], [new])
    for b, at in enumerate(step.table[0]):
        if bits == 8:
            step.ks[at] *= 1.0 + 2.0 * b
        else:
            step.k[at] = (step.k[at].float() * (1.0 + 2.0 * b)).bfloat16()
    wide = torch.zeros(new, 8, 128, dtype=BF16, device="cuda")
    wide[:, 1:7] = step.q.cuda()
    got = bsa.paged_attention(step.cache(), wide[:, 1:7], _i32(step.table), _i32([700]), scale=0.3)
    k, v = step.values()
    want, tol = att.attention(k, v, step.q, step.table, step.cu, [700], scale=0.3, bits=bits)
    ref.assert_within(got, want, tol, "strided")


@pytest.mark.parametrize("new", [1, 40])
def test_scales_of_every_size(new):
    """8-bit pages: scales and queries over many orders; the largest weights
    come late, and early."""
    g = torch.Generator().manual_seed(13)
    cases = [(0, 0, 0, 1.0), (-40, 40, 60, 2.0 ** 25), (60, -60, -100, 2.0 ** -30), (-100, 90, 80, 2.0 ** 12),
             (30, -30, -126, 2.0 ** 30), (0, 0, 0, 0.0)]
    step = Step(13, 64, 16, 1, 2, 8, [150] * len(cases), [new] * len(cases))
    for s, (a, b, c, late) in enumerate(cases):
        pages = step.table[s]
        step.ks[pages] *= 2.0 ** a
        step.vs[pages] *= 2.0 ** c
        step.vs[pages[5:]] *= late
        step.q[step.cu[s]:step.cu[s + 1]] *= 2.0 ** b
    step.check(bounds=False)


def test_an_empty_step():
    step = Step(14, 64, 16, 1, 1, 16, [5], [1])
    q = torch.empty(0, 1, 64, dtype=BF16, device="cuda")
    out = bsa.paged_attention(step.cache(), q, _i32(step.table), _i32([5]))
    assert out.shape == (0, 1, 64) and bsa.device_status() == 0


def test_refusals():
    step = Step(15, 64, 16, 1, 2, 16, [5], [2])
    c, q, t, s = step.cache(), step.q.cuda(), _i32(step.table), _i32([5])
    for kw in (dict(window=-1), dict(window=3, sinks=-1)):
        with pytest.raises(bsa.BsaError):
            bsa.paged_attention(c, q, t, s, **kw)
    for kw in (dict(sinks=2), dict(out=q.float()), dict(window=2.5)):
        with pytest.raises(ValueError):
            bsa.paged_attention(c, q, t, s, **kw)
    with pytest.raises(TypeError):
        bsa.paged_attention(c, q, t, s, tree=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(bsa.BsaError):
        bsa.paged_attention(c, q, t, s, out=q)
    with pytest.raises(ValueError):
        bsa.paged_attention(c, q.requires_grad_(), t, s)
    with torch.no_grad():
        bsa.paged_attention(c, q, t, s)
    assert bsa.device_status() == 0


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("new", [1, 24])
def test_a_captured_step_follows_its_buffers(bits, new):
    """Append, attend and read back captured once and replayed with other
    tokens and lengths, on a stream of its own."""
    step = Step(16, 64, 16, 2, 4, bits, [40, 77], [new, new], poison=False, width=16)
    cache = step.cache()
    g = step.g
    fresh = [_randn(g, 2 * new, 12, 64) for _ in range(2)]
    starts = [[40, 77], [100, 3]]
    qkv, start, table = fresh[0].cuda(), _i32(starts[0]), _i32(step.table)
    out = torch.empty(2 * new, 8, 64, dtype=BF16, device="cuda")
    back = torch.empty(2, 2 * new, 2, 64, dtype=BF16, device="cuda")

    def go():
        bsa.cache_append(cache, qkv[:, 8:10], qkv[:, 10:], table, start)
        bsa.paged_attention(cache, qkv[:, :8], table, start, window=60, sinks=2, out=out)
        bsa.cache_read(cache, table, start, 2 * new, out=(back[0], back[1]))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for x, st in zip(reversed(fresh), reversed(starts)):
        qkv.copy_(x)
        start.copy_(_i32(st))
        graph.replay()
        if bits == 8:
            k, v = (att.values(a.cpu(), b.cpu()) for a, b in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
        else:
            k, v = cache.k.cpu(), cache.v.cpu()
        want, tol = att.attention(k, v, x[:, :8], step.table, step.cu, st, None, 60, 2, bits=bits)
        ref.assert_within(out, want, tol, "replayed")
        for i, (rows, name) in enumerate(((x[:, 8:10], "k"), (x[:, 10:], "v"))):
            codes, scale = att.quantise(rows)
            want = (codes.float() * scale[..., None]).bfloat16() if bits == 8 else rows
            assert torch.equal(back[i].cpu(), want), name
    assert bsa.device_status() == 0
