"""8-bit pages on the GPU: the scale of a key counts only in the rows that see
the key, however large it is.  Every row is held to a bound made of the keys
that it sees itself."""
import math

import pytest
import torch

from content_dependent_block_gb300 import _build, bsa
from tests import attention_reference as att
from tests import paged_reference as ref
from tests.test_gpu_paged_attention import Step, _i32, _randn

pytestmark = pytest.mark.gpu

HUGE = (2.0 ** 40, 2.0 ** 100)          # beside scales of 0.01 to 0.03


@pytest.fixture(scope="module", autouse=True)
def _lib():
    _build.build()


@pytest.fixture(autouse=True)
def _clean_status():
    bsa.device_status()
    yield
    torch.cuda.synchronize()


def _row(kk, vv, vs, q):
    """(out, tol) [d] fp64 of one row over the keys it sees, kk, vv [n, d] and
    the scales of vv: the bounds of attention_reference.attention, of these keys
    alone.  A weight enters the product as p vs 2^(s - E), E the exponent of the
    largest vs and s at least 6, in fp16; below 2^-14 that is off by 2^-25, so
    the output by 2^-25 2^(E - s) |c| <= 2^-31 127 max vs for the key, in any
    channel (also in one where the key with the largest scale has code 0)."""
    n, d = kk.shape
    if n == 0:
        return torch.zeros(d, dtype=torch.float64), torch.zeros(d, dtype=torch.float64)
    scale = 1.0 / math.sqrt(d)
    w = torch.softmax(kk @ q * scale, 0)
    o, size = w @ vv, w @ vv.abs()
    slip = float((kk.abs() @ q.abs()).amax()) * scale * (d + 6) * 2.0 ** -24
    rel = 2.0 ** -11 + 2 * slip + 2.0 ** -20 + 2 * n * 2.0 ** -24
    t = rel * size * 1.01 + n * 2.0 ** -31 * 127 * vs.double().amax()
    return o, t + 2.0 ** -8 * (o.abs() + t)


def _check(step, words, window, sinks, what):
    """One sequence, one cache head."""
    start, n, group = step.start[0], step.new[0], step.q.shape[1]
    tree = None if words is None else torch.tensor(words, dtype=torch.int64, device="cuda")
    got = bsa.paged_attention(step.cache(), step.q.cuda(), _i32(step.table), _i32(step.start), tree=tree,
                              window=window, sinks=sinks)
    k, v = step.values()
    kk, vv = (x[step.table[0], 0].reshape(-1, x.shape[-1])[:start + n] for x in (k, v))
    vs = step.vs[step.table[0], 0].reshape(-1)[:start + n]
    seen = att.sight(start, n, words, window, sinks)
    want = [[_row(kk[seen[i]], vv[seen[i]], vs[seen[i]], step.q[i, h].double()) for h in range(group)]
            for i in range(n)]
    want, tol = (torch.stack([torch.stack([x[j] for x in row]) for row in want]) for j in (0, 1))
    ref.assert_within(got, want, tol, what)
    assert bsa.device_status() == 0


def _step(seed, d, group, start, new, keys, huge, page=16):
    step = Step(seed, d, page, 1, group, 8, [start], [new])
    for j in keys:
        step.vs[step.table[0][j // page], 0, j % page] = huge
    return step


FEW = [(1, 1), (1, 8), (3, 4), (4, 4)]          # new tokens, heads: few rows


@pytest.mark.parametrize("huge", HUGE)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [1, 16, 100])
@pytest.mark.parametrize("new,group", FEW)
def test_keys_before_a_window(new, group, window, d, huge):
    """Keys that no row sees, in the tile where the window begins."""
    step = _step(40, d, group, 203, new, range(203 + 1 - window), huge)
    _check(step, None, window, 0, f"window {window}")


@pytest.mark.parametrize("huge", HUGE)
@pytest.mark.parametrize("new,group", FEW)
def test_keys_behind_the_sinks(new, group, huge):
    step = _step(41, 64, group, 300, new, range(3, 300 + 1 - 20), huge)
    _check(step, None, 20, 3, "sinks")


@pytest.mark.parametrize("huge", HUGE)
@pytest.mark.parametrize("new,group", [(3, 4), (4, 4), (4, 1)])
def test_drafts_that_nobody_sees(new, group, huge):
    """The second draft is seen by no token, itself among them."""
    words = [w & ~2 for w in att.tree_masks(range(-1, new - 1))]
    step = _step(42, 64, group, 37, new, [38], huge)
    _check(step, words, 0, 0, "draft")
    _check(step, words, 9, 1, "draft in a window")


@pytest.mark.parametrize("huge", HUGE)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,group", [(3, 4), (4, 2)])
def test_keys_that_other_rows_see(new, group, d, huge):
    """Branches of a tree, and tokens whose window has passed a key: rows that
    see it and rows that do not share a tile."""
    words = [1 << i for i in range(new)]
    step = _step(43, d, group, 90, new, [91], huge)
    _check(step, words, 0, 0, "branches")
    step = _step(44, d, group, 90, new, [90 - 20 + 2], huge)
    _check(step, None, 20, 0, "window")


@pytest.mark.parametrize("huge", HUGE)
@pytest.mark.parametrize("page,seqs", [(16, 3), (64, 40)])
@pytest.mark.parametrize("d", [64, 128])
def test_decoding_heads_that_select_unlike_blocks(d, page, seqs, huge):
    """Two heads of a cache head pick a block each; the scales of one's count
    nothing for the other."""
    g = torch.Generator().manual_seed(45)
    blocks = 4
    k, v = (torch.randint(-127, 128, (seqs * blocks, 1, page, d), generator=g).to(torch.int8) for _ in range(2))
    ks, vs = (0.01 + 0.02 * torch.rand(seqs * blocks, 1, page, generator=g) for _ in range(2))
    table = torch.arange(seqs * blocks).view(seqs, blocks)
    kbar = torch.zeros(seqs * blocks, 1, d)
    kbar[table[:, 1], 0, 0], kbar[table[:, 2], 0, 0] = 4.0, -4.0
    vs[table[:, 1]] = huge
    q = _randn(g, seqs, 2, d)
    q[:, 0, 0], q[:, 1, 0] = 1.0, -1.0                  # head 0: block 1, head 1: block 2
    cache = bsa.PagedCache8(*(x.cuda() for x in (k, v, ks, vs, kbar)))
    out, idx = bsa.paged_decode(cache, q.cuda(), _i32(table), _i32([blocks * page] * seqs), 1, local_block=False)
    assert idx.cpu().tolist() == [[[1], [2]]] * seqs
    kk, vv = att.values(k, ks), att.values(v, vs)
    want = [[_row(*(x[table[s, 1 + h], 0] for x in (kk, vv, vs)), q[s, h].double()) for h in range(2)]
            for s in range(seqs)]
    want, tol = (torch.stack([torch.stack([x[j] for x in row]) for row in want]) for j in (0, 1))
    ref.assert_within(out, want, tol, "decode")
    assert bsa.device_status() == 0


MANY = [(40, 1), (40, 4), (64, 2), (1, 24)]             # many rows


@pytest.mark.parametrize("huge", HUGE)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,group", MANY)
def test_many_rows(new, group, d, huge):
    """The same with tiles of 128 rows."""
    for window in (1, 16, 100):
        step = _step(46, d, group, 203, new, range(203 + 1 - window), huge)
        _check(step, None, window, 0, f"window {window}")
    step = _step(47, d, group, 300, new, range(3, 300 + 1 - 20), huge)
    _check(step, None, 20, 3, "sinks")
    words = [w & ~2 for w in att.tree_masks(range(-1, new - 1))]
    step = _step(48, d, group, 37, new, [38] if new > 1 else [], huge)
    _check(step, words, 0, 0, "a draft that nobody sees")
    _check(step, att.tree_masks([-1] * new), 0, 0, "branches")
    step = _step(49, d, group, 90, new, [90 - 20 + new // 2] if new > 1 else [], huge)
    _check(step, None, 20, 0, "a key that the window of half of the tokens has passed")


@pytest.mark.parametrize("huge", HUGE)
@pytest.mark.parametrize("d", [64, 128])
def test_many_rows_over_many_tiles(d, huge):
    """Pairs of tiles, long prefixes dealt to a cluster, keys of the edge of a
    window seen by some rows only."""
    step = _step(50, d, 4, 700, 150, [600, 640, 720, 800], huge)
    _check(step, None, 130, 2, "window")
    step = _step(51, d, 4, 5000, 40, [5003, 5010], huge)
    words = att.tree_masks([-1] + [(i - 1) // 2 for i in range(1, 40)])
    _check(step, words, 0, 0, "tree")
    _check(step, words, 3000, 5, "tree in a window")
