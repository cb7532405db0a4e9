"""Host side of the rotary positions and of the paged cache: refusals,
frequencies and their table, and the page manager against a model."""
import ctypes
import math
import random

import numpy as np
import pytest

from content_dependent_block_gb300 import _build, bsa
from tests import paged_reference as ref

FAKE = ctypes.c_void_p(0x100000)          # aligned, never dereferenced
OTHER = ctypes.c_void_p(0x40000000)
MISALIGNED = ctypes.c_void_p(0x100008)
ODD = ctypes.c_void_p(0x100002)


@pytest.fixture(scope="module")
def L():
    _build.build()
    return bsa.lib()


# ------------------------------------------------------------- frequencies
@pytest.mark.parametrize("rot,kw", [
    (64, {}), (128, dict(theta=500000.0)), (2, {}), (34, dict(scaling="linear", factor=4.0)),
    (64, dict(scaling="base", factor=8.0)), (32, dict(scaling="parts", factor=4.0, original=8192.0)),
    (128, dict(scaling="parts", factor=32.0, original=4096.0, low=1.0, high=4.0)),
])
def test_frequencies_follow_the_formula(L, rot, kw):
    p = bsa.RopeParams(rot, bsa.ROPE_SCALING[kw.get("scaling", "none")], kw.get("theta", 10000.0),
                       kw.get("factor", 1.0), kw.get("original", 0.0), kw.get("low", 1.0),
                       kw.get("high", 32.0))
    got = np.empty(rot // 2)
    assert L.bsa_rope_frequencies(p, got.ctypes.data_as(ctypes.c_void_p)) == 0
    want = ref.inv_freq(rot, **kw).numpy()
    np.testing.assert_allclose(got, want, rtol=1e-14)


def test_table_holds_turns_modulo_one(L):
    f = np.array([1.0, 0.5, 2 * math.pi, 7.25, 1e-9, 0.0, -0.3, 1000.0, -1e-25])
    t = np.empty(f.size, dtype=np.uint64)
    assert L.bsa_rope_table(f.ctypes.data_as(ctypes.c_void_p), f.size,
                            t.ctypes.data_as(ctypes.c_void_p)) == 0
    for x, u in zip(f, t):
        want = (x / (2 * math.pi)) % 1.0
        got = int(u) / 2.0 ** 64
        off = abs(got - want)
        assert min(off, 1 - off) <= 2.0 ** -52 * max(1.0, abs(x)), (x, got, want)


@pytest.mark.parametrize("p,code", [
    (bsa.RopeParams(3, 0, 1e4, 1, 0, 0, 0), 1), (bsa.RopeParams(0, 0, 1e4, 1, 0, 0, 0), 1),
    (bsa.RopeParams(64, 0, 0.0, 1, 0, 0, 0), 1), (bsa.RopeParams(64, 0, math.nan, 1, 0, 0, 0), 1),
    (bsa.RopeParams(64, 4, 1e4, 1, 0, 0, 0), 1), (bsa.RopeParams(64, 1, 1e4, 0.0, 0, 0, 0), 1),
    (bsa.RopeParams(64, 3, 1e4, 2, 0.0, 1, 32), 1), (bsa.RopeParams(64, 3, 1e4, 2, 4096, 4, 4), 1),
    (bsa.RopeParams(2, 2, 1e4, 2, 0, 0, 0), 1),
])
def test_bad_frequencies_are_refused(L, p, code):
    assert L.bsa_rope_frequencies(p, (ctypes.c_double * 64)()) == code
    assert L.bsa_last_error() != b""


def test_bad_tables_are_refused(L):
    out = (ctypes.c_uint64 * 4)()
    assert L.bsa_rope_frequencies(bsa.RopeParams(64, 0, 1e4, 1, 0, 0, 0), None) == 1
    assert L.bsa_rope_table(None, 4, out) == 1
    assert L.bsa_rope_table((ctypes.c_double * 4)(), 0, out) == 1
    assert L.bsa_rope_table((ctypes.c_double * 4)(1.0, math.inf), 4, out) == 1
    assert L.bsa_rope_table((ctypes.c_double * 4)(1.0, 2e6), 4, out) == 1


# ----------------------------------------------------------------- refusals
def _rope(L, shape=None, x=FAKE, xs=None, pos=None, rot=None, out=OTHER, os=None):
    shape = shape or bsa.Heads(2, 8, 4, 64, bsa.BF16)
    n, h, d = shape.n, shape.heads, shape.d
    st = bsa.Strides(h * n * d, n * d, d)
    rot = rot or bsa.Rotation(0x200000, 64, 0, 1.0)
    return [f(shape, x, xs or st, pos, 0, rot, out, os or st, None)
            for f in (L.bsa_rope, L.bsa_rope_backward)]


@pytest.mark.parametrize("kw,code", [
    (dict(shape=bsa.Heads(0, 8, 4, 64, 0)), 1), (dict(shape=bsa.Heads(1, 8, 0, 64, 0)), 1),
    (dict(shape=bsa.Heads(1, 8, 4, 96, 0)), 2), (dict(shape=bsa.Heads(1, 8, 4, 64, 2)), 1),
    (dict(x=None), 1), (dict(x=MISALIGNED), 7), (dict(out=None), 1), (dict(pos=ODD), 7),
    (dict(rot=bsa.Rotation(0x200000, 63, 0, 1.0)), 1), (dict(rot=bsa.Rotation(0x200000, 66, 0, 1.0)), 1),
    (dict(rot=bsa.Rotation(0x200000, 0, 0, 1.0)), 1), (dict(rot=bsa.Rotation(None, 64, 0, 1.0)), 1),
    (dict(rot=bsa.Rotation(0x200004, 64, 0, 1.0)), 7),
    (dict(rot=bsa.Rotation(0x200000, 64, 0, math.inf)), 1),
    (dict(xs=bsa.Strides(2048, 512, -64)), 2), (dict(xs=bsa.Strides(2048, 512, 68)), 7),
    (dict(os=bsa.Strides(2048, 512, 0)), 1), (dict(os=bsa.Strides(1024, 512, 64)), 1),
    (dict(os=bsa.Strides(2048, 512, 32)), 1),
    (dict(shape=bsa.Heads(1, 1 << 41, 1, 64, 0)), 2),
    # out is x shifted, or x with other strides
    (dict(out=ctypes.c_void_p(0x100010)), 1), (dict(out=FAKE, os=bsa.Strides(2048, 64, 256)), 1),
])
def test_rope_refusals(L, kw, code):
    assert _rope(L, **kw) == [code, code], L.bsa_last_error()


def _cache(**kw):
    c = dict(k=0x100000, v=0x4000000, kbar=0x8000000, num_pages=8, heads=2, page=64, d=64)
    c.update(kw)
    return bsa.Cache(*[c[x] for x in ("k", "v", "kbar", "num_pages", "heads", "page", "d")])


BAD_CACHES = [(dict(d=96), 2), (dict(page=48), 2), (dict(page=0), 2), (dict(num_pages=0), 1),
              (dict(heads=0), 1), (dict(heads=70000), 2), (dict(k=None), 1), (dict(v=0x4000008), 7),
              (dict(kbar=None), 1), (dict(num_pages=1 << 31), 2)]


@pytest.mark.parametrize("bad,code", BAD_CACHES)
def test_bad_caches_are_refused(L, bad, code):
    c = _cache(**bad)
    assert L.bsa_cache_append(c, FAKE, 128, FAKE, 128, 4, 4, None, FAKE, FAKE, 4, None) == code
    assert L.bsa_cache_copy_pages(c, FAKE, 1, None) == code
    assert L.bsa_paged_decode(c, FAKE, 1 << 20, 4, max(1, c.heads), FAKE, 4, 4, None, FAKE, 4, None,
                              0.0, FAKE, None, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), 1), (dict(v=MISALIGNED), 7), (dict(ks=64), 1), (dict(vs=132), 7),
    (dict(tokens=-1), 1), (dict(seqs=0), 1), (dict(width=0), 1), (dict(tokens=5), 1),
    (dict(cu=ODD), 7), (dict(start=None), 1), (dict(table=ODD), 7), (dict(ks=1 << 31), 2),
    (dict(tokens=1 << 31, cu=FAKE), 2), (dict(tokens=0), 0),
])
def test_append_refusals(L, kw, code):
    a = dict(k=FAKE, ks=128, v=FAKE, vs=128, tokens=4, seqs=4, cu=None, start=FAKE, table=FAKE, width=4)
    a.update(kw)
    assert L.bsa_cache_append(_cache(), a["k"], a["ks"], a["v"], a["vs"], a["tokens"], a["seqs"],
                              a["cu"], a["start"], a["table"], a["width"], None) == code


def test_copy_refusals(L):
    assert L.bsa_cache_copy_pages(_cache(), None, 1, None) == 1
    assert L.bsa_cache_copy_pages(_cache(), ODD, 1, None) == 7
    assert L.bsa_cache_copy_pages(_cache(), FAKE, -1, None) == 1
    assert L.bsa_cache_copy_pages(_cache(), None, 0, None) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(q=MISALIGNED), 7), (dict(qs=192), 1), (dict(qs=258), 7),
    (dict(tokens=0), 0), (dict(tokens=-1), 1), (dict(heads=5), 1), (dict(heads=0), 1),
    (dict(heads=2 * 129), 2),
    (dict(topk=0), 2), (dict(topk=33), 2), (dict(width=16385), 2), (dict(width=0), 1),
    (dict(seqs=3), 1), (dict(seqs=0, ts=FAKE), 1), (dict(table=None), 1), (dict(lens=None), 1),
    (dict(ts=ODD), 7), (dict(idx=ODD), 7), (dict(out=None), 1), (dict(scale=math.nan), 1),
])
def test_decode_refusals(L, kw, code):
    a = dict(q=FAKE, qs=256, tokens=4, heads=4, table=FAKE, width=4, seqs=4, ts=None, lens=FAKE, topk=2,
             scale=0.0, out=FAKE, idx=None)
    a.update(kw)
    if a["heads"] > 4:
        a["qs"] = a["heads"] * 64
    assert L.bsa_paged_decode(_cache(), a["q"], a["qs"], a["tokens"], a["heads"], a["table"], a["width"],
                              a["seqs"], a["ts"], a["lens"], a["topk"], None, a["scale"], a["out"],
                              a["idx"], None) == code, L.bsa_last_error()


def test_tensors_that_overlap_are_refused(L):
    """New rows inside the cache, an output on its queries or inside the cache."""
    c = _cache()
    inside = [c.k, c.k + 8 * 2 * 64 * 64 * 2 - 16, c.v, c.kbar + 8 * 2 * 64 * 4 - 16]
    for p in inside:
        p = ctypes.c_void_p(p)
        assert L.bsa_cache_append(c, p, 128, OTHER, 128, 4, 4, None, FAKE, FAKE, 4, None) == 1
        assert L.bsa_cache_append(c, OTHER, 128, p, 128, 4, 4, None, FAKE, FAKE, 4, None) == 1
        assert L.bsa_paged_decode(c, OTHER, 256, 4, 4, FAKE, 4, 4, None, FAKE, 2, None, 0.0, p, None,
                                  None) == 1
        assert b"overlap" in L.bsa_last_error()
    for shift in (0, 16, 4 * 256 * 2 - 16):
        out = ctypes.c_void_p(OTHER.value + shift)
        assert L.bsa_paged_decode(c, OTHER, 256, 4, 4, FAKE, 4, 4, None, FAKE, 2, None, 0.0, out, None,
                                  None) == 1


def test_copies_from_the_host_must_not_chain():
    import torch
    c = type("C", (), {"k": torch.zeros(1)})()
    for pairs in ([[0, 1], [2, 1]], [[0, 1], [1, 2]], [[3, 3]]):
        with pytest.raises(ValueError):
            bsa.copy_pages(c, np.array(pairs, dtype=np.int32))


# ------------------------------------------------------------- page manager
def test_page_table_refusals(L):
    h = ctypes.c_void_p()
    assert L.bsa_pages_create(0, 64, 1, 1, ctypes.byref(h)) == 1 and not h
    assert L.bsa_pages_create(4, 48, 1, 1, ctypes.byref(h)) == 2
    assert L.bsa_pages_create(4, 64, 0, 1, ctypes.byref(h)) == 1
    assert L.bsa_pages_create(4, 64, 1, 0, ctypes.byref(h)) == 1
    assert L.bsa_pages_create(4, 64, 1, 1, None) == 1
    assert L.bsa_pages_destroy(None) == 0
    assert L.bsa_pages_reserve(None, 0, 1) == 1 and L.bsa_pages_free_pages(None) == -1
    n = ctypes.c_int64()
    assert L.bsa_pages_take_copies(None, None, 0, ctypes.byref(n)) == 1
    assert L.bsa_pages_compact(None, None, 0, ctypes.byref(n)) == 1
    assert L.bsa_pages_tables(None, None, None) == 1
    t = bsa.PageTable(4, 16, 2, 3)
    for call in (lambda: t.reserve(2, 1), lambda: t.reserve(-1, 1), lambda: t.reserve(0, -1),
                 lambda: t.reserve(0, 1 << 31), lambda: t.fork(0, 0), lambda: t.fork(0, 5),
                 lambda: t.truncate(0, 1)):
        with pytest.raises(bsa.BsaError) as e:
            call()
        assert e.value.code == 1
    with pytest.raises(bsa.BsaError) as e:          # the table holds three pages
        t.reserve(0, 49)
    assert e.value.code == 4 and t.free_pages == 4
    t.reserve(0, 48)
    with pytest.raises(bsa.BsaError) as e:          # one page is left
        t.reserve(1, 17)
    assert e.value.code == 4 and t.free_pages == 1 and t.tables()[1].tolist() == [48, 0]
    t.fork(0, 1)
    with pytest.raises(bsa.BsaError) as e:          # not an empty sequence
        t.fork(0, 1)
    assert e.value.code == 1
    t.truncate(0, 40)
    t.reserve(0, 1)                                 # a copy is queued
    with pytest.raises(bsa.BsaError) as e:
        t.compact()
    assert e.value.code == 1
    assert L.bsa_pages_take_copies(t._h, (ctypes.c_int32 * 2)(), 0, ctypes.byref(n)) == 4
    assert t.take_copies().shape == (1, 2) and t.take_copies().shape == (0, 2)


class Model:
    """Every token is a number; pages hold what the copies and appends put."""

    def __init__(self, pages, page):
        self.mem = np.full((pages, page), -1, dtype=np.int64)
        self.page = page

    def copy(self, pairs):
        targets = [p for _, p in pairs.tolist()]
        sources = [p for p, _ in pairs.tolist()]
        assert len(set(targets)) == len(targets) and not set(targets) & set(sources)
        self.mem[targets] = self.mem[sources]


@pytest.mark.parametrize("seed", range(8))
def test_page_table_against_a_model(L, seed):
    """Random reserves, forks, truncations and compactions; tokens are appended
    only after the queued copies ran, and every sequence reads back its own."""
    rng = random.Random(seed)
    page, pool, seqs, width = 16, rng.choice([12, 30, 64]), 6, 9
    t, m = bsa.PageTable(pool, page, seqs, width), Model(pool, page)
    want = [[] for _ in range(seqs)]
    stamp = 0

    def check():
        table, lens = t.tables()
        held = set()
        for s in range(seqs):
            assert lens[s] == len(want[s])
            used = -(-len(want[s]) // page)
            assert (table[s, used:] == -1).all()
            got = [m.mem[table[s, i // page], i % page] for i in range(len(want[s]))]
            assert got == want[s]
            held |= set(table[s, :used].tolist())
        assert t.free_pages == pool - len(held)

    for _ in range(150):
        grown = []
        for _ in range(rng.randint(1, 4)):           # a step: several of these, then the copies
            s = rng.randrange(seqs)
            what = rng.random()
            pending = {x for x, _, _ in grown}
            if what < 0.5:
                n = rng.choice([1, 1, 2, 5, 16, 33])
                try:
                    t.reserve(s, n)
                    grown.append((s, len(want[s]), n))
                    want[s] = want[s] + list(range(stamp, stamp + n))
                    stamp += n
                except bsa.BsaError as e:
                    assert e.code == 4
            elif what < 0.7:
                empty = [x for x in range(seqs) if not want[x]]
                if empty and s != empty[0] and s not in pending:
                    t.fork(s, empty[0])
                    want[empty[0]] = list(want[s])
            elif s not in pending:
                n = rng.choice([0, len(want[s]) // 2, max(0, len(want[s]) - 1)])
                t.truncate(s, n)
                want[s] = want[s][:n]
        m.copy(t.take_copies())
        table, _ = t.tables()
        for s, at, n in grown:
            for i in range(at, at + n):
                m.mem[table[s, i // page], i % page] = want[s][i]
        check()
        if rng.random() < 0.2:
            pairs = t.compact()
            assert len(pairs) <= pool // 2
            m.copy(pairs)
            check()
            table, _ = t.tables()
            assert table.max() < pool - t.free_pages


def test_a_queued_copy_keeps_its_source_and_forgets_a_dropped_target(L):
    t = bsa.PageTable(6, 16, 4, 4)
    t.reserve(0, 20)                       # two pages, the second partly filled
    last = int(t.tables()[0][0, 1])
    t.fork(0, 1)
    t.reserve(1, 1)                        # splits the shared page: a copy from `last`
    t.free(0)                              # nobody but the queue holds `last`
    free = t.free_pages
    t.reserve(2, 16 * free)                # everything that is free
    assert last not in t.tables()[0][2].tolist()
    t.fork(1, 3)                           # shares the page that is still to be written
    t.free(2)
    t.reserve(3, 1)                        # splits again: reads the first source
    pairs = t.take_copies()
    assert len(pairs) == 2 and (pairs[:, 0] == last).all() and len(set(pairs[:, 1])) == 2
    t.free(3)
    t.reserve(0, 1)
    t.fork(0, 2)
    t.reserve(2, 1)
    t.free(2)                              # the copy's target is gone again
    assert len(t.take_copies()) == 0
    t.free(0)
    t.free(1)
    assert t.free_pages == 6
