"""The page manager's order of forks, reserves and appends, on the host."""
import ctypes
import random

import numpy as np
import pytest
import torch

from content_dependent_block_gb300 import _build, bsa


@pytest.fixture(scope="module")
def L():
    _build.build()
    return bsa.lib()


def refused(call):
    with pytest.raises(bsa.BsaError) as e:
        call()
    return e.value.code


# -------------------------------------------- forks between reserve and append
@pytest.mark.parametrize("first,then", [(20, 1), (10, 3), (0, 5), (16, 1)])
@pytest.mark.parametrize("grows", [0, 1])
def test_a_copy_that_would_miss_reserved_tokens_is_refused(L, first, then, grows):
    """`then` tokens reserved and not appended, a fork, and one of the two grows:
    the copy runs before the append, so the other would never get the tokens."""
    t = bsa.PageTable(8, 16, 3, 4)
    t.reserve(0, first)
    t.take_copies()
    t.reserve(0, then)
    t.fork(0, 1)
    t.reserve(grows, 1)
    assert refused(t.take_copies) == 1
    n = ctypes.c_int64()
    pair = (ctypes.c_int32 * 2)()
    assert L.bsa_pages_take_copies(t._h, pair, 1, ctypes.byref(n)) == 1 and n.value == 1
    assert refused(t.compact) == 1                      # still queued
    if grows == 1:
        t.free(1)                                       # the way out: fork after the append
        assert len(t.take_copies()) == 0
        t.fork(0, 1)
        t.reserve(1, 1)
        assert len(t.take_copies()) == 1
    else:
        t.tables()                                      # or: they are appended by now
        assert len(t.take_copies()) == 1


def test_forks_before_the_reserve_and_after_the_append_are_served(L):
    t = bsa.PageTable(12, 16, 4, 4)
    t.reserve(0, 20)
    assert len(t.take_copies()) == 0                    # appended after this
    t.fork(0, 1)
    t.reserve(0, 1)
    t.reserve(1, 2)
    assert len(t.take_copies()) == 1
    t.fork(1, 2)
    t.fork(1, 3)
    t.reserve(2, 1)
    t.reserve(3, 1)
    t.reserve(1, 1)
    assert len(t.take_copies()) == 2
    # a fork that does not grow before the append shares what is appended
    t.reserve(0, 1)
    t.free(3)
    t.fork(0, 3)
    assert len(t.take_copies()) == 0
    t.reserve(3, 1)
    assert len(t.take_copies()) == 1


def test_a_fork_cut_back_to_written_rows_may_grow(L):
    t = bsa.PageTable(8, 16, 3, 4)
    t.reserve(0, 20)
    t.take_copies()
    t.reserve(0, 3)
    t.fork(0, 1)
    t.truncate(1, 20)
    t.reserve(1, 1)
    assert len(t.take_copies()) == 1


def test_reserved_rows_move_with_a_compaction(L):
    t = bsa.PageTable(8, 16, 4, 4)
    t.reserve(2, 32)
    t.reserve(0, 4)
    t.take_copies()
    t.reserve(0, 2)
    t.free(2)
    assert len(t.compact()) == 1                        # sequence 0's page goes down
    t.fork(0, 1)
    t.reserve(1, 1)
    assert refused(t.take_copies) == 1


@pytest.mark.parametrize("seed", range(24))
def test_page_table_against_a_model_in_any_order(L, seed):
    """Reserves, forks and truncations of any sequences in any order within a
    step; a token is appended once, through a sequence that has it, after the
    copies.  A refused step frees its forks.  Every sequence reads back its own."""
    rng = random.Random(seed)
    page, pool, seqs, width = 16, rng.choice([24, 40, 64]), 6, 9
    t, mem = bsa.PageTable(pool, page, seqs, width), np.full((pool, page), -1, dtype=np.int64)
    want = [[] for _ in range(seqs)]
    stamp, refusals = 0, 0

    def copy(pairs):
        targets, sources = [p for _, p in pairs.tolist()], [p for p, _ in pairs.tolist()]
        assert len(set(targets)) == len(targets) and not set(targets) & set(sources)
        mem[targets] = mem[sources]

    def check():
        table, lens = t.tables()
        held = set()
        for s in range(seqs):
            assert lens[s] == len(want[s])
            used = -(-len(want[s]) // page)
            assert (table[s, used:] == -1).all()
            assert [mem[table[s, i // page], i % page] for i in range(len(want[s]))] == want[s]
            held |= set(table[s, :used].tolist())
        assert t.free_pages == pool - len(held)

    for step in range(2000):
        if step >= 200 and refusals > 0:
            break
        before, owner, forked = stamp, {}, set()
        s = 0
        for _ in range(rng.randint(1, 6)):
            s, what = rng.choice([s, rng.randrange(seqs)]), rng.random()
            if what < 0.5:
                n = rng.choice([1, 1, 2, 5, 16, 20])
                try:
                    t.reserve(s, n)
                except bsa.BsaError as e:
                    assert e.code == 4
                    continue
                owner.update((x, s) for x in range(stamp, stamp + n))
                want[s] = want[s] + list(range(stamp, stamp + n))
                stamp += n
            elif what < 0.75:
                empty = [x for x in range(seqs) if not want[x] and x != s]
                if empty and want[s]:
                    t.fork(s, empty[0])
                    want[empty[0]] = list(want[s])
                    forked.add(empty[0])
                    s = rng.choice([s, empty[0]])
            else:
                n = rng.choice([0, len(want[s]) // 2, max(0, len(want[s]) - 1)])
                t.truncate(s, n)
                want[s] = want[s][:n]
        try:
            pairs = t.take_copies()
        except bsa.BsaError as e:
            assert e.code == 1 and forked
            refusals += 1
            for s in forked:
                t.free(s)
                want[s] = []
            t.tables()
            pairs = t.take_copies()
        copy(pairs)
        table, _ = t.tables()
        for x in range(before, stamp):
            has = [s for s in range(seqs) if x in want[s]]
            if has:
                s = owner[x] if owner[x] in has else has[0]
                i = want[s].index(x)
                mem[table[s, i // page], i % page] = x
        check()
        if rng.random() < 0.2:
            copy(t.compact())
            check()
    assert refusals > 0


# ------------------------------------------------ numbers that do not fit in C
def test_numbers_that_do_not_fit_are_refused(L):
    """ctypes keeps the low bits of any number: 2^32 would be sequence 0."""
    t = bsa.PageTable(4, 16, 2, 3)
    t.reserve(np.int64(0), np.int32(5))
    for call in (lambda: t.reserve(1 << 32, 1), lambda: t.reserve(0, (1 << 64) + 1), lambda: t.reserve(0, 1.5),
                 lambda: t.fork(1 << 32, 1), lambda: t.fork(0, (1 << 32) + 1), lambda: t.truncate(-(1 << 32), 0),
                 lambda: t.truncate(0, 1 << 64), lambda: t.free(1 << 32),
                 lambda: bsa.PageTable((1 << 64) + 4, 16, 2, 3), lambda: bsa.PageTable(4, (1 << 32) + 16, 2, 3),
                 lambda: bsa.PageTable(4, 16, (1 << 32) + 2, 3), lambda: bsa.PageTable(4, 16, 2, (1 << 32) + 3),
                 lambda: bsa.Rope((1 << 32) + 64, device="cpu")):
        with pytest.raises(ValueError):
            call()
    assert t.tables()[1].tolist() == [5, 0]
    x, plan = torch.zeros(2, 3, 64), bsa.Rope(64, device="cpu")
    for first in (1 << 63, -(1 << 63) - 1, 1 << 64, 2.5):
        with pytest.raises(ValueError):
            bsa.rope(x, plan, first)
    c = type("C", (), {"k": torch.zeros(1)})()
    for pair in ([1 << 32, 1], [0, (1 << 32) + 1], [0.5, 1.0], [0, float("nan")], [0, 1 << 31]):
        with pytest.raises(ValueError):
            bsa.copy_pages(c, np.array([pair]))


@pytest.mark.parametrize("count", [1 << 31, 1 << 62, (1 << 62) + 1, (1 << 63) - 1])
def test_more_pairs_than_a_launch_takes_are_refused(L, count):
    """The launch's CTAs, a multiple of the count, wrapped modulo 2^64."""
    c = bsa.Cache(0x100000, 0x4000000, 0x8000000, 8, 2, 64, 64)
    assert L.bsa_cache_copy_pages(c, ctypes.c_void_p(0x100000), count, None) == 2
    assert b"count" in L.bsa_last_error()
