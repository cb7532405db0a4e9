"""The 8-bit cache, reading back and attention over the paged cache: what is
refused on the host, and the references' own pins (no GPU needed)."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

from content_dependent_block_gb300 import _build, bsa
from tests import attention_reference as att

BASE = 1 << 40
FAKE = ctypes.c_void_p(BASE)                 # aligned, never dereferenced
FAR = ctypes.c_void_p(1 << 44)
FURTHER = ctypes.c_void_p(1 << 45)
ODD = ctypes.c_void_p((1 << 44) + 8)         # not 16-byte aligned
ODDER = ctypes.c_void_p((1 << 44) + 2)       # not 4-byte aligned


@pytest.fixture(scope="module")
def L():
    _build.build()
    return bsa.lib()


def _cache16(**kw):
    a = dict(k=BASE, v=BASE + (1 << 30), kbar=BASE + (2 << 30), num_pages=16, heads=2, page=64, d=64)
    a.update(kw)
    return bsa.Cache(a["k"], a["v"], a["kbar"], a["num_pages"], a["heads"], a["page"], a["d"])


def _cache8(**kw):
    a = dict(k=BASE, v=BASE + (1 << 30), ks=BASE + (3 << 30), vs=BASE + (4 << 30), kbar=BASE + (2 << 30),
             num_pages=16, heads=2, page=64, d=64)
    a.update(kw)
    return bsa.Cache8(a["k"], a["v"], a["ks"], a["vs"], a["kbar"], a["num_pages"], a["heads"], a["page"], a["d"])


BAD = [(dict(k=None), 1), (dict(v=None), 1), (dict(kbar=None), 1), (dict(k=BASE + 8), 7), (dict(d=96), 2),
       (dict(page=48), 2), (dict(num_pages=0), 1), (dict(heads=0), 1), (dict(heads=65536), 2),
       (dict(num_pages=1 << 31), 2)]
BAD8 = BAD + [(dict(ks=None), 1), (dict(vs=None), 1), (dict(ks=BASE + 4), 7), (dict(vs=BASE + 8), 7)]

STRIDES = bsa.Strides(0, 64, 128)


def _read(L, c, eight, tokens=4, seqs=2, cu=None, start=FAR, table=FAR, width=4, k=FAR, v=FURTHER, st=STRIDES):
    fn = L.bsa_cache8_read if eight else L.bsa_cache_read
    return fn(c, tokens, seqs, cu, start, table, width, k, v, st, None)


def _attend(L, c, eight, q=FAR, qs=256, tokens=4, heads=4, table=FAR, width=4, seqs=2, cu=None, start=FAR, tree=None,
            window=None, scale=0.0, out=FURTHER):
    fn = L.bsa_paged_attention8 if eight else L.bsa_paged_attention
    return fn(c, q, qs, tokens, heads, table, width, seqs, cu, start, tree,
              None if window is None else ctypes.byref(bsa.Window(*window)), scale, out, None)


@pytest.mark.parametrize("bad,code", BAD8)
def test_bad_8_bit_caches_are_refused(L, bad, code):
    c = _cache8(**bad)
    assert L.bsa_cache8_append(c, FAR, 1 << 24, FAR, 1 << 24, 4, 4, None, FAR, FAR, 4, None) == code
    assert L.bsa_cache8_copy_pages(c, FAR, 1, None) == code
    assert L.bsa_paged_decode8(c, FAR, 1 << 24, 4, max(1, c.heads), FAR, 4, 4, None, FAR, 4, None, 0.0, FURTHER,
                               None, None) == code
    assert _read(L, c, True) == code
    assert _attend(L, c, True) == code


@pytest.mark.parametrize("bad,code", BAD)
def test_bad_caches_are_refused(L, bad, code):
    assert _read(L, _cache16(**bad), False) == code
    assert _attend(L, _cache16(**bad), False) == code


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), 1), (dict(seqs=0), 1), (dict(width=0), 1), (dict(tokens=3), 1), (dict(tokens=1 << 31), 2),
    (dict(seqs=1 << 23, tokens=1 << 23), 2), (dict(tokens=0), 0), (dict(tokens=0, k=None, v=None), 0),
    (dict(k=None), 1), (dict(v=None), 1), (dict(k=ODD), 7), (dict(v=ODD), 7), (dict(start=None), 1),
    (dict(table=None), 1), (dict(start=ODDER), 7), (dict(table=ODDER), 7), (dict(cu=ODDER), 7),
    (dict(v=FAR), 1), (dict(v=ctypes.c_void_p((1 << 44) + 512)), 1), (dict(k=FAKE), 1),
    (dict(v=ctypes.c_void_p(BASE + (1 << 30))), 1),
    (dict(st=bsa.Strides(0, 64, -128)), 2), (dict(st=bsa.Strides(0, 64, 1 << 41)), 2),
    (dict(st=bsa.Strides(0, 68, 136)), 7), (dict(st=bsa.Strides(0, 64, 64)), 1), (dict(st=bsa.Strides(0, 56, 128)), 1),
    (dict(st=bsa.Strides(0, 192, 64)), 1), (dict(st=bsa.Strides(0, 64, 0)), 1),
])
def test_read_refusals(L, eight, kw, code):
    assert _read(L, _cache8() if eight else _cache16(), eight, **kw) == code, L.bsa_last_error()


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-2), 1), (dict(seqs=0), 1), (dict(width=0), 1), (dict(tokens=3), 1), (dict(tokens=1 << 31), 2),
    (dict(heads=3), 1), (dict(heads=0), 1), (dict(heads=258, qs=1 << 20), 2), (dict(tokens=0), 0),
    (dict(tokens=0, q=None, out=None), 0), (dict(q=None), 1), (dict(out=None), 1), (dict(q=ODD), 7), (dict(out=ODD), 7),
    (dict(qs=192), 1), (dict(qs=260), 7), (dict(qs=1 << 31), 2), (dict(table=None), 1), (dict(start=None), 1),
    (dict(table=ODDER), 7), (dict(start=ODDER), 7), (dict(cu=ODDER), 7),
    (dict(tree=ctypes.c_void_p((1 << 44) + 4)), 7), (dict(window=(0, 0)), 1), (dict(window=(-1, 0)), 1),
    (dict(window=(4, -1)), 1), (dict(scale=math.nan), 1), (dict(out=FAR), 1),
    (dict(out=ctypes.c_void_p((1 << 44) + 4 * 512 - 16)), 1), (dict(out=FAKE), 1),
])
def test_attention_refusals(L, eight, kw, code):
    assert _attend(L, _cache8() if eight else _cache16(), eight, **kw) == code, L.bsa_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), 1), (dict(tokens=3), 1), (dict(k=None), 1), (dict(k=ODD), 7), (dict(ks=120), 1),
    (dict(ks=132), 7), (dict(start=None), 1), (dict(table=ODDER), 7), (dict(k=FAKE), 1),
    (dict(v=ctypes.c_void_p(BASE + (3 << 30))), 1), (dict(v=ctypes.c_void_p(BASE + (4 << 30))), 1),
    (dict(tokens=0, k=None), 0),
])
def test_append8_refusals(L, kw, code):
    a = dict(k=FAR, ks=128, v=FAR, vs=128, tokens=4, seqs=4, cu=None, start=FAR, table=FAR, width=4)
    a.update(kw)
    assert L.bsa_cache8_append(_cache8(), a["k"], a["ks"], a["v"], a["vs"], a["tokens"], a["seqs"], a["cu"], a["start"],
                               a["table"], a["width"], None) == code, L.bsa_last_error()


def test_the_scales_count_as_part_of_the_cache(L):
    for at in (BASE, BASE + (1 << 30), BASE + (2 << 30), BASE + (3 << 30), BASE + (4 << 30)):
        p = ctypes.c_void_p(at)
        assert _attend(L, _cache8(), True, out=p) == 1
        assert L.bsa_paged_decode8(_cache8(), FAR, 256, 4, 4, FAR, 4, 4, None, FAR, 2, None, 0.0, p, None, None) == 1
    assert L.bsa_cache8_copy_pages(_cache8(), FAR, 0, None) == 0
    assert L.bsa_cache8_copy_pages(_cache8(), FAR, 1 << 32, None) == 2
    assert L.bsa_cache8_copy_pages(_cache8(), ODDER, 1, None) == 7


# ------------------------------------------------------------- the references
def test_the_quantising_reference_is_exact():
    """Against rational arithmetic, ties among them."""
    g = torch.Generator().manual_seed(0)
    x = torch.randn(60, 16, generator=g).bfloat16()
    x[0, :4] = torch.tensor([127.0, 63.5, -0.5, 1.5])
    x[1, :4] = torch.tensor([2.0, 1.0, -1.0, 0.5])
    codes, scale = att.quantise(x)
    for r in range(x.shape[0]):
        row = [Fraction(float(v)) for v in x[r]]
        a = max(abs(v) for v in row)
        assert codes[r].tolist() == [round(127 * v / a) for v in row]       # ties to the even
        near = float(a) / 127
        assert float(scale[r]) == float(torch.tensor(near, dtype=torch.float64).float())
    bad = torch.ones(3, 4).bfloat16()
    bad[0, 1], bad[1, 2] = float("inf"), float("nan")
    codes, scale = att.quantise(bad)
    assert scale[:2].isnan().all() and not codes[:2].any() and codes[2].tolist() == [127] * 4
    codes, scale = att.quantise(torch.zeros(1, 4).bfloat16())
    assert scale.tolist() == [0.0] and not codes.any()


def test_sight_by_hand():
    # a chain: the last two keys and the first one
    s = att.sight(3, 2, None, 2, 1)
    assert s.tolist() == [[True, False, True, True, False], [True, False, False, True, True]]
    # a tree: 0, its children 1 and 2, and 3 under 2
    words = att.tree_masks([-1, 0, 0, 2])
    assert words == [1, 3, 5, 13]
    s = att.sight(2, 4, words, 0, 0)
    assert s[:, :2].all() and s[:, 2:].int().tolist() == [[1, 0, 0, 0], [1, 1, 0, 0], [1, 0, 1, 0], [1, 0, 1, 1]]
    # positions 2, 3, 3, 4: with a window of 2 token 3 sees positions 3 and 4
    s = att.sight(2, 4, words, 2, 0)
    assert s.int().tolist() == [[0, 1, 1, 0, 0, 0], [0, 0, 1, 1, 0, 0], [0, 0, 1, 0, 1, 0], [0, 0, 0, 0, 1, 1]]
    # without a prefix its root lies below the sinks
    s = att.sight(0, 4, words, 1, 1)
    assert s.int().tolist() == [[1, 0, 0, 0], [1, 1, 0, 0], [1, 0, 1, 0], [1, 0, 0, 1]]


def test_the_attention_reference_by_hand():
    k = torch.tensor([[[[0.0, 0.0], [1.0, 0.0], [0.0, 1.0], [9.0, 9.0]]]])
    v = torch.tensor([[[[1.0, 0.0], [0.0, 1.0], [1.0, 1.0], [float("nan"), 5.0]]]])
    q = torch.tensor([[[1.0, 0.0]], [[0.0, 2.0]]])
    out, tol = att.attention(k, v, q, [[0]], [0, 2], [1], scale=1.0)
    e = math.e
    assert torch.allclose(out[0, 0], torch.tensor([1 / (1 + e), e / (1 + e)], dtype=torch.float64))
    z = 2 + e ** 2
    assert torch.allclose(out[1, 0], torch.tensor([(1 + e ** 2) / z, (1 + e ** 2) / z], dtype=torch.float64))
    assert bool((tol > 0).all())
    # nothing seen
    out, _ = att.attention(k, v, q[:1], [[0]], [0, 1], [0], words=[0], scale=1.0)
    assert not out.any()
