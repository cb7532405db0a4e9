"""How far attention's weights are rounded, on the GPU, form by form.  The
values of the last key are chosen so that an output is nearly zero while the
sum of w |v| is not: what the weights are off by is not lost in the output's own
rounding."""
import math

import pytest
import torch

from content_dependent_block_gb300 import _build, bsa
from tests import attention_reference as att
from tests import paged_reference as ref
from tests.test_gpu_paged_attention import _i32, _randn

pytestmark = pytest.mark.gpu

# Half a step of a bf16 number is 2^-8 of it, and the remainder, at most 2^-8, is
# rounded by half a step of [2^-9, 2^-8), 2^-17; fp16 2^-11.
PAIR, ONE, HALF = 2.0 ** -17, 2.0 ** -8, 2.0 ** -11
PAGE = 16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    _build.build()


def half_step(y):
    """Half of the distance between the bf16 numbers around |y| (normal range)."""
    return torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -120))) - 8)


def problem(seed, lens, group, d, bits):
    """(k, v or codes and scales of both, q) of sequences of one token each over
    one cache head: the first query head's output is nearly zero."""
    g = torch.Generator().manual_seed(seed)
    width = -(-max(lens) // PAGE)
    k, v = (_randn(g, len(lens) * width, 1, PAGE, d) for _ in range(2))
    q = _randn(g, len(lens), group, d)
    if bits == 8:
        k, v = att.quantise(k), att.quantise(v)
    for s, n in enumerate(lens):
        pages, at = list(range(s * width, (s + 1) * width)), (s * width + (n - 1) // PAGE, 0, (n - 1) % PAGE)
        kk, vv = (_rows(x, pages, n) for x in (k, v))
        w = torch.softmax(kk @ q[s, 0].double() / math.sqrt(d), 0)
        last = (-(w[:-1] @ vv[:-1]) / w[-1]).bfloat16()
        if bits == 8:
            v[0][at], v[1][at] = att.quantise(last)
        else:
            v[at] = last
    return k, v, q, torch.arange(len(lens) * width).view(len(lens), width)


def _rows(x, pages, n):
    x = att.values(*x) if isinstance(x, tuple) else x.double()
    return x[pages, 0].reshape(-1, x.shape[-1])[:n]


def bounds(k, v, q, table, lens, weight):
    """(out, tol) in fp64: the weights' rounding, of the scores (a dot product of
    d terms and the factors), the exponentials and the sums as in
    attention_reference.attention, and the output's to the nearest bf16."""
    d = q.shape[-1]
    out = torch.zeros(q.shape, dtype=torch.float64)
    tol = torch.zeros_like(out)
    for s, n in enumerate(lens):
        kk, vv = (_rows(x, table[s].tolist(), n) for x in (k, v))
        for r in range(q.shape[1]):
            qd = q[s, r].double()
            w = torch.softmax(kk @ qd / math.sqrt(d), 0)
            out[s, r] = w @ vv
            slip = float((kk.abs() @ qd.abs()).max()) / math.sqrt(d) * (d + 6) * 2.0 ** -24
            off = (weight + 2 * slip + 2.0 ** -20 + 2 * n * 2.0 ** -24) * (w @ vv.abs())
            if weight == HALF:
                off = off + n * 2.0 ** -29 * vv.abs().amax()
            tol[s, r] = off + half_step(out[s, r].abs() + off)
    return out, tol


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bits,group,weight", [
    (16, 1, PAIR), (16, 5, PAIR), (16, 8, PAIR), (16, 16, PAIR),        # few rows
    (16, 17, ONE), (16, 128, ONE),                                      # tiles of 128 rows
    (8, 1, HALF), (8, 8, HALF), (8, 16, HALF), (8, 17, HALF), (8, 100, HALF),
])
def test_weights_are_off_by_what_their_form_says(bits, group, weight, d):
    lens = [2, 3, 4, 5, 7, 9, 15, 16, 17, 33] * 3
    k, v, q, table = problem(group + d, lens, group, d, bits)
    want, tol = bounds(k, v, q, table, lens, weight)
    kbar = torch.zeros(table.numel(), 1, d, device="cuda")
    if bits == 8:
        cache = bsa.PagedCache8(k[0].cuda(), v[0].cuda(), k[1].cuda(), v[1].cuda(), kbar)
    else:
        cache = bsa.PagedCache(k.cuda(), v.cuda(), kbar)
    out = bsa.paged_attention(cache, q.cuda(), _i32(table), _i32([n - 1 for n in lens]))
    ref.assert_within(out, want, tol, "attention")
    assert bsa.device_status() == 0
