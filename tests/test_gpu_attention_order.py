"""What the warps of attention's tiles hand one another, on the GPU: long
sequences, so that every ring of tiles is used many times over, in calls that
are repeated and have to agree."""
import pytest
import torch

from content_dependent_block_gb300 import _build, bsa
from tests import attention_reference as att
from tests import paged_reference as ref
from tests.test_gpu_paged_attention import Step, _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    _build.build()


@pytest.fixture(autouse=True)
def _clean_status():
    bsa.device_status()
    yield
    torch.cuda.synchronize()


def _repeat(step, times, **kw):
    """The calls' outputs, all of them equal (bit for bit: some are NaN)."""
    cache, q, table, start = step.cache(), step.q.cuda(), _i32(step.table), _i32(step.start)
    outs = [bsa.paged_attention(cache, q, table, start, **kw) for _ in range(times)]
    assert all(torch.equal(outs[0].view(torch.int16), x.view(torch.int16)) for x in outs[1:])
    return outs[0]


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("d,new", [(64, 20), (128, 20), (64, 150)])
def test_pages_that_are_not_there_along_a_sequence(d, new, bits):
    """Which pages of a tile are there is noted by one warp and read by others:
    tiles with another set of them each, many more than the notes that are
    kept."""
    step = Step(60, d, 16, 1, 4, bits, [4000], [new], poison=False)
    bad = set()
    for b in range(250):
        if torch.randint(0, 3, (1,), generator=step.g).item() == 0:
            step.table[0][b] = 10 ** 6
            bad.add(b)
    assert 40 < len(bad) < 130
    got = _repeat(step, 10)
    assert bsa.device_status() == 3
    k, v = step.values()
    want, tol = att.attention(k, v, step.q, step.table, step.cu, step.start, bits=bits, skipped=(10 ** 6,))
    ref.assert_within(got, want, tol, "pages that are not there")


@pytest.mark.parametrize("d,heads", [(64, 8), (128, 8)])
def test_rows_that_are_computed_again(d, heads):
    """Rows whose tile met a masked value that is not finite are written twice,
    by one lane and then by all: most rows of pairs of tiles."""
    step = Step(61, d, 16, heads, 4, 16, [70], [900])
    clean = step.v.clone()
    for j in range(0, 900, 64):
        step.v[step.table[0][j // 16], :, j % 16, 5] = float("nan")
    got = _repeat(step, 10, window=24).cpu()
    hit = att.sight(70, 900, None, 24, 0)[:, :900:64].any(1)
    assert 250 < int(hit.sum()) < 400 and bool(got[hit][..., 5].isnan().all())
    assert bool(torch.isfinite(got[~hit]).all())
    clean[~torch.isfinite(clean)] = 0.0
    want, tol = att.attention(step.k, clean, step.q, step.table, [0, 900], [70], None, 24, 0)
    ref.assert_within(got[~hit], want[~hit], tol[~hit], "rows that see none")
    assert bsa.device_status() == 0
