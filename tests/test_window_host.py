"""The window of an attention call follows its arguments' values (no GPU needed)."""
import numpy as np
import pytest
import torch

from content_dependent_block_gb300 import _build, bsa


@pytest.fixture(scope="module", autouse=True)
def _lib():
    _build.build()


def _numbers(w):
    w = w._obj                              # what the reference refers to
    return w.window, w.sinks


def test_a_tensor_that_changes_in_place():
    w, s = torch.tensor(256), torch.tensor(4)
    assert _numbers(bsa._window(w, s)) == (256, 4)
    w.add_(1)
    s.sub_(3)
    assert _numbers(bsa._window(w, s)) == (257, 1)
    w.zero_()
    s.zero_()
    assert bsa._window(w, s) is None


def test_an_array_that_changes_in_place():
    w = np.array(100)
    assert _numbers(bsa._window(w, 0)) == (100, 0)
    w += 5
    assert _numbers(bsa._window(w, 0)) == (105, 0)


def test_whole_numbers_of_any_kind():
    for w in (7, 7.0, np.int64(7), np.float32(7), torch.tensor(7.0)):
        assert _numbers(bsa._window(w, np.int32(2))) == (7, 2)
    assert _numbers(bsa._window(True, False)) == (1, 0)
    for w, s in ((0, 0), (False, 0), (0.0, np.int64(0))):
        assert bsa._window(w, s) is None


@pytest.mark.parametrize("w,s", [(2.5, 0), (torch.tensor(2.5), 0), (1 << 31, 0), (3, 1 << 40), (float("nan"), 0),
                                 (3, 0.5), (0, 1), (torch.tensor(0), np.array(1))])
def test_refusals_whatever_was_asked_before(w, s):
    for asked in ((2, 0), (3, 0), (3, 1), (1, 0)):
        bsa._window(*asked)
    with pytest.raises(ValueError):
        bsa._window(w, s)
