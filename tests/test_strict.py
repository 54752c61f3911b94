"""The strict comparison's own refusals."""

import numpy as np
import pytest
import torch

from tests.strict import assert_within


def test_takes_what_is_close():
    want = np.linspace(-2, 2, 12).reshape(3, 4)
    assert_within(want + 1e-3, want, 1.1e-3)
    assert_within(torch.tensor(want).to(torch.bfloat16), want, 2.0 ** -8 * np.abs(want))
    assert_within(np.zeros((0, 4)), np.zeros((0, 4)), 0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 0.5])
@pytest.mark.parametrize("at", [(0, 0), (2, 3), ...])
def test_refuses_what_is_not(bad, at):
    want = np.ones((3, 4))
    got = torch.ones(3, 4)
    got[at] = bad
    for t in (got, got.to(torch.bfloat16), got.numpy()):
        with pytest.raises(AssertionError):
            assert_within(t, want, 0.25)


def test_refuses_a_tolerance_or_a_reference_that_is_none():
    nan = float("nan")
    for got, want, room in ((1.0, 1.0, nan), (nan, nan, 1.0), (1.0, nan, 1.0),
                            (float("inf"), float("inf"), 1.0), (1.0, float("inf"), float("inf"))):
        with pytest.raises(AssertionError):
            assert_within(np.array([got]), np.array([want]), room)
    with pytest.raises(AssertionError):
        assert_within(np.ones(4), np.ones((4, 1)), 1)
