"""A comparison that a NaN does not pass.  (`|got - want| > tol` is false for a NaN,
so that a check for any such element takes it for a good one.)"""

import numpy as np
import torch


def _array(a):
    if isinstance(a, torch.Tensor):
        a = a.detach().double().cpu().numpy()
    return np.asarray(a, dtype=np.float64)


def assert_within(got, want, room, what=""):
    """Every element of `got` lies within `room` of `want`; a NaN or infinity on
    either side, of `room` too, does not."""
    got, want = _array(got), _array(want)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    with np.errstate(invalid="ignore"):
        good = (np.abs(got - want) <= np.broadcast_to(_array(room), got.shape)) & np.isfinite(want)
    good &= np.isfinite(got)
    assert good.all(), (what, int((~good).sum()), np.argwhere(~good)[:6].tolist())
