"""Softmax choices in float32 where its error is largest: experts far below the peak, sums
of many equal small terms, and biases that bring choices to within that error of each
other; the chosen experts are float64's exactly."""

import numpy as np
import pytest
import torch

import bit_grouped_moe_amd as gq
from tests import test_gpu_moe_route as mr
from tests.gpu_common import device, say, to_dev

pytestmark = pytest.mark.gpu


def _same(dev, z, bias, topk, groups, open_, top):
    ids, _ = gq.gq_moe_route(to_dev(z, dev), topk, bias=to_dev(bias, dev), groups=groups,
                             topk_groups=open_, group_top=top)
    torch.cuda.synchronize()
    want = mr._select(z, topk, "softmax", bias, groups, open_, top)
    assert np.array_equal(ids.cpu().numpy(), want), np.argwhere(
        (ids.cpu().numpy() != want).any(axis=1))[:4].tolist()


@pytest.mark.parametrize("rows", [40, 4200])
@pytest.mark.parametrize("E,groups", [(64, 8), (256, 8), (1024, 8)])
def test_far_below_the_peak(E, groups, rows):
    """Scores from 1 down to float32's least, alone the choices: what a float32 exponential
    gets wrong by several 2^-19 of itself."""
    dev = device()
    g = np.random.default_rng(E + rows)
    z = g.uniform(-88, 0, (rows, E)).astype(np.float32)
    z[:, 0::2] = z[:, 1::2] + np.float32(2.0 ** -18)       # neighbours that differ little
    zero = np.zeros(E, dtype=np.float32)
    for G, open_, top in ((1, 1, 1), (groups, 3, 1), (groups, 3, 2)):
        say("route far", E, rows, G, top)
        _same(dev, z, zero, 8, G, open_, top)


@pytest.mark.parametrize("rows", [40, 4200])
@pytest.mark.parametrize("E,x", [(64, 2.9), (256, 4.3), (1024, 5.4)])
def test_largest_error_of_the_sum(E, x, rows):
    """One expert at the peak and all others x below it, where their roundings weigh most
    in the sum; biases that level all choices, rows that differ by about the error."""
    dev = device()
    g = np.random.default_rng(E)
    z = np.full((rows, E), -x, dtype=np.float32)
    z[:, E // 3] = 0
    z += (g.uniform(0, 4e-6, (rows, 1)) * g.standard_normal((rows, E))).astype(np.float32)
    s = mr._scores(z[:1], "softmax")[0]
    bias = (1 - s).astype(np.float32)
    for G, open_, top in ((1, 1, 1), (8, 3, 1), (8, 3, 2)):
        say("route sum's error", E, rows, G, top)
        _same(dev, z, bias, 8, G, open_, top)
