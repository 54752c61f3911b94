"""Sizes of the norm gradient's workspace, on the host: one that was made for a
number of rows serves every smaller number."""

import ctypes

import pytest

import bit_grouped_moe_amd as gq

INVALID, NOT_SUPPORTED = 1, 801


@pytest.mark.parametrize("H", [1, 512, 513, 600, 1024, 1025, 2048, 2049, 8192, 8193, 32768])
def test_size_never_falls(H):
    size = gq.load_library().gq_rms_norm_backward_workspace
    at = [size(rows, H) for rows in range(1101)]
    assert at[0] == 0 and at[1] >= 4 * H
    assert all(a <= b for a, b in zip(at, at[1:])), [
        rows for rows, (a, b) in enumerate(zip(at, at[1:])) if a > b]
    # a row of partial sums each for at most 512 workgroups, none without a row
    assert all(s <= 4 * H * min(rows, 512) for rows, s in enumerate(at))
    assert size(1 << 40, H) >= at[-1]


@pytest.mark.parametrize("H", [512, 600, 1024])
def test_size_for_the_most_rows_is_taken_for_fewer(H):
    """The entry point's own check: a buffer of the size for 300 rows passes it for 1
    to 300 rows, and the call is refused for what is looked at behind it, a stride
    past 2^60 elements."""
    lib = gq.load_library()
    F, D = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x200000)

    def call(rows, bytes_, stride):
        return lib.gq_rms_norm_backward(F, stride, F, stride, None, stride, 0, rows, H, F, 0, 1e-6,
                                        D, D, D, bytes_, None)

    most = lib.gq_rms_norm_backward_workspace(300, H)
    for rows in (1, 75, 76, 77, 255, 256, 257, 299, 300):
        assert call(rows, most, 1 << 61) == NOT_SUPPORTED, rows
    assert call(300, 0, 1 << 61) == INVALID
