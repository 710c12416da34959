"""Arguments of the sequence-mixer operators at and past the limits of the address arithmetic: refused before the
first CUDA call, so no GPU is needed."""
import ctypes

import pytest

from test_mixer_refusals import BAD, N, conv, conv_b, conv_s, norm, norm_b, scan, scan_b, scan_s, table

T = 1 << 20
PLAIN = (8 * T * 2, 8 * T, 8)            # [2, 2, T, 8], contiguous
TABLES = {conv: 2, conv_b: 3, conv_s: 2, scan: 6, scan_b: 9, scan_s: 6, norm: 2, norm_b: 3}


def sizes(fn):
    return {} if fn in (conv_s, scan_s) else dict(T=T)


@pytest.mark.parametrize("fn", list(TABLES))
def test_extents_past_64_bits(fn):
    """Each stride on its own is below the limit, the tensor's extent in bytes is past 2^64 (or its elements past 2^63):
    a sum that wraps would pass for a small tensor, or for one that overlaps nothing."""
    for i in range(TABLES[fn]):
        for row, more in (((1 << 42, 8 * T, 8), dict(B=1 << 20)), ((8 * T * 2, 1 << 42, 8), dict(H=1 << 20)),
                          ((8 * T * 2, 8 * T, 1 << 42), {}), ((8 * T * 2, 8 * T, (1 << 42) - 1), {})):
            if not more and fn in (conv_s, scan_s):
                continue                                  # one token: its stride is not used
            rows = [PLAIN] * TABLES[fn]
            rows[i] = row
            if "H" in more and fn in (scan, scan_b, scan_s) and i in (2, 3):
                more = dict(more, G=1 << 20)              # Bm and Cm are strided by group
            assert fn(strides=table(*rows), **{**sizes(fn), **more}) == BAD, (i, row)


@pytest.mark.parametrize("fn", [conv, conv_b, scan, scan_b, norm, norm_b])
def test_elements_past_the_limit(fn):
    """2^59 elements: contiguous, each size within its own limit."""
    assert fn(B=1 << 10, H=1, d=1 << 20, T=1 << 29) == BAD


def test_workspace_queries_of_sizes_past_the_limit():
    """Sizes whose workspace would pass 2^64 bytes are refused, and the largest ones allowed are counted right."""
    lib, n = N.load(), ctypes.c_size_t()
    big = (1 << 10, 1, 1 << 29, 1 << 20)                  # B, H, T, d
    assert lib.tm_scan_backward_workspace_size(1 << 10, 1, 1, 1 << 29, 1 << 20, 128, N.TM_F32, ctypes.byref(n)) == BAD
    assert lib.tm_scan_workspace_size(1 << 10, 1, 1, 1 << 29, 1 << 20, 128, N.TM_F32, ctypes.byref(n)) == BAD
    assert lib.tm_conv_backward_workspace_size(*big, 8, N.TM_F32, ctypes.byref(n)) == BAD
    for over in (0, 1):
        for back in (0, 1):
            assert lib.tm_group_norm_workspace_size(*big, over, back, ctypes.byref(n)) == BAD
    assert lib.tm_scan_backward_workspace_size(1, 1, 1, 1 << 26, 1 << 20, 128, N.TM_F32, ctypes.byref(n)) == N.TM_OK
    assert n.value >= (1 << 24) * (1 << 20) * 128 * 4     # the states at every 4th token alone
