"""Sizes of libgdn_step.so's calls that one launch does not hold are refused on the host, before
anything is enqueued (fake pointers are never read)."""

import ctypes
import re

import pytest

from bitwise_consistent_linear_amd import api

FAKE = 0x100000
F32 = api.GDN_DTYPE_F32


def quantize(rows, k, qt=FAKE):
    return api.step_lib().gdn_quantize_f8(FAKE, rows, k, 0, F32, 0, FAKE, FAKE, qt, qt, None)


def backward(m, n, dw=FAKE):
    shape = api.GdnLinearF8Shape(m, n, 64, 0, F32, 0, F32, F32)
    return api.step_lib().gdn_linear_f8_bwd(ctypes.byref(shape), FAKE, FAKE, FAKE, FAKE, FAKE, None,
                                            dw, FAKE, 1 << 62, None)


# 2^24 tiles of 128 x 128 values by 256 threads each are 2^32 threads, one more than a launch holds
@pytest.mark.parametrize("rows,k", [(2 ** 20, 2 ** 20), (2 ** 19, 2 ** 19), (2 ** 20, 2 ** 18),
                                    (2 ** 18, 2 ** 20 - 127), (2 ** 20 - 127, 2 ** 18 - 1)])
def test_by_columns(rows, k):
    assert quantize(rows, k) == api.GDN_E_SHAPE
    assert re.match("gdn_quantize_f8: .*one launch", api.step_lib().gdn_step_last_error().decode())
    assert backward(rows, k) == api.GDN_E_SHAPE
    assert re.match("gdn_linear_f8_bwd: .*one launch", api.step_lib().gdn_step_last_error().decode())
