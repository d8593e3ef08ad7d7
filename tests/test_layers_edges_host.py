"""Group norm and dropout without a GPU: the edges of the accepted sizes and
arguments."""

import ctypes

import pytest
import torch

from transposed_convolution_02_b200 import ct


def workspace(dtype, n, s, c, groups):
    """(forward, backward) workspace bytes of a group norm."""
    d = ct.ct_group_norm_desc(dtype, 0, 0, 0, n, s, c, groups, 1e-5)
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert ct.lib().ct_group_norm_workspace_bytes(ctypes.byref(d), ctypes.byref(f), ctypes.byref(b)) == 0
    return f.value, b.value


@pytest.mark.parametrize("dtype", [ct.CT_F32, ct.CT_F16])
@pytest.mark.parametrize("n,c,groups", [(3, 8, 2), (700, 4099, 1), (1 << 21, (1 << 24) - 1, 1),
                                        (1 << 30, 1 << 24, 1 << 24)])
def test_no_pixels_need_no_workspace(dtype, n, c, groups):
    assert workspace(dtype, n, 0, c, groups) == (0, 0)
