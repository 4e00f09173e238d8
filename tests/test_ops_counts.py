"""Counts of segments and adapters that 32-bit piece and part numbers cannot hold
are refused before any launch (no GPU; the addresses are never used)."""
import ctypes

import pytest

from sketched_parameter_sharing_amd import _lib
from test_ops_abi import AD, SG, adb, adf

TOP = 2 ** 31 - 1


@pytest.mark.parametrize("call", [adf, adb])
@pytest.mark.parametrize("count", [1 << 30, TOP])
def test_too_many_segments_or_adapters(call, count):
    assert call(sg=SG(count=count)) == _lib.ERR_SHAPE
    assert call(ad=AD(count=count)) == _lib.ERR_SHAPE


def test_the_query_refuses_them_too():
    lib, n = _lib.load(), ctypes.c_size_t(0)
    for f in (lib.ss1_adapter_forward_query, lib.ss1_adapter_backward_query):
        assert f(5, ctypes.byref(AD(count=1 << 30)), ctypes.byref(n)) == _lib.ERR_SHAPE
        assert f(5, ctypes.byref(AD(count=(1 << 30) - 1)), ctypes.byref(n)) == _lib.OK
