"""The selective scan's workspace for packed rows: states where sequences are cut, none for sequences that are not."""
import ctypes

import pytest

import chunk_wise_weight_amd as cw
from chunk_wise_weight_amd import _lib


def size(name, n, num, dtype, H=64, G=8, P=64, N=128, B=1):
    out = ctypes.c_size_t(0)
    shape = _lib.ScanShape(B, n, H, G, P, N)
    assert getattr(cw.lib(), name)(ctypes.byref(shape), dtype, num, ctypes.byref(out)) == cw.TTT_OK
    return out.value


@pytest.mark.parametrize("dtype", [cw.TTT_BF16, cw.TTT_F32])
@pytest.mark.parametrize("n", [1000, 16456, 65536])
def test_more_sequences_take_no_more(n, dtype):
    """A row of n tokens is cut at most n / segment times however many sequences it holds."""
    one = size("ttt_selective_scan_workspace_bytes", n, 1, dtype)
    assert 0 < one < 1 << 28
    for num in (2, 12, 1024, 4096):
        assert size("ttt_selective_scan_workspace_bytes", n, num, dtype) == one
    assert size("ttt_selective_scan_workspace_bytes", n, 0, dtype) == 0


@pytest.mark.parametrize("dtype", [cw.TTT_BF16, cw.TTT_F32])
def test_the_backward_grows_by_chunks_alone(dtype):
    """A sequence more is a chunk more: two states and some 8 KB a head, nothing for segments."""
    n, H, P, N = 65536, 64, 64, 128
    at = lambda num: size("ttt_selective_scan_backward_workspace_bytes", n, num, dtype)
    per = H * (8 * P * N + 16 * 1024)
    for a, b in ((100, 101), (1024, 1025), (1024, 4096)):
        assert H * 8 * P * N * (b - a) <= at(b) - at(a) <= per * (b - a)
