"""Sizes whose launch would hold 2^32 threads or more in its grid's one dimension are refused: the
runtime does not refuse them, it leaves workgroups out. Addresses are fake; the refusal comes
before anything is launched."""
import ctypes

import pytest

import gated_deltanet_linear_prefill_amd as gdn

SHAPE = 2
ADDR = [(1 << 42) + (i << 42) for i in range(10)]


def dims(n, t, h_qk, h_v, d, dtype=gdn.GDN_BF16):
    return ctypes.byref(gdn.Dims(n, t, h_qk, h_v, d, d, dtype, 1e-6))


# (sequence, V head) pairs: workgroups of 256 threads (64 of them a pair for d = 16 in decode)
@pytest.mark.parametrize("n,h,d", [(1 << 22, 16, 16), (1 << 20, 16, 32), (1 << 20, 32, 64), (1 << 21, 32, 128)])
def test_decode(n, h, d):
    assert gdn._load().gdn_decode_step(dims(n, 1, h, h, d), *ADDR[:8], None) == SHAPE


@pytest.mark.parametrize("n,h,d", [(1 << 20, 16, 16), (1 << 19, 16, 32), (1 << 18, 16, 64), (1 << 16, 32, 128)])
def test_scan(n, h, d):
    assert gdn._load().gdn_prefill_scan(dims(n, 1, h, h, d), *ADDR[:8], None, 0, None) == SHAPE


def test_scan_blockwise():
    d = dims(1, 1, 1 << 24, 1 << 24, 16)
    assert gdn._load().gdn_prefill_scan_blockwise(d, 1, *ADDR[:8], None, 0, None) == SHAPE


# the preparation of many chunks; the sequential pass of many heads
@pytest.mark.parametrize("n,t,h,d,chunk", [(1, 1 << 24, 16, 16, 16), (1, 1 << 25, 16, 16, 32), (16, 1 << 22, 16, 16, 64),
                                           (1 << 20, 1, 16, 16, 16), (1 << 18, 1, 16, 64, 64), (1 << 18, 1, 32, 128, 64),
                                           (1 << 18, 1, 32, 128, 128), (1 << 18, 1, 32, 128, 16)])
@pytest.mark.parametrize("dtype", [gdn.GDN_BF16, gdn.GDN_F32])
def test_chunked(n, t, h, d, chunk, dtype):
    x = dims(n, t, h, h, d, dtype)
    ws = gdn._load().gdn_workspace_bytes(x, chunk)
    assert ws > 0
    assert gdn._load().gdn_prefill_chunked(x, chunk, *ADDR[:9], ws, None) == SHAPE
