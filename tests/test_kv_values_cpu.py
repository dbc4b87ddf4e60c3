"""The batched INT4 KV cache on the host: the largest sizes that are taken."""
import ctypes

import pytest

import bit_weight_only_quantize_amd as w4

pytestmark = pytest.mark.cpu


def _pages(Hkv=1, D=64):
    return w4._W4KvPages(D, 4, Hkv, 16, 16, 16, 16, 16)


def _batch(rows, starts=16):
    return w4._W4KvBatch(1, rows, 0, 0, 16, starts, 16, 2, 2)


def _rows(rs, hs):
    return w4._W4Rows(16, 1, rs, hs)


@pytest.mark.parametrize("rows,heads", [(2 ** 31 - 4095, 1), (2 ** 31 - 1, 1), (2 ** 30 - 1000, 2), (2 ** 26 - 1, 32)])
def test_rows_that_positions_in_31_bits_would_pass(rows, heads):
    """Kernels step past the last row: rows * heads keeps a distance from 2^31, whatever the strides."""
    r = ctypes.byref
    L = w4.lib()
    few = _rows(64, 64)                                    # read by overlapping windows: memory would allow it
    assert L.w4_kv_write(r(_pages(heads)), r(_batch(rows)), r(few), None, None) == -2
    assert L.w4_kv_read(r(_pages(heads)), r(_batch(rows)), r(_rows(64 * heads, 64)), None, None) == -2
    q = _rows(64 * heads, 64)
    assert L.w4_kv_attention(r(_pages(1)), r(_batch(rows)), r(q), heads, 1.0, 0, 0, r(q), None, 16, 1 << 60, None) == -2
    assert L.w4_kv_attention_workspace_bytes(r(_pages(1)), r(_batch(rows)), heads, 0, 0) == 0


def test_largest_sizes_that_are_taken():
    """At the border the checks of the sizes pass: what is refused then is the missing tensor."""
    r = ctypes.byref
    L = w4.lib()
    assert L.w4_kv_write(r(_pages()), r(_batch(2 ** 31 - 4096)), None, None, None) == -1
    assert L.w4_kv_attention(r(_pages()), r(_batch(2 ** 30 - 2048)), None, 2, 1.0, 0, 0, None, None, None, 0, None) == -1
