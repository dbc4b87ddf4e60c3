"""The batched INT4 KV cache on the host: refusals before anything is launched, and
the oracle's attention against closed forms."""
import ctypes

import numpy as np
import pytest

import bit_weight_only_quantize_amd as w4
import oracle

pytestmark = pytest.mark.cpu


def _pages(D=128, num_pages=4, Hkv=2, page_size=16, kc=16, ks=16, vc=16, vs=16):
    return w4._W4KvPages(D, num_pages, Hkv, page_size, kc, ks, vc, vs)


def _batch(B=2, rows=2, max_rows=0, max_len=0, lens=16, starts=None, table=16, width=2, stride=2):
    return w4._W4KvBatch(B, rows, max_rows, max_len, lens, starts, table, width, stride)


def _rows(data=16, dtype=0, rs=256, hs=128):
    return w4._W4Rows(data, dtype, rs, hs)


def _write(p, b, k=None, v=None, read=False):
    f = w4.lib().w4_kv_read if read else w4.lib().w4_kv_write
    r = lambda x: None if x is None else ctypes.byref(x)
    return f(r(p), r(b), r(k), r(v), None)


def _attend(p, b, q=None, out=None, Hq=4, scale=1.0, window=0, sinks=0, lse=None, ws=None, nbytes=0):
    r = lambda x: None if x is None else ctypes.byref(x)
    return w4.lib().w4_kv_attention(r(p), r(b), r(q), Hq, scale, window, sinks, r(out), lse, ws, nbytes, None)


def test_nothing_to_do():
    assert _write(_pages(), _batch(B=0, rows=0), _rows()) == 0
    assert _write(_pages(), _batch(rows=0), None, None) == 0
    assert _attend(_pages(), _batch(rows=0)) == 0


@pytest.mark.parametrize("p,b,code", [
    (None, _batch(), -1), (_pages(), None, -1),
    (_pages(D=96), _batch(), -2), (_pages(D=0), _batch(), -2),
    (_pages(Hkv=0), _batch(), -2), (_pages(num_pages=0), _batch(), -2), (_pages(page_size=0), _batch(), -2),
    (_pages(page_size=24), _batch(), -2), (_pages(page_size=8), _batch(), -2),      # with a table
    (_pages(page_size=24), _batch(table=None, B=5, rows=5), -2),                     # fewer pages than sequences
    (_pages(), _batch(B=-1), -2), (_pages(), _batch(rows=-1), -2), (_pages(), _batch(max_rows=-1), -2),
    (_pages(), _batch(max_len=-1), -2), (_pages(), _batch(rows=3), -2),              # 3 rows over 2 sequences
    (_pages(), _batch(width=0), -2), (_pages(), _batch(width=3), -2),                # wider than its stride
    (_pages(), _batch(width=2 ** 28, stride=2 ** 28), -2),                           # positions past 31 bits
    (_pages(page_size=2 ** 31 - 64, num_pages=2), _batch(table=None), -2),
    (_pages(num_pages=2 ** 30, page_size=2 ** 26, Hkv=64), _batch(), -2),
    (_pages(), _batch(rows=2 ** 31), -2), (_pages(), _batch(B=2 ** 21, rows=2 ** 21), -2),
    (_pages(kc=None), _batch(), -1), (_pages(vs=None), _batch(), -1), (_pages(), _batch(lens=None), -1),
    (_pages(kc=8), _batch(), -3), (_pages(vs=20), _batch(), -3), (_pages(), _batch(lens=18), -3),
    (_pages(), _batch(table=17), -3), (_pages(), _batch(starts=18), -3),
])
def test_cache_and_batch_refusals(p, b, code):
    assert _write(p, b, _rows(), _rows()) == code
    assert _write(p, b, _rows(), _rows(), read=True) == code
    assert _attend(p, b, _rows(rs=512), _rows(rs=512), ws=16, nbytes=1 << 30) == code
    assert len(w4.lib().w4_last_error()) > 0
    r = lambda x: None if x is None else ctypes.byref(x)
    assert w4.lib().w4_kv_attention_workspace_bytes(r(p), r(b), 4, 0, 0) == 0


@pytest.mark.parametrize("t,code", [
    (_rows(data=None), -1), (_rows(dtype=2), -1), (_rows(data=24), -3), (_rows(rs=258), -3), (_rows(hs=130), -3),
    (_rows(dtype=1, hs=132), -3), (_rows(rs=-256), -2), (_rows(hs=-128), -2), (_rows(rs=2 ** 41), -2),
])
def test_row_tensor_refusals(t, code):
    for read in (False, True):
        assert _write(_pages(), _batch(), t, _rows(), read) == code
        assert _write(_pages(), _batch(), _rows(), t, read) == code
    big = dict(Hq=4, ws=16, nbytes=1 << 30)
    assert _attend(_pages(), _batch(), t, _rows(rs=512), **big) == code
    assert _attend(_pages(), _batch(), _rows(rs=512), t, **big) == code


def test_written_rows_must_not_overlap():
    for t in (_rows(rs=0), _rows(hs=0), _rows(rs=128), _rows(hs=64, rs=256), _rows(rs=252)):
        assert _write(_pages(), _batch(), t, None, read=True) == -2
        assert b"overlap" in w4.lib().w4_last_error()
        assert _attend(_pages(), _batch(), _rows(rs=512), t, Hq=2, ws=16, nbytes=1 << 30) == -2


def test_attention_refusals():
    p, b, q = _pages(), _batch(), _rows(rs=512)
    big = dict(ws=16, nbytes=1 << 30)
    assert _write(p, b) == -1                                                        # neither k nor v
    assert _attend(p, b, None, q, **big) == -1 and _attend(p, b, q, None, **big) == -1
    for Hq in (0, -2, 3, 2 ** 31):
        assert _attend(p, b, q, q, Hq=Hq, **big) == -2
    assert _attend(p, b, q, q, window=-1, **big) == -2 and _attend(p, b, q, q, sinks=-1, **big) == -2
    for scale in (float("nan"), float("inf")):
        assert _attend(p, b, q, q, scale=scale, **big) == -1
    assert _attend(p, b, q, q, lse=24, **big) == -3


def test_attention_workspace():
    """Few sequences over a long cache split their keys and need a workspace, whose absence is refused."""
    L = w4.lib()
    p, b, q = _pages(page_size=4096, num_pages=64), _batch(width=32, stride=32), _rows(rs=512)
    need = L.w4_kv_attention_workspace_bytes(ctypes.byref(p), ctypes.byref(b), 4, 0, 0)
    assert need > 0
    assert _attend(p, b, q, q) == -5 and _attend(p, b, q, q, ws=16, nbytes=need - 1) == -5
    assert b"workspace" in L.w4_last_error()
    assert _attend(p, b, q, q, ws=8, nbytes=need) == -3
    # the largest windows and sinks are those that reach past every position
    for big in (2 ** 31, 2 ** 62, 2 ** 63 - 1):
        assert L.w4_kv_attention_workspace_bytes(ctypes.byref(p), ctypes.byref(b), 4, big, big) == need
        assert L.w4_kv_attention_workspace_bytes(ctypes.byref(p), ctypes.byref(b), 4, 0, big) == need
    # a window leaves little to split; a bound on the lengths as well
    assert L.w4_kv_attention_workspace_bytes(ctypes.byref(p), ctypes.byref(b), 4, 64, 4) < need
    short = _batch(width=32, stride=32, max_len=100)
    assert L.w4_kv_attention_workspace_bytes(ctypes.byref(p), ctypes.byref(short), 4, 0, 0) < need


def test_oracle_attention_against_closed_forms():
    rng = np.random.default_rng(0)
    v = rng.standard_normal((2, 9, 4))
    # equal scores: the mean of what is visible
    out, lse, *_ = oracle.kv_attention(np.zeros((3, 2, 4)), rng.standard_normal((2, 9, 4)), v, 1.0)
    for i in range(3):
        for h in range(2):
            assert np.allclose(out[i, h], v[h, :7 + i].mean(0)) and np.isclose(lse[i, h], np.log(7 + i))
    out, lse, *_ = oracle.kv_attention(np.zeros((1, 4, 4)), np.zeros((2, 9, 4)), v, 1.0, window=3, sinks=2)
    assert np.allclose(out[0, 3], v[1, [0, 1, 6, 7, 8]].mean(0)) and np.allclose(lse, np.log(5))
    # one dominant key; rows before the first position see nothing
    k = np.zeros((1, 5, 4))
    k[0, 2] = 100
    out, lse, *_ = oracle.kv_attention(np.ones((7, 1, 4)), k, v[:1, :5], 1.0)
    assert np.all(out[:2] == 0) and np.all(np.isneginf(lse[:2]))
    assert np.allclose(out[6, 0], v[0, 2]) and np.isclose(lse[6, 0], 400)
