"""Limits of the 8-bit cache calls that the C ABI checks before it launches anything (no GPU, no memory behind
the pointers)."""
import ctypes

import pytest


@pytest.mark.parametrize("n_seqs,total_q,max_q,heads,nq", [
    (1, 2 ** 31 - 1, 2 ** 31 - 1, 2, 4),      # 2^32 rows of one sequence
    (2, 2 ** 31 - 1, 2 ** 30 + 1, 1, 2),      # 2^31 rows of the longer one
    (2, 2 ** 31 - 1, 2 ** 22, 2048, 65536),   # few enough rows a sequence, too many items in the step
])
def test_too_many_rows_are_unsupported(qlin, n_seqs, total_q, max_q, heads, nq):
    p, at = 1 << 20, ctypes.addressof
    c = qlin.KvCacheStruct(qlin.KV_INT8, 8, heads, 64, 32, p, p)
    b = qlin.KvBatchStruct(n_seqs, total_q, max_q, 100, 4, 4, p, p, p)
    q = qlin.HeadsStruct(p, 128, 64)
    st = qlin.lib().qlin_kv_attend(at(c), at(b), at(q), nq, 0.125, 0, 0, p, None, p, 1 << 40, None)
    assert st == qlin.QLIN_ERR_UNSUPPORTED


@pytest.mark.parametrize("window,sinks,width,ok", [
    (2 ** 30 + 1, 0, 2 ** 26 - 1, False),       # a table of 2^31 - 32 tokens, a window that hides half of them
    (100, 2 ** 30 + 1, 2 ** 26 - 1, False),
    (2 ** 31 - 1, 0, 2 ** 26 - 1, True),        # covers the table
    (100, 2 ** 31 - 1, 2 ** 26 - 1, True),
    (2 ** 31 - 1, 2 ** 31 - 1, 4, True),
    (0, 2 ** 31 - 1, 2 ** 26 - 1, True),        # no window
    (2 ** 30, 2 ** 30, 2 ** 26 - 1, True),
])
def test_windows_past_the_range(qlin, window, sinks, width, ok):
    p, at = 1 << 20, ctypes.addressof
    c = qlin.KvCacheStruct(qlin.KV_INT8, 8, 2, 64, 32, p, p)
    q = qlin.HeadsStruct(p, 128, 64)
    b = qlin.KvBatchStruct(1, 1, 1, 100, width, width, p, p, p)
    # (an output that is not aligned is refused behind the check of the window, before any launch)
    st = qlin.lib().qlin_kv_attend(at(c), at(b), at(q), 4, 0.125, window, sinks, p + 4, None, p, 1 << 40, None)
    assert st == (qlin.QLIN_ERR_INVALID_ARG if ok else qlin.QLIN_ERR_UNSUPPORTED)
