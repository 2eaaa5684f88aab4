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
