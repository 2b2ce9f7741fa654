"""Windowed chunks whose query rows overlap: two sequences would write one row of the output (no GPU)."""
import ctypes as C

import numpy as np
import pytest

from mla_latent_kv_02_gb300 import _build, _lib


@pytest.fixture(scope="module")
def lib():
    if _build.is_stale():
        _build.build()
    return _lib.lib()


def _call(lib, starts, q, fp8):
    n = [max(m, 500) for m in q]
    arrs = [np.array(x, np.int32) for x in (range(len(q)), starts, q, n)]
    P32 = C.POINTER(C.c_int32)
    p = [C.c_void_p(0x10000 + 0x1000 * i) for i in range(9)]
    cache = (p[2], p[8]) if fp8 else (p[2],)
    f = lib.mla_prefill_window_batch_fp8 if fp8 else lib.mla_prefill_window_batch
    # a workspace too small ends every call that gets past the rows
    return f(p[0], p[1], *[a.ctypes.data_as(P32) for a in arrs], len(q), 100, 4, *cache, 100, p[3], 64, 64, p[4], p[5],
             0.07, p[6], 16, p[7], p[7], None), lib.mla_last_error().decode()


@pytest.mark.parametrize("fp8", [False, True])
def test_overlapping_rows_are_refused(lib, fp8):
    for starts, q in [([0, 0], [1, 1]), ([0, 299], [300, 10]), ([100, 0], [50, 101]), ([5, 900, 0], [20, 3, 6]),
                      ([0, 1], [500, 2]), (list(range(0, 640, 10)), [11] + [10] * 63)]:
        status, why = _call(lib, starts, q, fp8)
        assert status == 1 and "overlap" in why, (starts, q, why)
    for starts, q in [([0, 300], [300, 10]), ([300, 0], [10, 300]), ([7], [5]), (list(range(0, 640, 10)), [10] * 64)]:
        status, why = _call(lib, starts, q, fp8)
        assert status == 1 and "workspace" in why, (starts, q, why)
