"""The C planners that upload: refused, not thrown out of, whatever the buffer's size is said to be (no GPU)."""
import os
import subprocess
import sys

import pytest

from mla_latent_kv_02_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SCRIPT = """
import ctypes as C, sys
import numpy as np
from mla_latent_kv_02_gb300 import _lib
lib, P32 = _lib.lib(), C.POINTER(C.c_int32)
kind, seq, q, nbytes = sys.argv[1], int(sys.argv[2]), int(sys.argv[3]), int(sys.argv[4])
sl, ql = np.array([seq], np.int32), np.array([q], np.int32)
head, tail = (sl.ctypes.data_as(P32), ql.ctypes.data_as(P32), 1), (4, C.c_void_p(0x10000), nbytes)
if kind == "full":
    st = lib.mla_decode_plan(*head, *tail, C.byref(_lib.mla_plan_info()), None)
else:
    st = lib.mla_window_plan(*head, 100, 4, *tail, C.byref(_lib.mla_window_info()), None)
print(st)
"""


@pytest.fixture(scope="module", autouse=True)
def built():
    if _build.is_stale():
        _build.build()


@pytest.mark.parametrize("kind", ["full", "window"])
@pytest.mark.parametrize("seq,q,nbytes", [(500, 600, 1 << 62), (500, 600, 2 ** 64 - 1), (500, -1, 1 << 62), (500, 1, 16),
                                          (2 ** 31 - 1, 2 ** 31 - 1, 1 << 62)])
def test_upload_is_refused_whatever_the_size(kind, seq, q, nbytes):
    r = subprocess.run([sys.executable, "-c", SCRIPT, kind, str(seq), str(q), str(nbytes)], cwd=ROOT, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "1", (r.returncode, r.stdout, r.stderr[-500:])
