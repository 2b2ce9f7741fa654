"""The package on a PyTorch that was built without CUDA: the host-only calls import and run."""
import os
import subprocess
import sys

import pytest

from mla_latent_kv_02_gb300 import _build

pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import torch
for name in [n for n in vars(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import numpy as np
from mla_latent_kv_02_gb300 import api
assert api.mla_decode_plan_host([700, 64], [2, 1], 4)[1].T == 3
assert api.mla_window_plan_host([700, 64], [2, 1], 100, 4, 4)[1].plan.T == 3
assert api.mla_prefill_window_workspace_size([300], [1000], 511, 4) > 0
pool = api.MlaPool(4)
ids = pool.alloc(2)
assert pool.available() == 2
assert api.mla_slot_mapping(np.array([ids]), np.array([0]), np.array([65]))[0] == int(ids[1]) * 64 + 1
print("fine")
"""


def test_host_calls_need_no_cuda_build():
    if _build.is_stale():
        _build.build()
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr[-2000:]
