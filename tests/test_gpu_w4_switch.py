"""The 4-bit projections around the token counts where their kernels and tiles change.

Up to 8, 16 and 32 tokens take one, two and four token tiles of eight; more take
128-token tiles.  Bounds as in test_gpu_w4.py.
"""
import numpy as np
import pytest

from _helpers import to_bf16
from _window_ref import bf16
from test_gpu_w4 import SHAPES, _call, _check, _random_weights

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from mla_latent_kv_02_gb300 import api as a
    a.mla_version()
    return a


@pytest.mark.parametrize("T", [7, 15, 18, 24, 25, 31, 32, 33, 40, 64, 65, 96, 97, 160])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("kind", ["absorb", "up"])
def test_w4_around_the_switch(api, kind, group, T):
    K, N = SHAPES[kind]
    words, scales = _random_weights(K, N, group, 10 * T + group)
    x = to_bf16(bf16(np.random.default_rng(T), (T, 128, K)), "cuda")
    guard = torch.full((T + 2, 128, N), 3.0, dtype=torch.bfloat16, device="cuda")
    out = guard[1:T + 1]
    out.fill_(float("nan"))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    _call(api, kind, x, words, scales, out, err)
    assert api.mla_check(err) == 0
    _check(x, words, scales, out)
    assert bool((guard[0] == 3.0).all()) and bool((guard[-1] == 3.0).all()), "a row past T was written"
