"""Windowed decodes whose waits may run out: a call that reports nothing has to be right."""
import pytest

from test_gpu_window import Cache, _check_decode, _decode, _queries

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from mla_latent_kv_02_gb300 import api as a
    a.mla_version()
    return a


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("limit", [64, 3000, 5000, 8000, 12000, 20000, 40000, 1 << 20])
def test_a_call_within_its_waits_is_right(api, kind, limit):
    seq, q, window, sinks = [700, 900, 333], [2, 1, 2], 257, 6
    cache = Cache(api, seq, kind, 25)
    q_abs, q_r = _queries(5, 26)
    plan = api.mla_window_plan(seq, q, window, sinks, num_clusters=3)
    calls = []
    try:
        api.mla_debug_set_decode_wait_limit(limit)
        for _ in range(3):
            calls.append(_decode(api, cache, q_abs, q_r, plan))
            torch.cuda.synchronize()
    finally:
        api.mla_debug_set_decode_wait_limit(0)
    words = [int(err.item()) for _, _, err in calls]
    assert all(w in (0, api.DEVERR_TIMEOUT) for w in words)
    if limit == 64:
        assert all(words)
    if limit == 1 << 20:                                     # half a millisecond, a tile takes one or two microseconds
        assert not any(words)
    for (o, lse, _), w in zip(calls, words):
        if w == 0:
            _check_decode(cache, q_abs, q_r, o, lse, q, window, sinks)
    o, lse, err = _decode(api, cache, q_abs, q_r, plan)
    assert api.mla_check(err) == 0
    _check_decode(cache, q_abs, q_r, o, lse, q, window, sinks)
