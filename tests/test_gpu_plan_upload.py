"""The C planners that upload, mla_decode_plan and mla_window_plan: what arrives, and a decode with it."""
import ctypes as C

import numpy as np
import pytest

from mla_latent_kv_02_gb300 import _lib

from test_gpu_window import Cache, _check_decode, _decode, _queries

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
P32 = C.POINTER(C.c_int32)


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from mla_latent_kv_02_gb300 import api as a
    a.mla_version()
    return a


def _upload(seq, q, window, sinks, clusters, plan, stream):
    """(status, info) of mla_window_plan, or of mla_decode_plan where window is None."""
    sl, ql = np.array(seq, np.int32), np.array(q, np.int32)
    head = (sl.ctypes.data_as(P32), ql.ctypes.data_as(P32), len(seq))
    tail = (clusters, C.c_void_p(plan.data_ptr()), plan.numel() * 4)
    if window is None:
        info = _lib.mla_plan_info()
        return _lib.lib().mla_decode_plan(*head, *tail, C.byref(info), C.c_void_p(stream.cuda_stream)), info
    info = _lib.mla_window_info()
    return _lib.lib().mla_window_plan(*head, window, sinks, *tail, C.byref(info), C.c_void_p(stream.cuda_stream)), info


def _host(api, seq, q, window, sinks, clusters):
    return api.mla_decode_plan_host(seq, q, clusters) if window is None else \
        api.mla_window_plan_host(seq, q, window, sinks, clusters)


CASES = [([700, 900, 333], [2, 1, 2], 257, 6, 5), ([64 * 40 + 1], [1], 64, 1, 2), ([1], [1], 1, 0, 76),
         ([700, 900, 333], [2, 1, 2], None, None, 5), (list(range(1, 400)), [1] * 399, 50, 4, 76)]


@pytest.mark.parametrize("side", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_uploaded_plan_is_the_host_plan(api, case, side):
    seq, q, window, sinks, clusters = CASES[case]
    want, winfo = _host(api, seq, q, window, sinks, clusters)
    stream = torch.cuda.Stream() if side else torch.cuda.current_stream()
    plan = torch.full((want.size + 9,), -7, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    status, info = _upload(seq, q, window, sinks, clusters, plan, stream)
    assert status == 0 and bytes(info) == bytes(winfo)
    torch.cuda.synchronize()
    words = (winfo if window is None else winfo.plan).plan_bytes // 4
    got = plan.cpu().numpy()
    assert np.array_equal(got[:words], want[:words]) and (got[words:] == -7).all()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_decode_with_an_uploaded_plan(api, kind):
    seq, q, window, sinks, clusters = CASES[0]
    cache = Cache(api, seq, kind, 91)
    q_abs, q_r = _queries(sum(q), 92)
    py = api.mla_window_plan(seq, q, window, sinks, num_clusters=clusters)
    status, info = _upload(seq, q, window, sinks, clusters, py.plan.zero_(), torch.cuda.current_stream())
    assert status == 0
    py.info = info
    o, lse, err = _decode(api, cache, q_abs, q_r, py)
    assert api.mla_check(err) == 0
    _check_decode(cache, q_abs, q_r, o, lse, q, window, sinks)


@pytest.mark.parametrize("case", [0, 3])
def test_upload_into_a_capture_is_refused(api, case):
    """The copy's source is the call's own memory, gone when a captured copy is replayed."""
    seq, q, window, sinks, clusters = CASES[case]
    want, winfo = _host(api, seq, q, window, sinks, clusters)
    plan = torch.full((want.size,), -7, dtype=torch.int32, device="cuda")
    x = torch.zeros(4, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x.add_(1)
        status, _ = _upload(seq, q, window, sinks, clusters, plan, torch.cuda.current_stream())
    assert status == 3 and b"capture" in _lib.lib().mla_last_error()
    g.replay()                                               # the capture itself goes on
    torch.cuda.synchronize()
    assert x.tolist() == [1.0] * 4 and bool((plan == -7).all())
    assert _upload(seq, q, window, sinks, clusters, plan, torch.cuda.current_stream())[0] == 0
