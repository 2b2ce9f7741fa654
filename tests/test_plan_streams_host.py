"""Plans and streams, on the CPU: whose blocks a plan takes, and which streams the allocator is told of.

PyTorch's allocator hands a freed block out again as soon as the stream it
belongs to may use it.  An upload on another stream than the block's would run
into work still queued on the block's own, and a plan that is dropped while a
decode on another stream reads it would lose its buffers to the next plan.  CUDA
is replaced by a recorder here; test_gpu_plan_streams.py runs the calls.
"""
import contextlib
import types

import numpy as np
import pytest

from mla_latent_kv_02_gb300 import _build

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def api():
    if _build.is_stale():
        _build.build()
    from mla_latent_kv_02_gb300 import api as a
    a.mla_version()
    return a


class Stream:
    def __init__(self, raw):
        self.cuda_stream = raw


@pytest.fixture
def cuda(api, monkeypatch):
    """Streams by their handles: the current one, where each tensor was taken, and what is recorded."""
    rec = types.SimpleNamespace(now=7, taken={}, recorded=[], copied=[])

    @contextlib.contextmanager
    def stream(s):
        before, rec.now = rec.now, rec.now if s is None else s.cuda_stream
        yield
        rec.now = before

    empty, copy_ = torch.empty, torch.Tensor.copy_

    def taken(*args, **kw):
        t = empty(*args, **kw)
        rec.taken[t.data_ptr()] = rec.now
        return t

    def copied(self, src, non_blocking=False):
        rec.copied.append((self.data_ptr(), rec.now))
        return copy_(self, src)

    monkeypatch.setattr(torch, "empty", taken)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: Stream(rec.now))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw, device=None: Stream(raw))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(torch.Tensor, "pin_memory", lambda self: self)
    monkeypatch.setattr(torch.Tensor, "copy_", copied)
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda self, s: rec.recorded.append((self.data_ptr(), s.cuda_stream)), raising=False)
    monkeypatch.setattr(api, "_raw_stream", lambda dev: rec.now)
    return rec


def _plan(api, kind, **kw):
    if kind == "window":
        return api.mla_window_plan([500, 70], [1, 2], 100, 4, device="cpu", num_clusters=4, **kw)
    return api.mla_decode_plan([500, 70], [1, 2], device="cpu", num_clusters=4, **kw)


KINDS = ["window", "full"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("raw", [None, 11])
def test_buffers_are_those_of_the_uploading_stream(api, cuda, kind, raw):
    plan = _plan(api, kind, stream=None if raw is None else Stream(raw))
    want = 7 if raw is None else raw
    assert cuda.taken[plan.plan.data_ptr()] == want and cuda.taken[plan.workspace.data_ptr()] == want
    assert cuda.copied[-1] == (plan.plan.data_ptr(), want) and cuda.now == 7
    assert np.array_equal(plan.plan.numpy()[:16], plan.host.numpy()[:16]) and not cuda.recorded


@pytest.mark.parametrize("kind", KINDS)
def test_reused_buffers_are_recorded_on_the_uploading_stream(api, cuda, kind):
    first = _plan(api, kind)
    again = _plan(api, kind, stream=Stream(11), into=first)
    assert again.plan is first.plan and again.info is not first.info
    assert sorted(cuda.recorded) == sorted([(first.plan.data_ptr(), 11), (first.workspace.data_ptr(), 11)])
    _plan(api, kind, stream=Stream(11), into=again)          # told once
    assert len(cuda.recorded) == 2


class Lib:
    """A library whose decodes do nothing."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args[-1]))
            return 0
        return call


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kind", KINDS)
def test_the_decoding_stream_is_recorded_once(api, cuda, kind, fp8, monkeypatch):
    plan = _plan(api, kind, stream=Stream(11))
    lib = Lib()
    monkeypatch.setattr(api, "lib", lambda: lib)
    monkeypatch.setattr(api, "_need", lambda *a, **k: None)
    monkeypatch.setattr(api, "_in", lambda t, *a: t.data_ptr())
    T = 3
    q_abs, q_r = torch.zeros((T, 128, 512), dtype=torch.bfloat16), torch.zeros((T, 128, 64), dtype=torch.bfloat16)
    cache = [torch.zeros((1, 64, 640), dtype=torch.uint8), torch.zeros((1, 64))] if fp8 else \
        [torch.zeros((1, 64, 576), dtype=torch.bfloat16)]
    f = {("window", False): api.mla_decode_window, ("window", True): api.mla_decode_window_fp8,
         ("full", False): api.mla_decode_paged, ("full", True): api.mla_decode_paged_fp8}[kind, fp8]
    args = (q_abs, q_r, *cache, torch.zeros((2, 8), dtype=torch.int32), plan, torch.zeros_like(q_abs),
            torch.zeros(1, dtype=torch.int32))
    f(*args, stream=Stream(11))                              # the blocks' own stream
    assert not cuda.recorded
    for stream, raw in [(None, 7), (Stream(13), 13), (None, 7), (Stream(13), 13)]:
        f(*args, stream=stream)
        got = lib.calls[-1][1]
        assert getattr(got, "value", got) == raw
    both = [(t.data_ptr(), raw) for t in (plan.plan, plan.workspace) for raw in (7, 13)]
    assert sorted(cuda.recorded) == sorted(both)
