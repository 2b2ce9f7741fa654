"""Windowed chunks and decodes in flight at once on several streams, each with its own workspace.

The chunk form's kernels are launched early behind one another; a call must wait
for its own kernels, whatever else the GPU runs.  Results are those of the same
calls alone, bit for bit.
"""
import numpy as np
import pytest

from _helpers import to_bf16
from _window_ref import bf16
from test_gpu_window import Cache, _queries, _weights

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from mla_latent_kv_02_gb300 import api as a
    a.mla_version()
    return a


class Chunks:
    def __init__(self, api, kind, n, q, window, sinks, seed):
        self.api, self.args = api, (q, n, window, sinks)
        self.cache = Cache(api, n, kind, seed)
        rng = np.random.default_rng(seed)
        T = sum(q)
        self.q_c, self.q_r = to_bf16(bf16(rng, (T, 128, 128)), "cuda"), to_bf16(bf16(rng, (T, 128, 64)), "cuda")
        self.weights = _weights(seed)
        self.starts = [sum(q[:i]) for i in range(len(q))]
        self.ws = torch.empty(api.mla_prefill_window_workspace_size(*self.args), dtype=torch.uint8, device="cuda")
        self.out = torch.empty((T, 128, 128), dtype=torch.bfloat16, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, stream=None):
        q, n, window, sinks = self.args
        c = self.cache
        tail = (c.table, range(len(n)), self.starts, q, n, window, sinks, *self.weights, self.ws, self.out, self.err)
        if c.kind == "bf16":
            self.api.mla_prefill_window_batch(self.q_c, self.q_r, c.kv, *tail, stream=stream)
        else:
            self.api.mla_prefill_window_batch_fp8(self.q_c, self.q_r, c.rows, c.scales, *tail, stream=stream)


class Decodes:
    def __init__(self, api, kind, seed):
        seq, q = [900, 2000, 333], [2, 1, 2]
        self.api, self.cache, self.q = api, Cache(api, seq, kind, seed), _queries(sum(q), seed)
        self.plan = api.mla_window_plan(seq, q, 400, 5)
        self.out = torch.empty((sum(q), 128, 512), dtype=torch.bfloat16, device="cuda")
        self.lse = torch.empty((sum(q), 128), device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, stream=None):
        c = self.cache
        cache = (c.kv,) if c.kind == "bf16" else (c.rows, c.scales)
        f = self.api.mla_decode_window if c.kind == "bf16" else self.api.mla_decode_window_fp8
        f(*self.q, *cache, c.table, self.plan, self.out, self.err, lse=self.lse, stream=stream)


@pytest.mark.parametrize("captured", [False, True])
def test_calls_in_flight_at_once(api, captured):
    calls = [Chunks(api, "fp8", [1000, 700], [300, 256], 200, 4, 3), Chunks(api, "bf16", [1500], [600], 333, 64, 4),
             Decodes(api, "bf16", 5), Decodes(api, "fp8", 6)]
    for c in calls:
        c.run()
    torch.cuda.synchronize()
    want = [c.out.clone() for c in calls]
    graphs = []
    if captured:
        for c in calls:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                c.run()
                c.run()
            graphs.append(g)
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        for c in calls:
            c.out.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(6):
            for i, (c, s) in enumerate(zip(calls, streams)):
                if captured:
                    with torch.cuda.stream(s):
                        graphs[i].replay()
                else:
                    c.run(stream=s)
        torch.cuda.synchronize()
        for i, (c, w) in enumerate(zip(calls, want)):
            assert int(c.err.item()) == 0 and torch.equal(c.out, w), i
