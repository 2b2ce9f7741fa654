"""Plans made on one stream and read on another, dropped as soon as their decode is queued.

Every step has other lengths, and the decoding stream is kept behind with
ordinary work, so that the plans of several steps exist only as queued work: a
block handed out too early would carry another step's plan or partials.  The
results have to be those of the same plans on one stream, bit for bit.
"""
import pytest

from test_gpu_window import Cache, _queries

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
STEPS = 8


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from mla_latent_kv_02_gb300 import api as a
    a.mla_version()
    return a


class Steps:
    """STEPS decode steps of three sequences that grow by one to three tokens a step."""

    def __init__(self, api, windowed, kind):
        self.api, self.windowed = api, windowed
        self.cache = Cache(api, [900, 1500, 700], kind, 81)
        self.q = [[1 + (i + b) % 3 for b in range(3)] for i in range(STEPS)]
        self.n = [[n - 60 + 7 * i for n in self.cache.n] for i in range(STEPS)]
        self.queries = [_queries(sum(q), 90 + i) for i, q in enumerate(self.q)]
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.clusters = api.mla_decode_max_clusters()

    def plan(self, i, stream=None):
        if self.windowed:
            return self.api.mla_window_plan(self.n[i], self.q[i], 300, 4, num_clusters=self.clusters, stream=stream)
        return self.api.mla_decode_plan(self.n[i], self.q[i], num_clusters=self.clusters, stream=stream)

    def outputs(self):
        return [(torch.zeros((sum(q), 128, 512), dtype=torch.bfloat16, device="cuda"),
                 torch.zeros((sum(q), 128), dtype=torch.float32, device="cuda")) for q in self.q]

    def decode(self, i, plan, out, stream=None):
        api, c = self.api, self.cache
        name = ("mla_decode_window" if self.windowed else "mla_decode_paged") + ("_fp8" if c.kind == "fp8" else "")
        cache = (c.kv,) if c.kind == "bf16" else (c.rows, c.scales)
        getattr(api, name)(*self.queries[i], *cache, c.table, plan, out[0], self.err, lse=out[1], stream=stream)


@pytest.fixture
def steps(api, request):
    s = Steps(api, *request.param)
    s.want = s.outputs()
    for i in range(STEPS):
        s.decode(i, s.plan(i), s.want[i])
    torch.cuda.synchronize()
    assert int(s.err.item()) == 0
    return s


def _keep_busy(x, times):
    """Ordinary work of some milliseconds on the current stream."""
    for _ in range(times):
        x = (x @ x).clamp_(-1, 1)
    return x


def _check(s, got):
    torch.cuda.synchronize()
    assert s.api.mla_check(s.err) == 0
    for i, ((o, lse), (wo, wl)) in enumerate(zip(got, s.want)):
        assert torch.equal(o, wo) and torch.equal(lse, wl), i


ALL = [(True, "bf16"), (True, "fp8"), (False, "bf16"), (False, "fp8")]


@pytest.mark.parametrize("steps", ALL, indirect=True)
def test_plans_uploaded_on_a_copy_stream(steps):
    copy, x = torch.cuda.Stream(), torch.rand((4096, 4096), device="cuda").to(torch.bfloat16)
    got = steps.outputs()
    torch.cuda.synchronize()
    for i in range(STEPS):
        _keep_busy(x, 20)
        plan = steps.plan(i, stream=copy)
        copy.record_event().wait()
        steps.decode(i, plan, got[i])
        del plan
    _check(steps, got)


@pytest.mark.parametrize("steps", ALL, indirect=True)
def test_plans_read_on_a_side_stream(steps):
    side, x = torch.cuda.Stream(), torch.rand((4096, 4096), device="cuda").to(torch.bfloat16)
    got = steps.outputs()
    torch.cuda.synchronize()
    for i in range(STEPS):
        plan = steps.plan(i)
        side.wait_event(torch.cuda.current_stream().record_event())
        with torch.cuda.stream(side):
            _keep_busy(x, 20)
            if i % 2:
                steps.decode(i, plan, got[i])
        if not i % 2:
            steps.decode(i, plan, got[i], stream=side)
        del plan
    _check(steps, got)


@pytest.mark.parametrize("steps", ALL[:3:2], indirect=True)
def test_plans_of_a_captured_step(steps):
    """The capturing stream is a stream like another: the plans are recorded there, and the caller keeps them."""
    plans, got = [steps.plan(i) for i in range(2)], steps.outputs()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i in range(2):
            steps.decode(i, plans[i], got[i])
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert steps.api.mla_check(steps.err) == 0
    for i in range(2):
        assert torch.equal(got[i][0], steps.want[i][0]) and torch.equal(got[i][1], steps.want[i][1])
    del g, plans
    for i in range(2, STEPS):                                # the freed blocks go on to other plans
        steps.decode(i, steps.plan(i), got[i])
    _check(steps, got)
