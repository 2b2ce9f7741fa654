"""Scales that fp16 does not hold: hidden tokens still have weight 0, seen ones nearly equal weights.

At a scale of 1e-6 or less, with raw scores under 2^9, the natural-log distances are under 2^-10 and
a weight's error is that of its roundings: P in bf16 and 2^x (2^-8 + 2^-9), the exponent and the
lagging reference (under 8 units of 2^-11), the factor of the exponent, at most 2^-24 off
(|raw| 2^-24 + M 2^-24 for lse, M the row's largest |raw|).
"""
import math

import pytest

from _tree_ref import masks, path, tree
from test_gpu_tree import Cache, queries, word
from _window_ref import seen_positions

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from mla_latent_kv_02_gb300 import api as a
    a.mla_version()
    return a


def check(cache, q_abs, q_r, o, lse, b, t, at, scale):
    c, r = cache.tokens(b, at)
    raw = q_abs[t].double() @ c.T + q_r[t].double() @ r.T
    top = raw.abs().amax(dim=-1, keepdim=True)
    assert float(top.max()) < 512
    p = torch.softmax(raw * scale, dim=-1)
    eps = 2.0 ** -8 + 2.0 ** -9 + 8 * math.log(2.0) * 2.0 ** -11 + (raw.abs() + top) * 2.0 ** -24 + raw.abs() * 3 * scale * 2.0 ** -11
    want = p @ c
    tol = 1.05 * ((p * eps) @ c.abs() + want.abs() * (p * eps).sum(-1, keepdim=True) + 2.0 ** -8 * want.abs()) + 1e-6
    assert bool(((o[t].double() - want).abs() <= tol).all()), t
    l = torch.logsumexp(raw * scale, dim=-1)
    assert bool(((lse[t].double() - l).abs() <= 1.05 * (p * eps).sum(-1) + 2.0 ** -22 * l.abs() + 1e-6).all()), (t, "lse")


@pytest.mark.parametrize("scale", [1e-6, 3e-8, 1e-9, 1e-38])
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("form", ["full", "window", "tree", "tree_unpacked"])
def test_decode(api, form, kind, scale):
    if form == "tree_unpacked":
        ctx, nodes = [1500], [40]
    else:
        ctx, nodes = [70, 0, 205], [3, 2, 5]
    cache = Cache(api, [n + q for n, q in zip(ctx, nodes)], kind, 5)
    if kind == "bf16":                                       # the full decode wants finite slots
        cache.kv.nan_to_num_(0.0)
    else:
        empty = torch.isnan(cache.scales)
        cache.rows[empty] = 0
        cache.scales[empty] = 1.0
    T = sum(nodes)
    q_abs, q_r = queries(T, 6)
    trees = [tree(b, n, 2, 4) for b, n in enumerate(nodes)]
    o = torch.full((T, 128, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse, err = torch.full((T, 128), float("nan"), dtype=torch.float32, device="cuda"), word()
    store = (cache.kv,) if kind == "bf16" else (cache.rows, cache.scales)
    suffix = "" if kind == "bf16" else "_fp8"
    if form == "full":
        api_call, plan, rest = "mla_decode_paged", api.mla_decode_plan(cache.n, nodes), ()
    elif form == "window":
        api_call, plan, rest = "mla_decode_window", api.mla_window_plan(cache.n, nodes, 50, 2), ()
    else:
        m = torch.from_numpy(masks(trees, 1)).cuda()
        api_call, plan, rest = "mla_decode_tree", api.mla_tree_plan(cache.n, nodes), (m,)
    getattr(api, api_call + suffix)(q_abs, q_r, *store, cache.table, *rest, plan, o, err, lse=lse, scale=scale)
    assert api.mla_check(err) == 0
    t = 0
    for b, q in enumerate(nodes):
        for i in range(q):
            p = ctx[b] + i
            if form == "full":
                at = list(range(p + 1))
            elif form == "window":
                at = seen_positions(p, 50, 2)
            else:
                at = list(range(ctx[b])) + [ctx[b] + k for k in path(trees[b], i)]
            if T < 20 or i % 13 == 0:
                check(cache, q_abs, q_r, o, lse, b, t, at, scale)
            t += 1


@pytest.mark.parametrize("scale", [3e-8, 1e-38])
def test_chunk(api, scale):
    """Chunks with and without a window: nearly equal weights over what a row sees.  K_c and V_c are rounded to bf16
    (V_c 2^-8 of the output), P and out as in the decode."""
    M, N = 40, 230
    g = torch.Generator(device="cuda")
    g.manual_seed(3)

    def rand(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)

    kv, w_uk, w_uv = rand(4, 64, 576), rand(128, 128, 512, std=0.04), rand(128, 512, 128, std=0.04)
    q_c, q_r, out, err = rand(M, 128, 128), rand(M, 128, 64), rand(M, 128, 128), word()
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    c = kv.view(-1, 576)[:N, :512].double()
    for window in (None, (60, 3)):
        args = ([M], [N])
        if window is None:
            ws = torch.empty(api.mla_prefill_batch_workspace_size([N]), dtype=torch.uint8, device="cuda")
            api.mla_prefill_decompress_batch(q_c, q_r, kv, table, [0], [0], [M], [N], w_uk, w_uv, ws, out, err, scale=scale)
        else:
            ws = torch.empty(api.mla_prefill_window_workspace_size(*args, *window), dtype=torch.uint8, device="cuda")
            api.mla_prefill_window_batch(q_c, q_r, kv, table, [0], [0], [M], [N], *window, w_uk, w_uv, ws, out, err, scale=scale)
        assert api.mla_check(err) == 0
        for row in (0, 1, 20, M - 1):
            p = N - M + row
            at = torch.tensor(seen_positions(p, *window) if window else list(range(p + 1)), device="cuda")
            for h in (0, 77):
                v = c[at] @ w_uv[h].double()
                want = v.mean(dim=0)
                tol = 1.05 * ((2.0 ** -8 + 2.0 ** -9 + 8 * math.log(2.0) * 2.0 ** -11 + 2.0 ** -14 + 2.0 ** -8) *
                              (v.abs().mean(dim=0) + want.abs()) + 2.0 ** -8 * want.abs()) + 1e-6
                assert bool(((out[row, h].double() - want).abs() <= tol).all()), (window, row, h)
