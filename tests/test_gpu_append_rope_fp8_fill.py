"""The rotating FP8 append at the sizes of a fill, where a warp takes several tokens.

Codes, scales and keys are those of the separate calls bit for bit (every row),
and those of the oracle (a sample of rows, tolerances as in
test_gpu_append_rope_fp8.py).  A warp takes its second token above 19 456
tokens, the grid grows again from 175 104 on, and a query thread takes its
second chunk above 2 432 tokens.
"""
import numpy as np
import pytest

import oracle

from test_gpu_append_rope_fp8 import _turn

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
MAX_POS = 70001


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from mla_latent_kv_02_gb300 import api as a
    a.mla_version()
    return a


@pytest.fixture(scope="module")
def table(api):
    t = torch.empty((MAX_POS, 32, 2), dtype=torch.float32, device="cuda")
    api.mla_rope_table(MAX_POS, t)
    return t


def _inputs(n, queries, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    c = (rand(n, 512) * torch.exp2(torch.randint(-20, 8, (n, 1), generator=g, device="cuda").float())).to(torch.bfloat16)
    c[n // 2] = 0.0                                          # an all-zero row: k = 0
    k = rand(n, 64).to(torch.bfloat16)
    q = rand(n, 128, 64).to(torch.bfloat16) if queries else None
    pos = torch.randint(0, MAX_POS, (n,), generator=g, device="cuda", dtype=torch.int32)
    pages = n // 64 + 2
    slots = torch.randperm(pages * 64, generator=g, device="cuda")[:n]
    return c, k, q, pos, pages, slots


@pytest.mark.parametrize("n,queries", [(19456, False), (19457, False), (20000, False), (175103, False), (175104, False),
                                       (200000, False), (2432, True), (2433, True), (3000, True), (20001, True)])
def test_append_rope_fp8_fill(api, table, n, queries):
    c, k, q, pos, pages, slots = _inputs(n, queries, n)
    rows = torch.full((pages, 64, 640), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((pages, 64), 7.0, dtype=torch.float32, device="cuda")
    rows2, scales2 = rows.clone(), scales.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_r = torch.full_like(q, 5.0) if queries else None
    api.mla_kv_append_rope_fp8(c, k, pos, table, slots, rows, scales, err, q_pe=q, q_r=q_r)
    # the separate calls: keys rotated into bf16 rows, then appended as they are
    kv = torch.zeros((pages, 64, 576), dtype=torch.bfloat16, device="cuda")
    api.mla_kv_append_rope(c, k, pos, table, slots, kv, err)
    turned = kv.view(-1, 576)[slots, 512:].contiguous()
    api.mla_kv_append_fp8(c, turned, slots, rows2, scales2, err)
    assert api.mla_check(err) == 0
    assert torch.equal(rows, rows2) and torch.equal(scales, scales2)
    if queries:
        want = torch.empty_like(q)
        api.mla_rope_q(q, pos, table, want, err)
        assert api.mla_check(err) == 0 and torch.equal(q_r.view(torch.int16), want.view(torch.int16))
    # the oracle on the first and last tokens, around the turns of the loops, and some between
    at = sorted({i for e in (0, 2432, 9728, 19456, n // 2, n) for i in range(max(e - 40, 0), min(e + 40, n))} |
                set(range(0, n, max(n // 500, 1))))
    codes, sc = oracle.fp8_cache.quantize_rows(c[at].float().cpu().numpy())
    got = rows.view(-1, 640)[slots[at]].cpu().numpy()
    assert np.array_equal(got[:, :512], codes)
    assert np.array_equal(scales.view(-1)[slots[at]].cpu().numpy().astype(np.float64), np.asarray(sc))
    cs = table[pos[at].long()].cpu().numpy().astype(np.float64)
    y, tol = _turn(k[at].float().cpu().numpy(), cs)
    key = got[:, 512:].copy().view(np.uint16).astype(np.uint32) << 16
    assert (np.abs(key.view(np.float32).astype(np.float64) - y) <= tol).all()
    if queries:
        y, tol = _turn(q[at].float().cpu().numpy(), cs[:, None])
        assert (np.abs(q_r[at].float().cpu().numpy().astype(np.float64) - y) <= tol).all()
    rest = torch.ones(pages * 64, dtype=torch.bool, device="cuda")
    rest[slots] = False
    assert bool((rows.view(-1, 640)[rest] == 0xA5).all()) and bool((scales.view(-1)[rest] == 7.0).all())
