"""The rotating append of the FP8 cache against the oracle.

Codes and scales are integer work (a power-of-two scale), so they equal the
oracle's bit for bit.  The rotation is fp32 with one bf16 rounding: against
the 64-bit rotation by the same table entries a result may be off by half a
bf16 step of its value (2^-8 relative) and by the two fp32 roundings before
it, at most 2 * 2^-24 * (|x0| + |x1|) since |cos|, |sin| <= 1.
"""
import numpy as np
import pytest

import oracle
from mla_latent_kv_02_gb300 import workloads as wl

from _helpers import to_bf16, to_np

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
f8 = oracle.fp8_cache
MAX_POS = 9001


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


def _turn(x, cs):
    """64-bit rotation of pairs and the bound of the kernel's error."""
    a, b = x[..., 0::2].astype(np.float64), x[..., 1::2].astype(np.float64)
    y = np.empty(x.shape, np.float64)
    y[..., 0::2] = a * cs[..., 0] - b * cs[..., 1]
    y[..., 1::2] = a * cs[..., 1] + b * cs[..., 0]
    tol = np.abs(y) * 2.0 ** -8 + 2.0 * 2.0 ** -24 * np.repeat(np.abs(a) + np.abs(b), 2, axis=-1)
    return y, tol


def _inputs(n, seed):
    rng = np.random.default_rng(seed)
    c = wl.bf16_round(rng.standard_normal((n, 512), dtype=np.float32) *
                      np.exp2(rng.integers(-20, 8, (n, 1))).astype(np.float32))
    if n > 2:
        c[n // 2] = 0.0                                     # an all-zero row: k = 0
    k = wl.bf16_round(rng.standard_normal((n, 64), dtype=np.float32))
    q = wl.bf16_round(rng.standard_normal((n, 128, 64), dtype=np.float32) * 4)
    pos = rng.integers(0, MAX_POS, n).astype(np.int32)
    pos[0] = MAX_POS - 1
    pages = n // 64 + 2
    slots = rng.permutation(pages * 64)[:n].astype(np.int64)
    return c, k, q, pos, pages, slots


def _run(api, table, c, k, q, pos, pages, slots, stream=None):
    n = c.shape[0]
    rows = torch.full((pages, 64, 640), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((pages, 64), 7.0, dtype=torch.float32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_r = None if q is None else torch.full((n, 128, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    args = (to_bf16(c, "cuda"), to_bf16(k, "cuda"), torch.from_numpy(pos).cuda(), table, torch.from_numpy(slots).cuda(),
            rows, scales, err)
    kw = dict(q_pe=None if q is None else to_bf16(q, "cuda"), q_r=q_r, stream=stream)
    torch.cuda.synchronize()
    api.mla_kv_append_rope_fp8(*args, **kw)
    torch.cuda.synchronize()
    return rows, scales, q_r, int(err.item())


def _check_rows(rows, scales, c, k, pos, slots, table, good):
    tab = table.cpu().numpy().astype(np.float64)
    codes, sc = f8.quantize_rows(c)
    got = rows.cpu().numpy().reshape(-1, 640)
    gs = scales.cpu().numpy().reshape(-1)
    s = slots[good]
    assert np.array_equal(got[s, :512], codes[good]), "codes differ"
    assert np.array_equal(gs[s].astype(np.float64), np.asarray(sc)[good]), "scales differ"
    y, tol = _turn(k[good], tab[pos[good]])
    bits = got[s, 512:].copy().view(np.uint16).astype(np.uint32) << 16
    assert (np.abs(bits.view(np.float32).astype(np.float64) - y) <= tol).all()
    rest = np.ones(got.shape[0], bool)
    rest[s] = False
    assert (got[rest] == 0xA5).all() and (gs[rest] == 7.0).all(), "a row nobody asked for was written"


@pytest.mark.parametrize("n", [1, 2, 7, 64, 129, 1000])
@pytest.mark.parametrize("queries", [False, True])
def test_append_rope_fp8(api, table, n, queries):
    c, k, q, pos, pages, slots = _inputs(n, 900 + n)
    rows, scales, q_r, err = _run(api, table, c, k, q if queries else None, pos, pages, slots)
    assert err == 0
    _check_rows(rows, scales, c, k, pos, slots, table, np.ones(n, bool))
    if queries:
        y, tol = _turn(q, table.cpu().numpy().astype(np.float64)[pos][:, None])
        assert (np.abs(to_np(q_r).astype(np.float64) - y) <= tol).all()


def test_same_values_as_the_separate_calls(api, table):
    """The codes and scales of mla_kv_append_fp8, the keys of mla_kv_append_rope and the rows of mla_rope_q, bit for bit."""
    n = 200
    c, k, q, pos, pages, slots = _inputs(n, 77)
    rows, scales, q_r, err = _run(api, table, c, k, q, pos, pages, slots)
    e = torch.zeros(1, dtype=torch.int32, device="cuda")
    tc, tk, tq, tp, ts = (to_bf16(c, "cuda"), to_bf16(k, "cuda"), to_bf16(q, "cuda"), torch.from_numpy(pos).cuda(),
                          torch.from_numpy(slots).cuda())
    r2 = torch.full_like(rows, 0xA5)
    s2 = torch.full_like(scales, 7.0)
    api.mla_kv_append_fp8(tc, tk, ts, r2, s2, e)
    kv = torch.zeros((pages, 64, 576), dtype=torch.bfloat16, device="cuda")
    api.mla_kv_append_rope(tc, tk, tp, table, ts, kv, e)
    q2 = torch.empty_like(q_r)
    api.mla_rope_q(tq, tp, table, q2, e)
    assert err == 0 and api.mla_check(e) == 0
    assert torch.equal(rows[..., :512], r2[..., :512]) and torch.equal(scales, s2)
    a, b = rows.view(-1, 640)[ts, 512:].contiguous(), kv.view(-1, 576)[ts, 512:].contiguous()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert torch.equal(q_r.view(torch.int16), q2.view(torch.int16))


def test_bad_slots_and_positions_are_skipped(api, table):
    n = 70
    c, k, q, pos, pages, slots = _inputs(n, 31)
    good = np.ones(n, bool)
    slots[3], slots[40] = -1, pages * 64
    pos[9], pos[69] = -1, MAX_POS
    good[[3, 40, 9, 69]] = False
    rows, scales, q_r, err = _run(api, table, c, k, q, pos, pages, slots)
    assert err == api.DEVERR_SLOT_OOB | api.DEVERR_POS_OOB
    _check_rows(rows, scales, c, k, pos, slots, table, good)
    got = to_np(q_r)
    assert (got[[9, 69]] == 5.0).all(), "a query with a bad position was written"
    ok = np.ones(n, bool)
    ok[[9, 69]] = False
    y, tol = _turn(q[ok], table.cpu().numpy().astype(np.float64)[pos[ok]][:, None])
    assert (np.abs(got[ok].astype(np.float64) - y) <= tol).all()


def test_captured_and_replayed_on_another_stream(api, table):
    n = 130
    c, k, q, pos, pages, slots = _inputs(n, 5)
    want_rows, want_scales, want_q, _ = _run(api, table, c, k, q, pos, pages, slots)
    rows = torch.full_like(want_rows, 0xA5)
    scales = torch.full_like(want_scales, 7.0)
    q_r = torch.full_like(want_q, 5.0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (to_bf16(c, "cuda"), to_bf16(k, "cuda"), torch.from_numpy(pos).cuda(), table, torch.from_numpy(slots).cuda())
    tq = to_bf16(q, "cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.mla_kv_append_rope_fp8(*args, rows, scales, err, q_pe=tq, q_r=q_r)
    for _ in range(2):
        rows.fill_(0xA5)
        scales.fill_(7.0)
        q_r.fill_(5.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(rows, want_rows) and torch.equal(scales, want_scales) and torch.equal(q_r, want_q)
