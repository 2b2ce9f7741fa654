"""Windowed decode at large scores: how far the 16-bit scores carry.

The kernel holds a row's scores unscaled in fp16, as the sum of two rounded
halves, and forms 2^(c2 s - c2 m) with the fp16 nearest to c2 = scale log2 e and
with c2 m rounded to fp16.  With S = |score after the scale| the weight of a
token is therefore off by a factor e^(+-eps),
  eps = (|h0| + |h1| + |h0 + h1|) scale 2^-11     the halves and their sum
      + max_j S_j 2^-11                           c2 m
      + D (2^-11 + rho) + 8 ln2 2^-11             the exponent, the nearest c2
      + 2^-8 + 2^-9                               P in bf16, the hardware's 2^x
      + 288 2^-23 scale sum |q| |k|               fp32 sums of 288 products
(D the natural-log distance to the row's maximum, rho the relative error of the
nearest c2; each rounding at most half a step): about 4 S 2^-11, 14 % for a
score of 1000 before the scale.  With weights p_j e^(d_j), |d_j| <= eps_j and
x_j = e^(eps_j) - 1,
  |o' - o| <= sum_j p_j x_j (|c_j| + |o|) / (1 - sum_j p_j x_j) + 2^-8 |o|,
  |lse' - lse| <= -log(1 - sum_j p_j x_j) + M (2^-11 + rho) + 2^-22 |lse|, M = max_j S_j.
The inputs make the loss visible: every token's score is near 1000 and their
differences are of order one after the scale.
"""
import math

import numpy as np
import pytest

import oracle
from mla_latent_kv_02_gb300 import workloads as wl

from _helpers import to_bf16
from _window_ref import SCALE, bf16, seen_positions
from test_gpu_window import Cache, _decode

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
C2 = SCALE / math.log(2.0)
RHO = abs(float(np.float16(np.float32(C2))) / C2 - 1.0)


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from mla_latent_kv_02_gb300 import api as a
    a.mla_version()
    return a


def _row(q_abs, q_r, c, r):
    """(o, lse, bounds of both, largest eps of a weight that counts) of one row in 64 bits."""
    h = [q_abs[:, 256 * i:256 * i + 256] @ c[:, 256 * i:256 * i + 256].T +
         q_r[:, 32 * i:32 * i + 32] @ r[:, 32 * i:32 * i + 32].T for i in range(2)]
    mass = q_abs.abs() @ c.abs().T + q_r.abs() @ r.abs().T
    raw = h[0] + h[1]
    s = raw * SCALE
    m = s.amax(dim=-1, keepdim=True)
    e = torch.exp(s - m)
    p, lse = e / e.sum(dim=-1, keepdim=True), (m + torch.log(e.sum(dim=-1, keepdim=True))).squeeze(-1)
    top = s.abs().amax(dim=-1, keepdim=True)
    eps = ((h[0].abs() + h[1].abs() + raw.abs()) * SCALE + top + 8 * math.log(2.0)) * 2.0 ** -11 + \
        (m - s) * (2.0 ** -11 + RHO) + 2.0 ** -8 + 2.0 ** -9 + mass * SCALE * 288 * 2.0 ** -23
    x = torch.expm1(eps)
    px = (p * x).sum(dim=-1, keepdim=True)
    assert bool((px < 0.5).all()), "the bound says nothing here"
    o = p @ c
    tol = ((p * x) @ c.abs() + px * o.abs()) / (1 - px) + 2.0 ** -8 * o.abs()
    tol_l = (-torch.log1p(-px) + top * (2.0 ** -11 + RHO)).squeeze(-1) + 2.0 ** -22 * lse.abs()
    return o, lse, 1.05 * tol + 1e-6, 1.05 * tol_l + 1e-6, p, raw


def _fill(api, cache, u):
    """The cache's latents become u + 0.35 of what they were."""
    rng = np.random.default_rng(5)
    for b, n in enumerate(cache.n):
        cache.c[b] = wl.bf16_round(u[None] + np.float32(0.35) * rng.standard_normal((n, 512), dtype=np.float32))
    seq = np.repeat(np.arange(len(cache.n), dtype=np.int32), cache.n)
    pos = np.concatenate([np.arange(n, dtype=np.int32) for n in cache.n])
    slots = torch.from_numpy(api.mla_slot_mapping(cache.bt, seq, pos)).cuda()
    c, r = to_bf16(np.concatenate(cache.c), "cuda"), to_bf16(np.concatenate(cache.r), "cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    if cache.kind == "bf16":
        api.mla_kv_append(c, r, slots, cache.kv, err)
    else:
        api.mla_kv_append_fp8(c, r, slots, cache.rows, cache.scales, err)
        for b in range(len(cache.n)):
            codes, sc = oracle.fp8_cache.quantize_rows(cache.c[b])
            cache.c[b] = oracle.fp8_cache.dequantize_rows(codes, sc)
    assert api.mla_check(err) == 0


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_scores_near_1000_before_the_scale(api, kind, sign):
    seq, q, window, sinks = [900, 1300], [1, 2], 500, 4
    cache = Cache(api, seq, kind, 33)
    rng = np.random.default_rng(34)
    u = np.where(rng.random(512) < 0.5, -1.0, 1.0).astype(np.float32)
    _fill(api, cache, u)
    T = sum(q)
    a = rng.uniform(1.6, 2.3, (T, 128, 1)).astype(np.float32) * np.float32(sign)
    q_abs = to_bf16(wl.bf16_round(a * u[None, None]), "cuda")
    q_r = to_bf16(bf16(rng, (T, 128, 64)), "cuda")
    plan = api.mla_window_plan(seq, q, window, sinks, num_clusters=4)
    o, lse, err = _decode(api, cache, q_abs, q_r, plan)
    assert api.mla_check(err) == 0
    t = 0
    for b, m in enumerate(q):
        for i in range(m):
            c, r = cache.tokens(b, seen_positions(cache.n[b] - m + i, window, sinks))
            wo, wlse, to, tl, p, raw = _row(q_abs[t].double(), q_r[t].double(), c, r)
            assert 700 < float(raw.abs().min()) and float(raw.abs().max()) < 1400
            assert float(p.max(dim=-1).values.median()) < 0.5, "one token takes it all: the loss would not show"
            d, dl = (o[t].double() - wo).abs(), (lse[t].double() - wlse).abs()
            assert bool((d <= to).all()), (t, float((d / to).max()))
            assert bool((dl <= tl).all()), (t, "lse", float((dl / tl).max()))
            t += 1
