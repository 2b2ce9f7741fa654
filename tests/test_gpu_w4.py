"""The per-head projections with 4-bit weights, and their packing, against 64 bits.

Codes are integers and every group's scale multiplies an fp32 sum, so against
the 64-bit product of the same codes and scales a result is off by half a bf16
step (2^-8 relative) and by the roundings of at most K + 8 fp32 additions and
scalings, each at most 2^-23 of sum |x| |W| (the tensor core may truncate).
"""
import numpy as np
import pytest

from mla_latent_kv_02_gb300 import workloads as wl

from _helpers import to_bf16
from _window_ref import bf16

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
SHAPES = {"absorb": (128, 512), "up": (512, 128)}


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from mla_latent_kv_02_gb300 import api as a
    a.mla_version()
    return a


def _unpack(words):
    """int codes [128, K, N] of words [128, K/8, N]."""
    w = words.to(torch.int64) & 0xFFFFFFFF
    nib = torch.stack([(w >> (4 * i)) & 15 for i in range(8)], dim=2)
    return torch.where(nib > 7, nib - 16, nib).reshape(128, -1, words.shape[2])


def _random_weights(K, N, group, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    words = torch.randint(-2 ** 31, 2 ** 31, (128, K // 8, N), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    scales = (torch.randn((128, K // group, N), generator=g, device="cuda") * 0.02).to(torch.bfloat16)
    scales[3, 0, ::7] = 0.0
    return words, scales


def _call(api, kind, x, words, scales, out, err, **kw):
    (api.mla_absorb_q_w4 if kind == "absorb" else api.mla_up_v_w4)(x, words, scales, out, err, **kw)


def _check(x, words, scales, out):
    K = words.shape[1] * 8
    w = _unpack(words).double() * scales.double().repeat_interleave(K // scales.shape[1], dim=1)
    for t0 in range(0, x.shape[0], 256):
        xt = x[t0:t0 + 256].double().transpose(0, 1)
        want = torch.matmul(xt, w).transpose(0, 1)
        mass = torch.matmul(xt.abs(), w.abs()).transpose(0, 1)
        tol = want.abs() * 2.0 ** -8 + mass * (K + 8) * 2.0 ** -23
        d = (out[t0:t0 + 256].double() - want).abs()
        assert bool((d <= tol).all()), (t0, float((d / tol.clamp(min=1e-300)).max()))


@pytest.mark.parametrize("T", [1, 2, 3, 5, 8, 9, 16, 17, 100, 127, 128, 129, 300])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("kind", ["absorb", "up"])
def test_w4(api, kind, group, T):
    K, N = SHAPES[kind]
    words, scales = _random_weights(K, N, group, 10 * T + group)
    x = to_bf16(bf16(np.random.default_rng(T), (T, 128, K)), "cuda")
    guard = torch.full((T + 2, 128, N), 3.0, dtype=torch.bfloat16, device="cuda")
    out = guard[1:T + 1]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    _call(api, kind, x, words, scales, out, err)
    assert api.mla_check(err) == 0
    _check(x, words, scales, out)
    assert bool((guard[0] == 3.0).all()) and bool((guard[-1] == 3.0).all()), "a row past T was written"


@pytest.mark.parametrize("kind,group,T", [("absorb", 64, 1100), ("up", 128, 2049), ("up", 64, 700), ("absorb", 128, 1025),
                                          ("up", 32, 513), ("absorb", 32, 640)])
def test_w4_many_tokens(api, kind, group, T):
    K, N = SHAPES[kind]
    words, scales = _random_weights(K, N, group, T)
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    x = torch.randn((T, 128, K), generator=g, device="cuda").to(torch.bfloat16)
    out = torch.empty((T, 128, N), dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    _call(api, kind, x, words, scales, out, err)
    assert api.mla_check(err) == 0
    _check(x, words, scales, out)


def test_w4_infinities_and_nan_stay_in_their_rows(api):
    words, scales = _random_weights(128, 512, 64, 4)
    for T in (6, 40):
        x = to_bf16(bf16(np.random.default_rng(5), (T, 128, 128)), "cuda")
        clean = torch.empty((T, 128, 512), dtype=torch.bfloat16, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        api.mla_absorb_q_w4(x, words, scales, clean, err)
        x[2, 7, 5] = float("inf")
        x[4, 9, 5] = float("nan")
        out = torch.empty_like(clean)
        api.mla_absorb_q_w4(x, words, scales, out, err)
        assert api.mla_check(err) == 0
        hit = torch.zeros((T, 128), dtype=torch.bool, device="cuda")
        hit[2, 7] = hit[4, 9] = True
        assert torch.equal(out[~hit], clean[~hit])
        assert bool(torch.isnan(out[4, 9]).all()) and not bool(torch.isfinite(out[2, 7]).any())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("kind", ["absorb", "up"])
def test_pack_w4(api, kind, group):
    """Scales and codes bit for bit: fp32 divisions rounded to nearest, as numpy's."""
    K, N = SHAPES[kind]
    rng = np.random.default_rng(group)
    w = bf16(rng, (128, K, N), 0.044)
    w[0, :group, 0] = 0.0                                    # a zero group
    w[1, :group, 1] = wl.bf16_round(np.full(group, 1e-39, np.float32))   # subnormal weights
    w[2, 0, 2] = 1e30
    words, scales = api.mla_pack_w4(to_bf16(w, "cuda"), group)
    torch.cuda.synchronize()
    wg = w.reshape(128, K // group, group, N)
    s = wl.bf16_round(np.abs(wg).max(axis=2) / np.float32(7.0))
    assert np.array_equal(scales.float().cpu().numpy(), s)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(s[:, :, None] > 0, np.clip(np.rint(wg / s[:, :, None]), -8, 7), 0).reshape(128, K, N)
    assert np.array_equal(_unpack(words).cpu().numpy(), q.astype(np.int64))


def test_packed_weights_serve_the_projection(api):
    """From bf16 weights to a projection: the result of the quantised weights, near that of the weights themselves."""
    rng = np.random.default_rng(3)
    w = to_bf16(bf16(rng, (128, 512, 128), 0.044), "cuda")
    words, scales = api.mla_pack_w4(w, 64)
    x = to_bf16(bf16(rng, (33, 128, 512)), "cuda")
    out, full = (torch.empty((33, 128, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.mla_up_v_w4(x, words, scales, out, err)
    api.mla_up_v(x, w, full, err)
    assert api.mla_check(err) == 0
    _check(x, words, scales, out)
    # a code is off by at most half a scale: relative error under (max / 7 / 2 / sqrt 3) / std, max about 2.4 std of 64
    rel = float((out.double() - full.double()).norm() / full.double().norm())
    assert rel < 0.15


def test_w4_captured_and_on_a_stream(api):
    words, scales = _random_weights(512, 128, 128, 8)
    for T in (4, 150):
        x = to_bf16(bf16(np.random.default_rng(9), (T, 128, 512)), "cuda")
        want, out = (torch.zeros((T, 128, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        api.mla_up_v_w4(x, words, scales, want, err)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        api.mla_up_v_w4(x, words, scales, out, err, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            api.mla_up_v_w4(x, words, scales, out, err)
        x2 = x.flip(0).contiguous()
        x.copy_(x2)
        g.replay()
        assert api.mla_check(err) == 0 and torch.equal(out, want.flip(0))


def test_w4_refusals(api):
    words, scales = _random_weights(128, 512, 64, 1)
    x = torch.zeros((2, 128, 128), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros((2, 128, 512), dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        api.mla_absorb_q_w4(x, words[:, :8], scales, out, err)
    with pytest.raises(ValueError):
        api.mla_absorb_q_w4(x, words, scales[:, :, ::2], out, err)
    with pytest.raises(TypeError):
        api.mla_absorb_q_w4(x, words, scales.float(), out, err)
    with pytest.raises(ValueError):
        api.mla_up_v_w4(x, words, scales, out, err)
    with pytest.raises(api.MlaError) as e:
        api.mla_absorb_q_w4(x, words, torch.zeros((128, 8, 512), dtype=torch.bfloat16, device="cuda"), out, err)
    assert e.value.status == 3                              # groups of 16
    with pytest.raises(api.MlaError) as e:
        api.mla_pack_w4(torch.zeros((128, 128, 512), dtype=torch.bfloat16, device="cuda"), 16)
    assert e.value.status == 3
    with pytest.raises(api.MlaError):
        api.mla_pack_w4(torch.zeros((128, 128, 128), dtype=torch.bfloat16, device="cuda"), 64)
    buf = torch.zeros((2, 128, 512), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(api.MlaError) as e:                  # the output over the input
        api.mla_absorb_q_w4(buf.view(-1)[:2 * 128 * 128].view(2, 128, 128), words, scales, buf, err)
    assert e.value.status == 1
    api.mla_absorb_q_w4(x[:0], words, scales, out[:0], err)
    assert api.mla_check(err) == 0
