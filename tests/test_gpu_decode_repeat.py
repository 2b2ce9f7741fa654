"""Many rows a cluster, passes by the hundred: the decode's rows leave through the buffers that
the next scores cross in, and every pass has to give the same bits, right ones."""
import numpy as np
import pytest

from _helpers import to_bf16
from _window_ref import bf16, decode_row, seen_positions

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from mla_latent_kv_02_gb300 import api as a
    a.mla_version()
    return a


# sequences' lengths, query rows of each, clusters (None: all); rows of two to seven tiles, whole and cut
CASES = [
    ([190, 256, 320, 130] * 12, [2] * 48, 2),
    ([200 + 11 * b for b in range(20)], [1 + b % 4 for b in range(20)], 3),
    ([400] * 152, [4] * 152, None),
    ([8194] * 8, [2] * 8, None),
]


@pytest.mark.parametrize("window", [None, (200, 4)])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_every_pass_gives_the_same_bits(api, case, window):
    n, q, clusters = CASES[case]
    rng = np.random.default_rng(case)
    T, pages = sum(q), [(x + 63) // 64 for x in n]
    table = np.zeros((len(n), max(pages)), np.int32)
    perm = rng.permutation(sum(pages)).astype(np.int32)
    for b, k in enumerate(pages):
        table[b, :k] = perm[sum(pages[:b]):sum(pages[:b]) + k]
    kv = to_bf16(bf16(rng, (sum(pages), 64, 576)), "cuda")
    q_abs, q_r = to_bf16(bf16(rng, (T, 128, 512), 0.5), "cuda"), to_bf16(bf16(rng, (T, 128, 64)), "cuda")
    bt, err = torch.from_numpy(table).cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    if window is None:
        plan, call = api.mla_decode_plan(n, q, num_clusters=clusters), api.mla_decode_paged
    else:
        plan, call = api.mla_window_plan(n, q, *window, num_clusters=clusters), api.mla_decode_window
    o, lse = (torch.full((T, 128, d), float("nan"), dtype=t, device="cuda") for d, t in ((512, torch.bfloat16), (1, torch.float32)))
    lse = lse[..., 0].contiguous()
    call(q_abs, q_r, kv, bt, plan, o, err, lse=lse)
    assert api.mla_check(err) == 0
    row = 0
    for b in range(len(n)):
        for i in range(q[b]):
            if row % max(1, T // 24) == 0 or row == T - 1:
                p = n[b] - q[b] + i
                at = torch.tensor(seen_positions(p, *window) if window else list(range(p + 1)), device="cuda")
                x = kv[bt[b].long()[at // 64], at % 64].double()
                wo, wl, to, tl = decode_row(q_abs[row].double(), q_r[row].double(), x[:, :512], x[:, 512:])
                assert bool(((o[row].double() - wo).abs() <= to).all()), row
                assert bool(((lse[row].double() - wl).abs() <= tl).all()), (row, "lse")
            row += 1
    want, want_lse = o.clone(), lse.clone()
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(400):
        o.fill_(float("nan"))
        call(q_abs, q_r, kv, bt, plan, o, err, lse=lse)
        wrong += (o.view(torch.int16) != want.view(torch.int16)).any() | (lse != want_lse).any()
    assert int(err.item()) == 0 and int(wrong.item()) == 0
