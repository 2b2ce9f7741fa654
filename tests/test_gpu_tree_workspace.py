"""The workspace that a tree plan takes for its decodes over an FP8 cache, and a plan that declines it."""
import pytest

from _tree_ref import masks, tree
from test_gpu_tree import Cache, decode, queries

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from mla_latent_kv_02_gb300 import api as a
    a.mla_version()
    return a


def test_a_plan_declines_the_larger_workspace(api):
    n0, q = 36000, 40                                        # 563 pages, 41 MB unpacked
    cache = Cache(api, [n0 + q], "fp8", 3)
    m = torch.from_numpy(masks([tree(0, q)], 1)).cuda()
    q_abs, q_r = queries(q, 3)
    lean, plan = api.mla_tree_plan(cache.n, [q], unpack=False), api.mla_tree_plan(cache.n, [q])
    need = api.mla_tree_workspace_size(plan.info, True)
    held = lean.workspace.numel()
    assert held < need
    o, lse, err = decode(api, cache, q_abs, q_r, m, lean)
    assert api.mla_check(err) == 0 and lean.workspace.numel() == held
    o2, lse2, err2 = decode(api, cache, q_abs, q_r, m, plan)
    assert api.mla_check(err2) == 0 and plan.workspace.numel() >= need
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    again = api.mla_tree_plan(cache.n, [q], into=lean)       # the next step may take it
    o3, _, err3 = decode(api, cache, q_abs, q_r, m, again)
    assert api.mla_check(err3) == 0 and again.workspace.numel() >= need and torch.equal(o, o3)
    kept = api.mla_tree_plan(cache.n, [q], into=again, unpack=False)
    o4, _, err4 = decode(api, cache, q_abs, q_r, m, kept)    # what is there already stays and serves
    assert api.mla_check(err4) == 0 and kept.workspace.data_ptr() == again.workspace.data_ptr() and torch.equal(o, o4)
