"""The draft-tree calls judge what they take a size from before they take it (no GPU)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def api(monkeypatch):
    from mla_latent_kv_02_gb300 import api as a
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return a


I32 = torch.zeros(4, dtype=torch.int32)
MASKS = torch.zeros((4, 1), dtype=torch.int64)
KV = torch.zeros((1, 64, 576), dtype=torch.bfloat16)


@pytest.mark.parametrize("bad, error", [([0] * 4, TypeError), (np.zeros(4, np.int32), TypeError), (None, TypeError),
                                        (torch.tensor(0, dtype=torch.int32), ValueError)])
def test_sizes_are_taken_from_tensors(api, monkeypatch, bad, error):
    for args in ((bad, I32, I32, MASKS, I32), (I32, I32, bad, MASKS, I32)):
        with pytest.raises(error):
            api.mla_tree_layout(*args)
    monkeypatch.setattr(api, "_layers", lambda *a: (0, 1, 1, 0))
    for name, cache in (("mla_tree_compact", (KV,)), ("mla_tree_compact_nvfp4", (KV,))):
        for args in ((I32, bad, I32, I32, I32, I32, I32), (I32, MASKS, I32, bad, I32, I32, I32)):
            with pytest.raises(error):
                getattr(api, name)(*cache, *args)
    with pytest.raises(error):
        api.mla_decode_tree(I32, I32, bad, I32, MASKS, None, I32, I32)
    with pytest.raises(error):
        api.mla_decode_tree_fp8(I32, I32, bad, I32, I32, MASKS, None, I32, I32)
