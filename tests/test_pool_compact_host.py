"""MlaPool.compact: what a call takes goes by the pool, not by the most moves that it may make (no GPU)."""
import tracemalloc

import pytest

from mla_latent_kv_02_gb300 import _build


@pytest.fixture(scope="module")
def api():
    if _build.is_stale():
        _build.build()
    from mla_latent_kv_02_gb300 import api as a
    return a


@pytest.mark.parametrize("pages", [1, 2, 3, 8, 9])
def test_any_number_of_moves(api, pages):
    pool = api.MlaPool(pages)
    pool.alloc(pages)
    pool.free(range(0, pages // 2))                          # as many free pages below as held ones above
    tracemalloc.start()
    src, dst = pool.compact(2 ** 31 - 1)
    peak = tracemalloc.get_traced_memory()[1]
    tracemalloc.stop()
    assert peak < 1 << 20
    assert dst.tolist() == list(range(pages // 2)) and src.tolist() == list(range(pages - 1, pages - 1 - pages // 2, -1))
    held = pages - pages // 2
    assert [pool.refs(i) for i in range(pages)] == [1] * held + [0] * (pages - held)
