"""Host side of the draft-tree operators: plans, shared pages, forks, moves, refusals (no GPU)."""
import ctypes as C

import numpy as np
import pytest

from mla_latent_kv_02_gb300 import _build, _lib


@pytest.fixture(scope="module")
def api():
    if _build.is_stale():
        _build.build()
    from mla_latent_kv_02_gb300 import api as a
    a.mla_version()
    return a


def _segments(plan):
    nc, ns = int(plan[3]), int(plan[4])
    off = [int(x) for x in plan[16:16 + nc + 1]]
    base = (16 + nc + 1 + 7) // 8 * 8
    return off, [[int(x) for x in plan[base + 8 * i:base + 8 * i + 8]] for i in range(ns)]


@pytest.mark.parametrize("clusters", [1, 3, 76])
@pytest.mark.parametrize("seq, q", [([1], [1]), ([5], [5]), ([64, 65, 129], [1, 2, 1]), ([300], [256]), ([70, 900], [0, 70]),
                                    ([5000] * 4, [40] * 4), ([200] * 3, [130] * 3), ([8] * 5, [0] * 5),
                                    ([2 ** 31 - 1], [2]), ([4096] * 64, [12] * 64), ([1000] * 2, [77] * 2)])
def test_tree_plan_covers_what_each_node_may_see(api, seq, q, clusters):
    plan, info = api.mla_tree_plan_host(seq, q, clusters)
    assert int(plan[0]) == info.plan.magic == 0x544C4D41 and info.max_nodes == max(q)
    rows = [(b, n - m, n - m + i + 1) for b, (n, m) in enumerate(zip(seq, q)) for i in range(m)]
    assert info.plan.T == len(rows) and info.plan.num_clusters <= clusters
    off, segs = _segments(plan)
    assert off[0] == 0 and off[-1] == len(segs) and all(a <= b for a, b in zip(off, off[1:]))
    tiles = {t: [] for t in range(len(rows))}
    base = [sum((n + 63) // 64 for n, m in list(zip(seq, q))[:b] if m) for b in range(len(seq))]
    for row, b, pb, pe, vis, slot, first, page in segs:
        assert rows[row] == (b, first, vis) and 0 <= pb < pe and page == base[b] and -1 <= slot < info.plan.num_partials
        tiles[row].append((pb, pe, slot))
    for t, (b, first, vis) in enumerate(rows):
        at = 0
        for pb, pe, slot in sorted(tiles[t]):
            assert pb == at and (slot < 0) == (len(tiles[t]) == 1)
            at = pe
        assert at == (vis - 1) // 64 + 1
    table = plan[(16 + info.plan.num_clusters + 1 + 7) // 8 * 8 + 8 * len(segs) + 4 * info.plan.num_split_rows:]
    trees = [[int(x) for x in table[8 * k:8 * k + 7]] for k in range(info.num_trees)]
    held = [b for b, m in enumerate(q) if m]
    assert trees == [[b, base[b], (seq[b] + 63) // 64, seq[b] - q[b], seq[b], sum(q[:b]), q[b]] for b in held]
    assert info.total_pages == sum((seq[b] + 63) // 64 for b in held)
    words = (16 + info.plan.num_clusters + 1 + 7) // 8 * 8 + 8 * len(segs) + 4 * info.plan.num_split_rows + 8 * len(held)
    assert info.plan.plan_bytes == 4 * words <= api.mla_tree_plan_bytes(len(rows), clusters)
    assert info.plan.total_tiles == sum((vis - 1) // 64 + 1 for _, _, vis in rows)


def test_tree_plan_refusals(api):
    for seq, q, status in (([300], [257], 3), ([5], [6], 1), ([0], [0], 1), ([5], [-1], 1)):
        with pytest.raises(api.MlaError) as e:
            api.mla_tree_plan_host(seq, q, 4)
        assert e.value.status == status
    with pytest.raises(api.MlaError):
        api.mla_tree_plan_host([5], [1], 0)
    with pytest.raises(ValueError):
        api.mla_tree_plan_host([2 ** 31], [1], 4)
    with pytest.raises(ValueError):
        api.mla_tree_plan_host([5, 5], [1], 4)


def _lib_call(name, *args):
    return getattr(_lib.lib(), name)(*args)


def test_decode_tree_refusals(api):
    """Everything is judged before a launch: no GPU is touched."""
    ok, odd = C.c_void_p(1 << 20), C.c_void_p((1 << 20) + 4)
    _, info = api.mla_tree_plan_host([200, 2000], [70, 3], 40)
    assert info.plan.num_partials > 0
    _, full = api.mla_decode_plan_host([200], [70], 4)
    ws = 1 << 28

    def call(masks=ok, words=2, info=info, scale=0.07, q=ok, cols=40, pages=9, w=ok, wb=ws, o=ok, err=ok, table=ok):
        return _lib_call("mla_decode_tree", q, ok, ok, pages, table, cols, masks, words, ok, C.byref(info), C.c_float(scale), w,
                         wb, o, None, err, None)

    assert call(words=1) == 1                               # 70 nodes need two words
    assert call(words=0) == 1 and call(words=5) == 1
    assert call(masks=None) == 1 and call(masks=odd) == 2
    assert call(scale=0.0) == 1 and call(q=None) == 1 and call(q=odd) == 2 and call(cols=31) == 1
    assert call(pages=0) == 1 and call(w=None) == 1 and call(wb=16) == 1 and call(o=None) == 1 and call(err=None) == 1
    wrong = _lib.mla_tree_info()
    wrong.plan = full
    wrong.max_nodes = 70
    assert call(info=wrong) == 1                            # another kind's plan
    assert _lib_call("mla_decode_paged", ok, ok, ok, 9, ok, 4, ok, C.byref(info.plan), C.c_float(0.07), ok, ws, ok, None, ok,
                     None) == 1
    _, none = api.mla_tree_plan_host([200], [0], 4)
    assert call(info=none, masks=None, q=None) == 0         # no rows
    assert _lib_call("mla_decode_tree_fp8", ok, ok, ok, None, 9, ok, 4, ok, 2, ok, C.byref(info), C.c_float(0.07), ok, ws, ok,
                     None, ok, None) == 1


def test_layout_and_compact_refusals(api):
    ok, odd = C.c_void_p(1 << 20), C.c_void_p((1 << 20) + 2)
    far = C.c_void_p(1 << 21)

    def layout(par=ok, B=2, T=5, words=1, table=ok, cols=3, pages=4, masks=ok, pos=ok, slots=ok, err=ok):
        return _lib_call("mla_tree_layout", par, ok, ok, B, T, words, table, cols, pages, masks, pos, slots, err, None)

    assert layout(par=None) == 1 and layout(words=0) == 1 and layout(words=5) == 1 and layout(B=-1) == 1 and layout(T=-1) == 1
    assert layout(table=None) == 1 and layout(cols=0) == 1 and layout(pages=0) == 1 and layout(err=None) == 1
    assert layout(masks=C.c_void_p((1 << 20) + 4)) == 2 and layout(par=odd) == 2 and layout(pos=odd) == 2
    assert layout(T=0) == 0 and layout(B=0) == 0

    def compact(kv=ok, pages=4, layers=2, stride=4 * 73728, table=ok, cols=3, masks=ok, words=1, q=ok, seq=ok, acc=ok, B=2, T=5,
                lens=far, err=ok):
        return _lib_call("mla_tree_compact", kv, pages, layers, stride, table, cols, masks, words, q, seq, acc, B, T, lens, err,
                         None)

    assert compact(kv=None) == 1 and compact(layers=0) == 1 and compact(stride=73728) == 1 and compact(stride=4 * 73728 + 8) == 2
    assert compact(pages=0) == 1 and compact(table=None) == 1 and compact(cols=0) == 1 and compact(words=9) == 1
    assert compact(lens=ok) == 1                            # the lengths would be read and written
    assert compact(lens=C.c_void_p((1 << 20) + 4)) == 1
    base = 1 << 24                                          # nor may they lie anywhere in the masks, the table or the word
    for at, kw in ((39, dict(masks=C.c_void_p(base), T=5)), (23, dict(table=C.c_void_p(base))), (3, dict(err=C.c_void_p(base)))):
        assert compact(lens=C.c_void_p(base + at // 4 * 4), **kw) == 1, kw
    assert compact(acc=None) == 1 and compact(masks=None) == 1 and compact(masks=odd) == 2 and compact(lens=odd) == 2
    assert compact(B=0) == 0
    assert _lib_call("mla_tree_compact_fp8", ok, None, 4, 1, 0, 0, ok, 3, ok, 1, ok, ok, ok, 2, 5, far, ok, None) == 1
    assert _lib_call("mla_tree_compact_fp8", ok, odd, 4, 1, 0, 0, ok, 3, ok, 1, ok, ok, ok, 2, 5, far, ok, None) == 2


def _i32(*v):
    return (C.c_int32 * len(v))(*v)


def test_copy_pages_refusals(api):
    ok = C.c_void_p(1 << 20)

    def copy(src, dst, n=None, kv=ok, pages=8, layers=2, stride=8 * 73728):
        return _lib_call("mla_copy_pages", kv, pages, layers, stride, src, dst, len(src) if n is None else n, None)

    assert copy(_i32(0, 1), _i32(2, 2)) == 1                # written twice
    assert copy(_i32(0, 1), _i32(1, 2)) == 1                # read and written
    assert copy(_i32(3), _i32(3)) == 1
    many = 1 << 21                                          # a pool of which few pages are named
    for src, dst in ((_i32(0, many - 1), _i32(2, 2)), (_i32(0, 1), _i32(1, 2)), (_i32(many), _i32(0)), (_i32(0), _i32(many))):
        assert copy(src, dst, pages=many, layers=1) == 1
    assert copy(_i32(8), _i32(0)) == 1 and copy(_i32(0), _i32(8)) == 1 and copy(_i32(-1), _i32(0)) == 1
    assert copy(_i32(0), _i32(1), kv=None) == 1 and copy(_i32(0), _i32(1), kv=C.c_void_p((1 << 20) + 8)) == 2
    assert copy(_i32(0), _i32(1), layers=0) == 1 and copy(_i32(0), _i32(1), stride=73728) == 1
    assert copy(_i32(0), _i32(1), stride=8 * 73728 + 4) == 2 and copy(_i32(0), _i32(1), n=-1) == 1
    assert copy(_i32(0), _i32(1), stride=2 ** 63 - 16) == 1
    assert copy(_i32(0), _i32(1), n=0, kv=None) == 0
    assert _lib_call("mla_copy_pages", ok, 8, 1, 0, None, _i32(1), 1, None) == 1


def test_pool_holders(api):
    pool = api.MlaPool(4)
    a, b = (int(x) for x in pool.alloc(2))
    pool.retain([a, a])
    assert [pool.refs(x) for x in range(4)] == [3, 1, 0, 0]
    pool.free([a, b])
    assert pool.refs(a) == 2 and pool.refs(b) == 0 and pool.available() == 3
    for bad in ([b], [4], [-1], [a, b]):
        with pytest.raises(api.MlaError):
            pool.retain(bad)
        with pytest.raises(api.MlaError):
            pool.free(bad)
    assert pool.refs(a) == 2
    with pytest.raises(api.MlaError):
        pool.free([a, a])                                   # one hold at a time
    pool.free([a])
    pool.free([a])
    assert pool.available() == 4 and pool.refs(a) == 0
    with pytest.raises(api.MlaError):
        pool.refs(4)
    with pytest.raises(ValueError):
        pool.retain([0.5])


@pytest.mark.parametrize("n_tokens", [0, 1, 63, 64, 65, 128, 150])
@pytest.mark.parametrize("children", [0, 1, 3])
def test_pool_fork(api, n_tokens, children):
    pool = api.MlaPool(20)
    parent = np.concatenate([pool.alloc(3), [-1]]).astype(np.int32)
    rows, src, dst = pool.fork(parent, n_tokens, children, max_pages=5)
    full, part = n_tokens // 64, n_tokens % 64 != 0
    assert rows.shape == (children, 5) and len(src) == len(dst) == (children if part else 0)
    for i in range(children):
        assert list(rows[i, :full]) == list(parent[:full])
        if part:
            assert rows[i, full] == dst[i] and src[i] == parent[full]
        assert (rows[i, full + part:] == -1).all()
    assert len(set(dst.tolist()) | set(parent[:3].tolist())) == len(dst) + 3
    for k in range(3):
        assert pool.refs(int(parent[k])) == (1 + children if k < full else 1)
    assert pool.available() == 17 - len(dst)
    for i in range(children):                               # everything comes back
        held = rows[i][rows[i] >= 0]
        pool.free(held)
    pool.free(parent[:3])
    assert pool.available() == 20


def test_pool_fork_refusals(api):
    pool = api.MlaPool(3)
    parent = pool.alloc(2)
    with pytest.raises(api.MlaError) as e:
        pool.fork(parent, 100, 2)                           # two fresh pages, one free
    assert e.value.status == 7 and pool.available() == 1 and [pool.refs(x) for x in range(3)] == [1, 1, 0]
    with pytest.raises(api.MlaError):
        pool.fork([0, 0], 128, 1)
    with pytest.raises(api.MlaError):
        pool.fork([0, 2], 128, 1)
    with pytest.raises(api.MlaError):
        pool.fork(parent, 128, 1, max_pages=1)
    for n in (-1, 129):
        with pytest.raises(ValueError):
            pool.fork(parent, n, 1)
    with pytest.raises(ValueError):
        pool.fork(parent, 128, -1)
    assert pool.available() == 1


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("most", [0, 1, 4, 1000])
def test_pool_compact(api, seed, most):
    rng = np.random.default_rng(seed)
    n = int(rng.integers(1, 60))
    pool = api.MlaPool(n)
    ids = pool.alloc(n)
    drop = rng.permutation(n)[:int(rng.integers(0, n + 1))].astype(np.int32)
    pool.free(drop)
    held = np.array([i for i in ids if i not in set(drop.tolist())], dtype=np.int32)
    for i in held:
        pool.retain([i] * int(rng.integers(0, 3)))
    before = [pool.refs(i) for i in range(n)]
    table = np.full((2, n + 1), -1, np.int32)
    table[0, :held.size] = rng.permutation(held)
    table[1, :held.size // 2] = rng.permutation(held)[:held.size // 2]
    src, dst = pool.compact(most)
    assert len(src) == len(dst) <= most and not set(src.tolist()) & set(dst.tolist())
    moved = dict(zip(src.tolist(), dst.tolist()))
    assert len(moved) == len(src) and all(d < s for s, d in moved.items())
    after = [pool.refs(i) for i in range(n)]
    assert after == [before[[s for s, d in moved.items() if d == i][0]] if i in moved.values() else
                     0 if i in moved else before[i] for i in range(n)]
    if most == 1000:
        assert all(after[:held.size]) and not any(after[held.size:])
    new = api.mla_remap_pages(table, src, dst)
    assert (new == np.vectorize(lambda x: moved.get(int(x), int(x)))(table)).all()
    assert pool.available() == n - held.size


def test_remap_refusals(api):
    t = np.array([[1, 2, -1]], np.int32)
    assert (api.mla_remap_pages(t, [], []) == t).all()
    for src, dst in (([1, 1], [3, 4]), ([-1], [2]), ([1], [-2])):
        with pytest.raises(api.MlaError):
            api.mla_remap_pages(t, src, dst)
    with pytest.raises(ValueError):
        api.mla_remap_pages(t, [1, 2], [3])
    assert (t == np.array([[1, 2, -1]])).all()
