"""Host side of the windowed operators: the plan's tiles against brute force, and refusals (no GPU)."""
import ctypes as C

import numpy as np
import pytest

from mla_latent_kv_02_gb300 import _build, _lib

from _window_ref import seen_positions


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


def _tile_tokens(v, lo, vis, sinks):
    """Tile v of a row as the kernel reads it: (tokens it loads, tokens the row sees), positions by place."""
    first, full, rest = lo // 64, sinks // 64, sinks % 64
    split = (rest + 7) // 8 * 8
    shared = lo > 0 and rest > 0 and first == full
    merged = lo > 0 and rest > 0 and not shared and split <= lo % 64
    if lo == 0:
        sink_tiles = skip = head = 0
    else:
        sink_tiles = full + (1 if rest > 0 and not shared and not merged else 0)
        skip = first - sink_tiles
        head = rest if shared or merged else 0
    if v < sink_tiles:
        return [v * 64 + j for j in range(64)], [v * 64 + j for j in range(64) if v * 64 + j < sinks]
    page = v + skip
    load = [page * 64 + j for j in range(64)]
    if merged and v == sink_tiles:
        load[:split] = [full * 64 + j for j in range(split)]
    seen = [load[j] for j in range(64)
            if (v == sink_tiles and j < head) or (j >= lo - page * 64 and j < vis - page * 64)]
    return load, seen


CASES = [([1], [1], 1, 0), ([200], [3], 100, 4), ([64, 65, 129], [1, 2, 1], 64, 64), ([1000], [2], 130, 70),
         ([4096], [1], 512, 63), ([70], [1], 1, 69), ([70], [1], 1, 68), ([257], [5], 3, 8), ([640], [1], 65, 128),
         (list(range(150, 215)), [1] * 65, 80, 4), (list(range(150, 215)), [2] * 65, 20, 75), ([500] * 8, [0] * 8, 5, 5),
         ([2 ** 31 - 1], [1], 130, 4), ([3000, 10], [4, 10], 2 ** 31 - 1, 2 ** 31 - 1)]


@pytest.mark.parametrize("clusters", [1, 3, 76])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_window_plan_covers_what_each_row_sees(api, case, clusters):
    seq, q, window, sinks = CASES[case]
    plan, info = api.mla_window_plan_host(seq, q, window, sinks, clusters)
    assert info.window == window and info.sinks == sinks and int(plan[0]) == info.plan.magic == 0x574C4D41
    rows = [(b, n - m + i) for b, (n, m) in enumerate(zip(seq, q)) for i in range(m)]
    assert info.plan.T == len(rows)
    off, segs = _segments(plan)
    assert off[0] == 0 and off[-1] == len(segs) and all(a <= b for a, b in zip(off, off[1:]))
    seen = {t: [] for t in range(len(rows))}
    pieces = {t: [] for t in range(len(rows))}
    tiles = 0
    for row, b, pb, pe, vis, slot, lo, zero in segs:
        assert rows[row] == (b, vis - 1) and 0 <= pb < pe and zero == 0
        assert lo == 0 or (sinks < lo < vis and lo == vis - window)
        pieces[row].append(slot)
        for v in range(pb, pe):
            load, s = _tile_tokens(v, lo, vis, sinks)
            assert min(load) >= 0 and max(load) // 64 <= (vis - 1) // 64 < info.plan.max_pages_needed
            assert s, "a tile with nothing to see"
            seen[row] += s
            tiles += 1
    assert tiles == info.plan.total_tiles
    for t, (b, p) in enumerate(rows):
        want = seen_positions(p, window, sinks) if p < 10 ** 6 else list(range(sinks)) + list(range(p - window + 1, p + 1))
        assert sorted(seen[t]) == want, (t, p)
    slots = [s for t in pieces for s in pieces[t] if len(pieces[t]) > 1]
    assert sorted(slots) == list(range(info.plan.num_partials))
    assert all(s == [-1] for s in pieces.values() if len(s) == 1)


def test_window_plan_is_the_decode_plan_when_it_covers_all(api):
    seq, q = [700, 64, 1, 1500], [2, 2, 1, 3]
    a, _ = api.mla_decode_plan_host(seq, q, 9)
    for window, sinks in [(1500, 0), (1, 1499), (2 ** 31 - 1, 2 ** 31 - 1)]:
        b, _ = api.mla_window_plan_host(seq, q, window, sinks, 9)
        assert np.array_equal(a[1:], b[1:])


@pytest.mark.parametrize("args", [([5], [1], 0, 4), ([5], [1], -1, 4), ([5], [1], 1, -1), ([0], [0], 1, 1),
                                  ([5], [6], 1, 1), ([5], [-1], 1, 1)])
def test_window_plan_refusals(api, args):
    seq, q, window, sinks = args
    info = _lib.mla_window_info()
    buf = np.zeros(4096, np.int32)
    sl, ql = np.array(seq, np.int32), np.array(q, np.int32)
    P32 = C.POINTER(C.c_int32)
    st = _lib.lib().mla_window_plan_host(sl.ctypes.data_as(P32), ql.ctypes.data_as(P32), 1, window, sinks, 4,
                                         buf.ctypes.data_as(C.c_void_p), buf.nbytes, C.byref(info))
    assert st == 1


def test_window_plan_call_bounds_its_buffers(api):
    """mla_window_plan: refused before anything is copied, whatever the buffer's size is said to be."""
    lib = _lib.lib()
    P32 = C.POINTER(C.c_int32)
    info = _lib.mla_window_info()
    sl, ql = np.array([500], np.int32), np.array([600], np.int32)

    def call(dev=0x10000, nbytes=1 << 62, B=1, window=5, sinks=0, clusters=4, q=ql):
        return lib.mla_window_plan(sl.ctypes.data_as(P32), q.ctypes.data_as(P32), B, window, sinks, clusters,
                                   C.c_void_p(dev), nbytes, C.byref(info), None)

    assert call() == 1                                       # 600 rows of 500 tokens
    for kw in [dict(dev=0), dict(dev=0x10008), dict(B=-1), dict(clusters=0)]:
        assert call(**kw) in (1, 2), kw
    one = np.array([1], np.int32)
    assert call(q=one, window=0) == 1 and call(q=one, sinks=-1) == 1 and call(q=one, nbytes=16) == 1


def _decode_args(info, kv=0x10000, q=0x20000, o=0x30000, bt=0x40000, plan=0x50000, err=0x60000, ws=0x70000, scale=0.07,
                 pages=10, cols=64):
    return [C.c_void_p(q), C.c_void_p(q), C.c_void_p(kv), pages, C.c_void_p(bt), cols, C.c_void_p(plan), C.byref(info),
            scale, C.c_void_p(ws), 1 << 40, C.c_void_p(o), None, C.c_void_p(err), None]


def test_window_decode_refusals(api):
    lib = _lib.lib()
    _, info = api.mla_window_plan_host([500], [1], 100, 4, 4)
    _, full = api.mla_decode_plan_host([500], [1], 4)
    bad = [dict(kv=0), dict(q=0x20008), dict(o=0), dict(err=0x60002), dict(scale=0.0), dict(scale=float("nan")),
           dict(pages=0), dict(cols=7), dict(plan=0x50004)]
    for kw in bad:
        assert lib.mla_decode_window(*_decode_args(info, **kw)) in (1, 2), kw
    # a plan of the other kind
    other = _lib.mla_window_info()
    C.memmove(C.byref(other), C.byref(full), C.sizeof(full))
    other.window, other.sinks = 100, 4
    assert lib.mla_decode_window(*_decode_args(other)) == 1 and b"window plan" in lib.mla_last_error()
    a = _decode_args(info)
    a[7] = C.byref(info.plan)
    assert lib.mla_decode_paged(*a) == 1
    assert lib.mla_decode_window(*(_decode_args(info)[:7] + [None] + _decode_args(info)[8:])) == 1
    # no rows: nothing to launch
    _, empty = api.mla_window_plan_host([500], [0], 100, 4, 4)
    assert lib.mla_decode_window(*_decode_args(empty, kv=0)) == 0


def test_chunk_window_workspace_and_refusals(api):
    size = api.mla_prefill_window_workspace_size
    per = lambda n: (n * 1152 + 15) // 16 * 16 + 2 * n * 128 * 128 * 2  # noqa: E731
    assert size([300], [1000], 511, 4) == per(4 + 511 + 299)
    assert size([300], [1000], 10000, 4) == per(1000) and size([300], [1000], 1, 701) == per(1000)
    assert size([300, 1], [1000, 77], 1, 0) == per(384 + 1)      # a sequence starts at a multiple of 128
    assert size([], [], 1, 0) == 0
    for args in [([0], [5], 1, 0), ([6], [5], 1, 0), ([1], [5], 0, 0), ([1], [5], 1, -1), ([1] * 65, [5] * 65, 1, 0)]:
        with pytest.raises(api.MlaError):
            size(*args)
    with pytest.raises(ValueError):
        size([1, 2], [5], 1, 0)
    for window, sinks in [(2 ** 32 + 1, 0), (1, 2 ** 31)]:   # not cut to 32 bits
        with pytest.raises(ValueError):
            size([1], [5], window, sinks)
        with pytest.raises(ValueError):
            api.mla_window_plan_host([5], [1], window, sinks, 4)
    lib = _lib.lib()
    P32 = C.POINTER(C.c_int32)

    def call(ids=(0,), starts=(0,), q=(300,), n=(1000,), window=100, sinks=4, batch=1, cols=16, ws=1 << 40, scale=0.07,
             out=0x90000):
        arrs = [np.array(x, np.int32) for x in (ids, starts, q, n)]
        p = [C.c_void_p(0x10000 + 0x1000 * i) for i in range(8)]
        return lib.mla_prefill_window_batch(p[0], p[1], *[a.ctypes.data_as(P32) for a in arrs], len(ids), window, sinks,
                                            p[2], 100, p[3], batch, cols, p[4], p[5], scale, p[6], ws, C.c_void_p(out),
                                            p[7], None)

    for kw in [dict(window=0), dict(sinks=-1), dict(ids=(1,)), dict(ids=(-1,)), dict(starts=(-1,)), dict(q=(0,)),
               dict(q=(1001,)), dict(cols=15), dict(ws=1000), dict(scale=-1.0), dict(out=0), dict(out=0x90008),
               dict(n=(2 ** 31 - 1,), window=2 ** 31 - 1)]:
        assert call(**kw) in (1, 2), kw


def test_append_rope_fp8_refusals(api):
    lib = _lib.lib()

    def call(n=4, c=0x10000, q=0x20000, q_r=0x900000, slots=0x30000, table=0x40000, pos=0x50000, max_pos=9, pages=3,
             scales=0x60000):
        v = lambda a: C.c_void_p(a) if a else None  # noqa: E731
        return lib.mla_kv_append_rope_fp8(v(c), v(0x70000), v(q), v(pos), v(table), max_pos, v(slots), n, v(0x80000),
                                          v(scales), pages, v(q_r), v(0xA0000), None)

    for kw in [dict(n=-1), dict(c=0), dict(q=0), dict(q_r=0), dict(q_r=0x20010), dict(max_pos=0), dict(pages=0)]:
        assert call(**kw) == 1, kw
    for kw in [dict(c=0x10008), dict(slots=0x30004), dict(pos=0x50002), dict(table=0x40004), dict(scales=0x60004),
               dict(q=0x20002)]:
        assert call(**kw) == 2, kw
    assert call(n=0, c=0) == 0


def test_w4_refusals(api):
    lib = _lib.lib()

    def call(f="mla_absorb_q_w4", x=0x10000, w=0x2000000, s=0x3000000, group=64, y=0x4000000, T=2, err=0x50000):
        v = lambda a: C.c_void_p(a) if a else None  # noqa: E731
        return getattr(lib, f)(v(x), v(w), v(s), group, v(y), T, v(err), None)

    for f in ("mla_absorb_q_w4", "mla_up_v_w4"):
        for kw, want in [(dict(T=-1), 1), (dict(T=2 ** 18 + 1), 1), (dict(group=16), 3), (dict(group=0), 3), (dict(x=0), 1),
                         (dict(w=0), 1), (dict(s=0), 1), (dict(y=0), 1), (dict(err=0), 1), (dict(x=0x10008), 2),
                         (dict(y=0x4000002), 2), (dict(err=0x50002), 2), (dict(y=0x10100), 1), (dict(T=0, x=0), 0)]:
            assert call(f, **kw) == want, (f, kw)
    p = C.c_void_p(0x10000)
    assert lib.mla_pack_w4(p, 128, 128, 64, p, p, None) == 3 and lib.mla_pack_w4(p, 128, 512, 48, p, p, None) == 3
    assert lib.mla_pack_w4(None, 128, 512, 64, p, p, None) == 1
    assert lib.mla_pack_w4(p, 512, 128, 64, C.c_void_p(0x10004), p, None) == 2


def test_pack_w4_group_is_not_cut_to_32_bits(api):
    torch = pytest.importorskip("torch")
    w = torch.zeros((128, 128, 512), dtype=torch.bfloat16)
    for group in (2 ** 32 + 32, 2 ** 33 + 64, -(2 ** 32) + 64, 0, 1024):
        with pytest.raises(ValueError, match="group"):
            api.mla_pack_w4(w, group)
    with pytest.raises(TypeError):
        api.mla_pack_w4(w, 64.0)


def test_sequence_lists_are_not_cut_to_32_bits(api):
    far = np.array([2 ** 32 + 500])                          # int32 would wrap to 500
    for lists in [(far, [1]), ([500], far), ([500.5], [1]), ([[500]], [[1]]), (500, 1)]:
        with pytest.raises(ValueError):
            api.mla_window_plan_host(*lists, 100, 4, 4)
        with pytest.raises(ValueError):
            api.mla_prefill_window_workspace_size(lists[1], lists[0], 100, 4)
    assert api.mla_prefill_window_workspace_size(np.array([1]), (500,), 600, 0) == 500 * 1152 + 2 * 500 * 128 * 128 * 2
    assert api.mla_window_plan_host([], [], 100, 4, 4)[1].plan.T == 0
