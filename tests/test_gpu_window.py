"""Windowed attention with sinks (single tokens and chunks, bf16 and FP8 caches) against 64 bits."""
import ctypes as C

import numpy as np
import pytest

import oracle
from mla_latent_kv_02_gb300 import workloads as wl

from _helpers import to_bf16, to_np
from _window_ref import bf16, chunk, decode_row, seen_positions

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from mla_latent_kv_02_gb300 import api as a
    a.mla_version()
    return a


class Cache:
    """A paged cache of n_b tokens a sequence; pages that no row may read are
    NaN and -1 in the table, and so are slots past a sequence's end (zero)."""

    def __init__(self, api, seq_lens, kind, seed, extra_pages=3, keep=None):
        rng = np.random.default_rng(seed)
        self.kind, self.n = kind, list(seq_lens)
        pages = [(n + 63) // 64 for n in self.n]
        pool = sum(pages) + extra_pages
        perm = rng.permutation(pool).astype(np.int32)
        self.bt = np.full((len(self.n), max(pages) + 1), -1, np.int32)
        k = 0
        for b, m in enumerate(pages):
            self.bt[b, :m] = perm[k:k + m]
            k += m
        self.c = [bf16(rng, (n, 512)) for n in self.n]
        self.r = [bf16(rng, (n, 64)) for n in self.n]
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        seq = np.repeat(np.arange(len(self.n), dtype=np.int32), self.n)
        pos = np.concatenate([np.arange(n, dtype=np.int32) for n in self.n])
        slots = torch.from_numpy(api.mla_slot_mapping(self.bt, seq, pos)).cuda()
        c, r = to_bf16(np.concatenate(self.c), "cuda"), to_bf16(np.concatenate(self.r), "cuda")
        if kind == "bf16":
            self.kv = torch.zeros((pool, 64, 576), dtype=torch.bfloat16, device="cuda")
            api.mla_kv_append(c, r, slots, self.kv, err)
        else:
            self.rows = torch.zeros((pool, 64, 640), dtype=torch.uint8, device="cuda")
            self.scales = torch.ones((pool, 64), dtype=torch.float32, device="cuda")
            api.mla_kv_append_fp8(c, r, slots, self.rows, self.scales, err)
            for b in range(len(self.n)):                     # the values the codes stand for
                codes, sc = oracle.fp8_cache.quantize_rows(self.c[b])
                self.c[b] = oracle.fp8_cache.dequantize_rows(codes, sc)
        if keep is not None:                                 # evict what no row sees
            for b in range(len(self.n)):
                for pg in range(pages[b]):
                    if pg not in keep[b]:
                        pid = int(self.bt[b, pg])
                        if kind == "bf16":
                            self.kv[pid] = float("nan")
                        else:
                            self.rows[pid] = 0x7F
                            self.scales[pid] = float("nan")
                        self.bt[b, pg] = -1
        self.table = torch.from_numpy(self.bt).cuda()
        torch.cuda.synchronize()
        assert int(err.item()) == 0

    def tokens(self, b, positions):
        c = torch.from_numpy(self.c[b][positions].astype(np.float64)).cuda()
        return c, torch.from_numpy(self.r[b][positions].astype(np.float64)).cuda()


def _kept_pages(seq_lens, q_lens, window, sinks):
    return [{j // 64 for i in range(q) for j in seen_positions(n - q + i, window, sinks)}
            for n, q in zip(seq_lens, q_lens)]


def _decode(api, cache, q_abs, q_r, plan, stream=None, o=None, lse=None, err=None):
    T = q_abs.shape[0]
    o = torch.full((T, 128, 512), float("nan"), dtype=torch.bfloat16, device="cuda") if o is None else o
    lse = torch.full((T, 128), float("nan"), dtype=torch.float32, device="cuda") if lse is None else lse
    err = torch.zeros(1, dtype=torch.int32, device="cuda") if err is None else err
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    if cache.kind == "bf16":
        api.mla_decode_window(q_abs, q_r, cache.kv, cache.table, plan, o, err, lse=lse, stream=stream)
    else:
        api.mla_decode_window_fp8(q_abs, q_r, cache.rows, cache.scales, cache.table, plan, o, err, lse=lse,
                                  stream=stream)
    return o, lse, err


def _queries(T, seed, q_std=0.5):
    rng = np.random.default_rng(seed)
    return to_bf16(bf16(rng, (T, 128, 512), q_std), "cuda"), to_bf16(bf16(rng, (T, 128, 64)), "cuda")


def _check_decode(cache, q_abs, q_r, o, lse, q_lens, window, sinks, rows=None):
    t = 0
    for b, q in enumerate(q_lens):
        for i in range(q):
            if rows is None or t in rows:
                c, r = cache.tokens(b, seen_positions(cache.n[b] - q + i, window, sinks))
                wo, wl_, to, tl = decode_row(q_abs[t].double(), q_r[t].double(), c, r)
                d = (o[t].double() - wo).abs()
                assert bool((d <= to).all()), (t, b, i, float((d / to).max()))
                dl = (lse[t].double() - wl_).abs()
                assert bool((dl <= tl).all()), (t, "lse", float((dl / tl).max()))
            t += 1


RESIDUES = list(range(200, 265))                             # every place of the window's start in its page
DECODE_CASES = [
    # seq_lens, q_lens, window, sinks, clusters
    ([1], [1], 1, 0, None),
    ([1, 2, 64, 65], [1, 1, 1, 1], 1, 4, None),
    ([1024], [1], 512, 4, None),
    ([1024], [1], 512, 0, 1),
    (RESIDUES, [1] * len(RESIDUES), 100, 4, None),           # merged, separate and shared sink tiles
    (RESIDUES, [1] * len(RESIDUES), 64, 64, 7),              # a full sink page
    (RESIDUES, [1] * len(RESIDUES), 30, 75, None),           # a full page and a rest
    (RESIDUES, [1] * len(RESIDUES), 70, 63, None),           # split of 64: never merged
    (RESIDUES, [2] * len(RESIDUES), 1, 8, None),
    ([300, 500], [1, 2], 4000, 4, 4),                        # the window covers all
    ([300, 500], [1, 2], 17, 4000, 4),                       # the sinks cover all
    ([130, 700, 90, 4096], [3, 0, 5, 2], 129, 5, None),
    ([700, 333, 130], [16, 16, 16], 65, 9, 3),               # equal row counts: lanes
    ([2000], [40], 333, 20, None),
    ([64 * 40 + 1], [1], 64, 1, 2),
]


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("case", range(len(DECODE_CASES)))
def test_decode_window(api, kind, case):
    seq, q, window, sinks, clusters = DECODE_CASES[case]
    cache = Cache(api, seq, kind, 100 + case, keep=_kept_pages(seq, q, window, sinks))
    q_abs, q_r = _queries(sum(q), 200 + case)
    plan = api.mla_window_plan(seq, q, window, sinks, num_clusters=clusters)
    o, lse, err = _decode(api, cache, q_abs, q_r, plan)
    assert api.mla_check(err) == 0
    _check_decode(cache, q_abs, q_r, o, lse, q, window, sinks)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_decode_window_that_covers_all_is_the_full_decode(api, kind):
    seq, q = [700, 64, 1, 1500], [2, 2, 1, 3]
    cache = Cache(api, seq, kind, 7)
    q_abs, q_r = _queries(sum(q), 8)
    want = torch.empty((sum(q), 128, 512), dtype=torch.bfloat16, device="cuda")
    wlse = torch.empty((sum(q), 128), dtype=torch.float32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    full = api.mla_decode_plan(seq, q, num_clusters=9)
    if kind == "bf16":
        api.mla_decode_paged(q_abs, q_r, cache.kv, cache.table, full, want, err, lse=wlse)
    else:
        api.mla_decode_paged_fp8(q_abs, q_r, cache.rows, cache.scales, cache.table, full, want, err, lse=wlse)
    assert api.mla_check(err) == 0
    for window, sinks in [(1500, 0), (2 ** 31 - 1, 3), (1, 1499), (1, 2 ** 31 - 1)]:
        plan = api.mla_window_plan(seq, q, window, sinks, num_clusters=9)
        o, lse, err = _decode(api, cache, q_abs, q_r, plan)
        assert api.mla_check(err) == 0
        assert torch.equal(o.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, wlse)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_decode_window_large_scores(api, kind):
    """Scores of tens: the running maximum moves by more than the lazy threshold between tiles."""
    seq, q, window, sinks = [900, 1200], [1, 2], 700, 4
    cache = Cache(api, seq, kind, 70)
    q_abs, q_r = _queries(3, 71, q_std=6.0)
    plan = api.mla_window_plan(seq, q, window, sinks, num_clusters=3)
    o, lse, err = _decode(api, cache, q_abs, q_r, plan)
    assert api.mla_check(err) == 0
    _check_decode(cache, q_abs, q_r, o, lse, q, window, sinks)


def _poison(cache, keep):
    """NaN and infinities in every slot of the pool but the tokens keep[b] of each sequence."""
    pool = (cache.kv if cache.kind == "bf16" else cache.rows).shape[0]
    hold = torch.zeros(pool * 64, dtype=torch.bool, device="cuda")
    for b, tokens in enumerate(keep):
        t = torch.tensor(sorted(tokens), dtype=torch.long, device="cuda")
        hold[cache.table[b].long()[t // 64] * 64 + t % 64] = True
    bad = (~hold).nonzero().flatten()
    if cache.kind == "bf16":
        flat = cache.kv.view(-1, 576)
        flat[bad[0::2]] = float("nan")
        flat[bad[1::2]] = float("inf")
    else:
        cache.rows.view(-1, 640)[bad] = 0x7F                 # NaN codes, and NaN in the RoPE bytes
        sc = cache.scales.view(-1)
        sc[bad[0::3]] = float("nan")
        sc[bad[1::3]] = float("inf")
        sc[bad[2::3]] = 0.0


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("window,sinks", [(100, 4), (64, 64), (30, 75), (1, 0)])
def test_decode_window_masked_slots_may_hold_anything(api, kind, window, sinks):
    seq, q = RESIDUES, [1] * len(RESIDUES)
    cache = Cache(api, seq, kind, 17)
    _poison(cache, [seen_positions(n - 1, window, sinks) for n in seq])
    q_abs, q_r = _queries(sum(q), 18)
    o, lse, err = _decode(api, cache, q_abs, q_r, api.mla_window_plan(seq, q, window, sinks))
    assert api.mla_check(err) == 0
    _check_decode(cache, q_abs, q_r, o, lse, q, window, sinks)


def test_decode_window_fp8_scale_out_of_range_is_reported(api):
    """A seen token's scale outside [2^-15, 2^7] sets the flag of the full decode."""
    seq, q = [300], [1]
    cache = Cache(api, seq, "fp8", 19)
    cache.scales[int(cache.bt[0, 4]), 40] = 2.0 ** 9          # position 296: in the window
    q_abs, q_r = _queries(1, 20)
    _, _, err = _decode(api, cache, q_abs, q_r, api.mla_window_plan(seq, q, 100, 4))
    assert int(err.item()) == api.DEVERR_FP8_RANGE


def test_decode_window_beyond_32_bit_offsets(api):
    """Pages past 4 GiB of the pool."""
    seq, q, window, sinks = [500, 260], [1, 2], 200, 4
    small = Cache(api, seq, "bf16", 12)
    pool = 62000                                             # 4.6 GB
    kv = torch.zeros((pool, 64, 576), dtype=torch.bfloat16, device="cuda")
    off = pool - small.kv.shape[0]
    kv[off:] = small.kv
    small.kv = kv
    small.table = torch.where(small.table >= 0, small.table + off, small.table)
    q_abs, q_r = _queries(3, 13)
    o, lse, err = _decode(api, small, q_abs, q_r, api.mla_window_plan(seq, q, window, sinks))
    assert api.mla_check(err) == 0
    _check_decode(small, q_abs, q_r, o, lse, q, window, sinks)


@pytest.mark.parametrize("n", [2 ** 31 - 1, 2 ** 31 - 63])
def test_decode_window_of_the_longest_sequence(api, n):
    """A sequence of 2^31 - 1 positions whose table maps the pages it sees only."""
    window, sinks = 100, 4
    first = n - window                                       # the window's first token
    pages = [0] + list(range(first // 64, (n - 1) // 64 + 1))
    cols = (n - 1) // 64 + 1
    table = torch.full((1, cols), -1, dtype=torch.int32, device="cuda")
    table[0, torch.tensor(pages, device="cuda")] = torch.arange(len(pages), dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(3)
    c, r = bf16(rng, (len(pages) * 64, 512)), bf16(rng, (len(pages) * 64, 64))
    kv = torch.cat([to_bf16(c, "cuda"), to_bf16(r, "cuda")], dim=1).view(len(pages), 64, 576).contiguous()
    q_abs, q_r = _queries(1, 4)
    plan = api.mla_window_plan([n], [1], window, sinks)
    o = torch.empty((1, 128, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((1, 128), dtype=torch.float32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.mla_decode_window(q_abs, q_r, kv, table, plan, o, err, lse=lse)
    assert api.mla_check(err) == 0
    at = list(range(sinks)) + [64 * pages.index(j // 64) + j % 64 for j in range(first, n)]
    wo, wl_, to, tl = decode_row(q_abs[0].double(), q_r[0].double(), torch.from_numpy(c[at].astype(np.float64)).cuda(),
                                 torch.from_numpy(r[at].astype(np.float64)).cuda())
    assert bool(((o[0].double() - wo).abs() <= to).all()) and bool(((lse[0].double() - wl_).abs() <= tl).all())


def test_decode_window_bad_pages_are_reported(api):
    seq, q, window, sinks = [1000], [1], 200, 4
    cache = Cache(api, seq, "bf16", 14)
    q_abs, q_r = _queries(1, 15)
    for page in (0, 15):                                     # the sinks' page of a merged tile, a window page
        table = cache.table.clone()
        table[0, page] = cache.kv.shape[0] if page else -1
        saved, cache.table = cache.table, table
        _, _, err = _decode(api, cache, q_abs, q_r, api.mla_window_plan(seq, q, window, sinks))
        with pytest.raises(api.MlaError):
            api.mla_check(err)
        assert int(err.item()) == api.DEVERR_PAGE_OOB
        cache.table = saved


def test_decode_window_two_streams_and_a_graph(api):
    """Two plans at once, and a captured call replayed after its inputs changed in place."""
    seq, q, window, sinks = [700, 900, 333], [2, 1, 2], 257, 6
    cache = Cache(api, seq, "fp8", 21)
    qs = [_queries(5, 22), _queries(5, 23)]
    plans = [api.mla_window_plan(seq, q, window, sinks, num_clusters=c) for c in (5, 11)]
    want = [_decode(api, cache, *qs[i], plans[i]) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [_decode(api, cache, *qs[i], plans[i], stream=streams[i]) for i in range(2)]
        torch.cuda.synchronize()
        for (o, lse, err), (wo, wl_, _) in zip(got, want):
            assert int(err.item()) == 0 and torch.equal(o, wo) and torch.equal(lse, wl_)
    q_abs, q_r = qs[0][0].clone(), qs[0][1].clone()
    o, lse, err = (x.clone() for x in want[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _decode(api, cache, q_abs, q_r, plans[0], o=o, lse=lse, err=err)
    q_abs.copy_(qs[1][0])
    q_r.copy_(qs[1][1])
    g.replay()
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    _check_decode(cache, q_abs, q_r, o, lse, q, window, sinks)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("limit", [64, 5000, 12000])
def test_decode_window_wait_expiry_is_reported(api, kind, limit):
    """Waits that run out early, at the set-up or among the tiles: reported, drained, and the next call is right."""
    seq, q, window, sinks = [700, 900, 333], [2, 1, 2], 257, 6
    cache = Cache(api, seq, kind, 25)
    q_abs, q_r = _queries(5, 26)
    plan = api.mla_window_plan(seq, q, window, sinks, num_clusters=3)
    try:
        api.mla_debug_set_decode_wait_limit(limit)
        _, _, err = _decode(api, cache, q_abs, q_r, plan)
    finally:
        api.mla_debug_set_decode_wait_limit(0)
    torch.cuda.synchronize()
    assert int(err.item()) in ((api.DEVERR_TIMEOUT,) if limit == 64 else (0, api.DEVERR_TIMEOUT))
    o, lse, err = _decode(api, cache, q_abs, q_r, plan)
    assert api.mla_check(err) == 0
    _check_decode(cache, q_abs, q_r, o, lse, q, window, sinks)


def test_decode_window_into_reuses_a_plan(api):
    seq, q = [700, 900], [1, 1]
    cache = Cache(api, seq, "bf16", 31)
    q_abs, q_r = _queries(2, 32)
    plan = api.mla_window_plan(seq, q, 300, 4)
    torch.cuda.synchronize()
    again = api.mla_window_plan(seq, q, 100, 2, into=plan)
    assert again.plan.data_ptr() == plan.plan.data_ptr()
    o, lse, err = _decode(api, cache, q_abs, q_r, again)
    assert api.mla_check(err) == 0
    _check_decode(cache, q_abs, q_r, o, lse, q, 100, 2)


# ------------------------------------------------------------------ chunks
CHUNK_CASES = [
    # n_tokens, q_lens, window, sinks
    ([1], [1], 1, 0),
    ([5, 300], [5, 1], 2, 1),
    ([1000], [300], 511, 4),
    ([1000], [300], 64, 0),                                  # rows that see nothing of their first tiles
    ([700, 260, 513], [256, 256, 257], 1, 0),
    ([2000, 129], [130, 128], 333, 130),
    ([900], [400], 5000, 4),                                 # the window covers all
    ([900], [400], 7, 2000),                                 # the sinks cover all
    ([1500, 1501, 1502], [1, 129, 512], 200, 64),
]


def _chunk(api, cache, q_c, q_r, ids, starts, q, n, window, sinks, w_uk, w_uv, out, stream=None, err=None):
    ws = torch.empty(api.mla_prefill_window_workspace_size(q, n, window, sinks), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda") if err is None else err
    tail = (cache.table, ids, starts, q, n, window, sinks, w_uk, w_uv, ws, out, err)
    if cache.kind == "bf16":
        api.mla_prefill_window_batch(q_c, q_r, cache.kv, *tail, stream=stream)
    else:
        api.mla_prefill_window_batch_fp8(q_c, q_r, cache.rows, cache.scales, *tail, stream=stream)
    return err


def _weights(seed):
    rng = np.random.default_rng(seed)
    std = 512 ** -0.5
    return to_bf16(bf16(rng, (128, 128, 512), std), "cuda"), to_bf16(bf16(rng, (128, 512, 128), std), "cuda")


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("case", range(len(CHUNK_CASES)))
def test_chunk_window(api, kind, case):
    n, q, window, sinks = CHUNK_CASES[case]
    cache = Cache(api, n, kind, 300 + case, keep=_kept_pages(n, q, window, sinks))
    w_uk, w_uv = _weights(1)
    gap = 3                                                  # rows of no chunk between the chunks, left as they were
    starts = [sum(q[:i]) + gap * (i + 1) for i in range(len(q))]
    T = starts[-1] + q[-1] + gap
    rng = np.random.default_rng(400 + case)
    q_c, q_r = to_bf16(bf16(rng, (T, 128, 128)), "cuda"), to_bf16(bf16(rng, (T, 128, 64)), "cuda")
    out = torch.full((T, 128, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    err = _chunk(api, cache, q_c, q_r, range(len(n)), starts, q, n, window, sinks, w_uk, w_uv, out)
    assert api.mla_check(err) == 0
    uk, uv = w_uk.double(), w_uv.double()
    inside = torch.zeros(T, dtype=torch.bool, device="cuda")
    for b, (N, M, s0) in enumerate(zip(n, q, starts)):
        keep = sorted({j for i in range(M) for j in seen_positions(N - M + i, window, sinks)})
        c, r = cache.tokens(b, keep)
        want, tol = chunk(q_c[s0:s0 + M].double(), q_r[s0:s0 + M].double(), c, r,
                          torch.arange(N - M, N, device="cuda"), torch.tensor(keep, device="cuda"), window, sinks, uk, uv)
        d = (out[s0:s0 + M].double() - want).abs()
        assert bool((d <= tol).all()), (b, float((d / tol).max()))
        inside[s0:s0 + M] = True
    assert bool((out[~inside] == 9.0).all()), "a row of no chunk was written"


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_chunk_window_reads_kept_tokens_only(api, kind):
    n, q, window, sinks = [1000, 700], [300, 256], 200, 5
    cache = Cache(api, n, kind, 43)
    keep = [sorted({j for i in range(m) for j in seen_positions(N - m + i, window, sinks)}) for N, m in zip(n, q)]
    w_uk, w_uv = _weights(5)
    rng = np.random.default_rng(44)
    T = sum(q)
    q_c, q_r = to_bf16(bf16(rng, (T, 128, 128)), "cuda"), to_bf16(bf16(rng, (T, 128, 64)), "cuda")
    want, out = (torch.empty((T, 128, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    err = _chunk(api, cache, q_c, q_r, [0, 1], [0, 300], q, n, window, sinks, w_uk, w_uv, want)
    assert api.mla_check(err) == 0
    _poison(cache, keep)
    err = _chunk(api, cache, q_c, q_r, [0, 1], [0, 300], q, n, window, sinks, w_uk, w_uv, out)
    assert api.mla_check(err) == 0 and torch.equal(out, want)


def test_chunk_window_keeps_sequences_apart(api):
    """NaN in one sequence's tokens stays in that sequence."""
    n, q, window, sinks = [500, 610, 430], [300, 256, 257], 200, 5
    cache = Cache(api, n, "bf16", 45)
    w_uk, w_uv = _weights(6)
    rng = np.random.default_rng(46)
    T = sum(q)
    q_c, q_r = to_bf16(bf16(rng, (T, 128, 128)), "cuda"), to_bf16(bf16(rng, (T, 128, 64)), "cuda")
    want, out = (torch.empty((T, 128, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    starts = [0, 300, 556]
    err = _chunk(api, cache, q_c, q_r, [0, 1, 2], starts, q, n, window, sinks, w_uk, w_uv, want)
    cache.kv[cache.table[1, :10].long()] = float("nan")
    err = _chunk(api, cache, q_c, q_r, [0, 1, 2], starts, q, n, window, sinks, w_uk, w_uv, out, err=err)
    assert api.mla_check(err) == 0
    assert torch.equal(out[:300], want[:300]) and torch.equal(out[556:], want[556:])
    assert bool(torch.isnan(out[300:556]).all())


def test_chunk_window_that_covers_all_is_the_branch_without(api):
    n, q = [700, 900], [300, 256]
    cache = Cache(api, n, "bf16", 41)
    w_uk, w_uv = _weights(2)
    rng = np.random.default_rng(42)
    T = sum(q)
    q_c, q_r = to_bf16(bf16(rng, (T, 128, 128)), "cuda"), to_bf16(bf16(rng, (T, 128, 64)), "cuda")
    want = torch.empty((T, 128, 128), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(api.mla_prefill_batch_workspace_size(n), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.mla_prefill_decompress_batch(q_c, q_r, cache.kv, cache.table, [0, 1], [0, 300], q, n, w_uk, w_uv, ws, want, err)
    assert api.mla_check(err) == 0
    for window, sinks in [(900, 0), (2 ** 31 - 1, 2 ** 31 - 1), (1, 900)]:
        out = torch.empty_like(want)
        err = _chunk(api, cache, q_c, q_r, [0, 1], [0, 300], q, n, window, sinks, w_uk, w_uv, out)
        assert api.mla_check(err) == 0
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))


def test_chunk_window_agrees_with_single_tokens(api):
    """The chunk form and the absorbed form of the same rows: out = o_lat . W_UV, q_abs = q_c . W_UK."""
    n, q, window, sinks = [1200], [300], 333, 4
    cache = Cache(api, n, "fp8", 51)
    w_uk, w_uv = _weights(3)
    rng = np.random.default_rng(52)
    q_c, q_r = to_bf16(bf16(rng, (300, 128, 128)), "cuda"), to_bf16(bf16(rng, (300, 128, 64)), "cuda")
    out = torch.empty((300, 128, 128), dtype=torch.bfloat16, device="cuda")
    err = _chunk(api, cache, q_c, q_r, [0], [0], q, n, window, sinks, w_uk, w_uv, out)
    assert api.mla_check(err) == 0
    q_abs = torch.empty((300, 128, 512), dtype=torch.bfloat16, device="cuda")
    api.mla_absorb_q(q_c, w_uk, q_abs, err)
    o, _, _ = _decode(api, cache, q_abs, q_r, api.mla_window_plan(n, q, window, sinks), err=err)
    out2 = torch.empty_like(out)
    api.mla_up_v(o, w_uv, out2, err)
    assert api.mla_check(err) == 0
    a, b = to_np(out).astype(np.float64), to_np(out2).astype(np.float64)
    # each side rounds about six times at 2^-8 (queries or keys, values, probabilities, output) in random directions
    assert np.linalg.norm(a - b) <= 12 * 2.0 ** -8 / np.sqrt(3) * np.linalg.norm(a)


def test_chunk_window_captured(api):
    n, q, window, sinks = [800], [280], 200, 4
    cache = Cache(api, n, "bf16", 61)
    w_uk, w_uv = _weights(4)
    rng = np.random.default_rng(62)
    q_c, q_r = to_bf16(bf16(rng, (280, 128, 128)), "cuda"), to_bf16(bf16(rng, (280, 128, 64)), "cuda")
    want = torch.empty((280, 128, 128), dtype=torch.bfloat16, device="cuda")
    err = _chunk(api, cache, q_c, q_r, [0], [0], q, n, window, sinks, w_uk, w_uv, want)
    assert api.mla_check(err) == 0
    out = torch.zeros_like(want)
    ws = torch.empty(api.mla_prefill_window_workspace_size(q, n, window, sinks), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.mla_prefill_window_batch(q_c, q_r, cache.kv, cache.table, [0], [0], q, n, window, sinks, w_uk, w_uv, ws, out, err)
    for _ in range(2):
        out.zero_()
        g.replay()
        assert api.mla_check(err) == 0 and torch.equal(out, want)
