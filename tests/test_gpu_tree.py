"""Draft trees over the paged cache: layout, attention, compaction and page copies against plain forms."""
import numpy as np
import pytest

import oracle

from _helpers import to_bf16
from _tree_ref import kept, masks, path, seen, tree, words_of
from _window_ref import bf16, decode_row

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from mla_latent_kv_02_gb300 import api as a
    a.mla_version()
    return a


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def starts_of(nodes):
    return [sum(nodes[:i]) for i in range(len(nodes) + 1)]


# ------------------------------------------------------------------ layout
LAYOUTS = [[1], [256], [64, 65, 1, 63], [0, 5, 0], [200, 129, 7], [32] * 100]


@pytest.mark.parametrize("shape", ["tree", "chain", "star"])
@pytest.mark.parametrize("nodes", LAYOUTS, ids=str)
def test_layout(api, nodes, shape):
    rng = np.random.default_rng(len(nodes))
    roots = {"tree": 3, "chain": 1, "star": 256}[shape]
    trees = [tree(7 * b, n, roots, 1 if shape == "chain" else 6) for b, n in enumerate(nodes)]
    T, words = sum(nodes), (max(nodes) + 63) // 64
    ctx = [int(x) for x in rng.integers(0, 300, len(nodes))]
    bt = rng.permutation(len(nodes) * 12).astype(np.int32).reshape(len(nodes), 12)
    pad = 3                                                  # rows past the last tree stay as they are
    m = torch.full((T + pad, words), 77, dtype=torch.int64, device="cuda")
    pos, slots = torch.full((T + pad,), 77, dtype=torch.int32, device="cuda"), torch.full((T + pad,), 77, dtype=torch.int64, device="cuda")
    par = torch.full((T + pad,), 99, dtype=torch.int32, device="cuda")
    par[:T] = i32([p for t in trees for p in t])
    err = word()
    q = i32(starts_of(nodes))
    api.mla_tree_layout(par, q, i32([c + n for c, n in zip(ctx, nodes)]), m, err, positions=pos, slots=slots,
                        block_table=torch.from_numpy(bt).cuda(), num_pages=len(nodes) * 12)
    assert int(err.item()) == 0
    assert (m[:T].cpu().numpy() == masks(trees, words)).all()
    want_p = [c + len(path(t, i)) - 1 for c, t in zip(ctx, trees) for i in range(len(t))]
    want_s = [int(bt[b, (c + i) // 64]) * 64 + (c + i) % 64 for b, (c, n) in enumerate(zip(ctx, nodes)) for i in range(n)]
    assert pos[:T].tolist() == want_p and slots[:T].tolist() == want_s
    assert (m[T:] == 77).all() and (pos[T:] == 77).all() and (slots[T:] == 77).all()
    again = torch.zeros((T + pad, 4), dtype=torch.int64, device="cuda")   # more words than the trees need, masks only
    api.mla_tree_layout(par, q, i32([c + n for c, n in zip(ctx, nodes)]), again, err)
    assert torch.equal(again[:T, :words], m[:T]) and not again[:, words:].any() and not again[T:].any()


def test_layout_judges_its_inputs(api):
    par = i32([-1, 0, 5, -2, 1, -1, 0, -1, 0])
    q, seq = i32([0, 5, 7, 9]), i32([70, 10, 1])            # the third has more nodes than tokens
    m = torch.full((9, 1), 5, dtype=torch.int64, device="cuda")
    pos, slots = torch.full((9,), 5, dtype=torch.int32, device="cuda"), torch.full((9,), 5, dtype=torch.int64, device="cuda")
    bt = torch.tensor([[0, 9], [4, 0], [1, 1]], dtype=torch.int32, device="cuda")
    err = word()
    api.mla_tree_layout(par, q, seq, m, err, positions=pos, slots=slots, block_table=bt, num_pages=4)
    assert int(err.item()) == api.DEVERR_TREE | api.DEVERR_PAGE_OOB
    assert m[:, 0].tolist() == [1, 3, 4, 8, 19, 1, 3, 5, 5]  # bad parents count as -1
    assert pos.tolist() == [65, 66, 65, 65, 67, 8, 9, 5, 5]
    assert slots.tolist() == [-1] * 7 + [5, 5]              # pages 9 and 4 of a pool of 4
    err.zero_()
    for bad in ([0, -1, 7, 9], [0, 5, 4, 9], [0, 5, 7, 10]):
        m.fill_(5)
        api.mla_tree_layout(i32([-1] * 9), i32(bad), i32([70, 70, 70]), m, err)
        assert int(err.item()) == api.DEVERR_TREE
        err.zero_()
    one = torch.zeros((65, 1), dtype=torch.int64, device="cuda")
    api.mla_tree_layout(i32([-1] * 65), i32([0, 65]), i32([70]), one, err)
    assert int(err.item()) == api.DEVERR_TREE and not one.any()   # 65 nodes do not fit a word


# ------------------------------------------------------------------ attention
class Cache:
    """A paged cache in which only the sequences' tokens are finite: other slots and pages hold NaN."""

    def __init__(self, api, seq_lens, kind, seed):
        rng = np.random.default_rng(seed)
        self.kind, self.n = kind, list(seq_lens)
        pages = [(n + 63) // 64 for n in self.n]
        pool = sum(pages) + 2
        perm = rng.permutation(pool).astype(np.int32)
        self.bt = np.full((len(self.n), max(pages) + 1), -1, np.int32)
        k = 0
        for b, m in enumerate(pages):
            self.bt[b, :m] = perm[k:k + m]
            k += m
        self.c = [bf16(rng, (n, 512)) for n in self.n]
        self.r = [bf16(rng, (n, 64)) for n in self.n]
        seq = np.repeat(np.arange(len(self.n), dtype=np.int32), self.n)
        pos = np.concatenate([np.arange(n, dtype=np.int32) for n in self.n])
        slots = torch.from_numpy(api.mla_slot_mapping(self.bt, seq, pos)).cuda()
        c, r = to_bf16(np.concatenate(self.c), "cuda"), to_bf16(np.concatenate(self.r), "cuda")
        err = word()
        if kind == "bf16":
            self.kv = torch.full((pool, 64, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
            api.mla_kv_append(c, r, slots, self.kv, err)
        else:
            self.rows = torch.full((pool, 64, 640), 0x7F, dtype=torch.uint8, device="cuda")
            self.scales = torch.full((pool, 64), float("nan"), dtype=torch.float32, device="cuda")
            api.mla_kv_append_fp8(c, r, slots, self.rows, self.scales, err)
            for b in range(len(self.n)):                     # the values the codes stand for
                self.c[b] = oracle.fp8_cache.dequantize_rows(*oracle.fp8_cache.quantize_rows(self.c[b]))
        self.table = torch.from_numpy(self.bt).cuda()
        assert int(err.item()) == 0

    def tokens(self, b, positions):
        c = torch.from_numpy(self.c[b][positions].astype(np.float64)).cuda()
        return c, torch.from_numpy(self.r[b][positions].astype(np.float64)).cuda()


def queries(T, seed, q_std=0.5):
    rng = np.random.default_rng(seed)
    return to_bf16(bf16(rng, (T, 128, 512), q_std), "cuda"), to_bf16(bf16(rng, (T, 128, 64)), "cuda")


def decode(api, cache, q_abs, q_r, m, plan, stream=None, o=None, lse=None, err=None):
    T = q_abs.shape[0]
    o = torch.full((T, 128, 512), float("nan"), dtype=torch.bfloat16, device="cuda") if o is None else o
    lse = torch.full((T, 128), float("nan"), dtype=torch.float32, device="cuda") if lse is None else lse
    err = word() if err is None else err
    if cache.kind == "bf16":
        api.mla_decode_tree(q_abs, q_r, cache.kv, cache.table, m, plan, o, err, lse=lse, stream=stream)
    else:
        api.mla_decode_tree_fp8(q_abs, q_r, cache.rows, cache.scales, cache.table, m, plan, o, err, lse=lse, stream=stream)
    return o, lse, err


def check(cache, q_abs, q_r, m, o, lse, nodes, rows=None):
    mask = m.cpu().numpy()
    t = 0
    for b, q in enumerate(nodes):
        for i in range(q):
            if rows is None or t in rows:
                at = seen(cache.n[b] - q, i, mask[t])
                if not at:
                    assert not o[t].any() and bool((lse[t] == -float("inf")).all()), (t, "sees nothing")
                else:
                    c, r = cache.tokens(b, at)
                    wo, wl, to, tl = decode_row(q_abs[t].double(), q_r[t].double(), c, r)
                    d = (o[t].double() - wo).abs()
                    assert bool((d <= to).all()), (t, b, i, float((d / to).max()))
                    dl = (lse[t].double() - wl).abs()
                    assert bool((dl <= tl).all()), (t, "lse", float((dl / tl).max()))
            t += 1


DECODES = [
    # tokens before the tree, nodes, clusters
    ([0], [1], None),
    ([0], [5], None),
    ([0, 0, 7], [130, 64, 65], 5),
    ([1, 63, 64, 65, 127, 128], [1, 2, 64, 63, 3, 65], None),
    ([1000], [8], None),
    ([1000], [8], 1),
    ([100, 900, 333], [12, 12, 12], 3),                      # equal trees
    ([130, 0, 700, 90], [30, 3, 0, 17], 4),
    ([2000], [40], None),
    ([70], [256], None),
    (list(range(50, 90)), [3] * 40, 7),                      # the tree's start at every place of a tile's end
]


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("case", range(len(DECODES)))
def test_decode_tree(api, kind, case):
    ctx, nodes, clusters = DECODES[case]
    cache = Cache(api, [c + n for c, n in zip(ctx, nodes)], kind, case)
    T, words = sum(nodes), (max(nodes) + 63) // 64
    m = torch.from_numpy(masks([tree(case + b, n) for b, n in enumerate(nodes)], words)).cuda()
    q_abs, q_r = queries(T, 100 + case)
    plan = api.mla_tree_plan(cache.n, nodes, num_clusters=clusters)
    o, lse, err = decode(api, cache, q_abs, q_r, m, plan)
    assert api.mla_check(err) == 0
    rows = None if T <= 80 else set(range(0, T, T // 40)) | {T - 1}
    check(cache, q_abs, q_r, m, o, lse, nodes, rows)
    again = decode(api, cache, q_abs, q_r, m, plan)         # the same bits twice
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("ctx", [0, 1, 40, 64, 200])
def test_masks_of_any_bits(api, kind, ctx):
    """Masks that are no tree's: empty, full, without the node itself, with bits of later nodes (not read)."""
    nodes = [150]
    cache = Cache(api, [ctx + 150], kind, ctx)
    rng = np.random.default_rng(ctx)
    rows = [words_of([], 3), words_of(range(150), 3), words_of([149], 3), words_of([0], 3)]
    rows += [words_of([k for k in range(150) if rng.random() < p], 3) for p in (0.02, 0.5, 0.9) for _ in range(20)]
    rows += [words_of([], 3)] * (148 - len(rows)) + [words_of([149], 3), words_of([], 3)]
    m = torch.from_numpy(np.array(rows, np.int64)).cuda()
    q_abs, q_r = queries(150, ctx)
    for clusters in (1, 9, None):
        plan = api.mla_tree_plan(cache.n, nodes, num_clusters=clusters)
        o, lse, err = decode(api, cache, q_abs, q_r, m, plan)
        assert api.mla_check(err) == 0
        check(cache, q_abs, q_r, m, o, lse, nodes, set(range(0, 150, 7)) | {0, 1, 2, 3, 148, 149})


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_chain_is_the_causal_decode(api, kind):
    """A tree that is a chain: mla_decode_paged's rows, bit for bit where the plans cut alike."""
    cache = Cache(api, [512, 320], kind, 5)                  # full pages: the causal decode wants them finite
    nodes = [4, 4]
    m = torch.from_numpy(masks([tree(0, 4, 1, 1)] * 2, 1)).cuda()
    q_abs, q_r = queries(8, 5)
    o, lse, _ = decode(api, cache, q_abs, q_r, m, api.mla_tree_plan(cache.n, nodes, num_clusters=1))
    p = api.mla_decode_plan(cache.n, nodes, num_clusters=1)
    o2, lse2, err = torch.empty_like(o), torch.empty_like(lse), word()
    if kind == "bf16":
        api.mla_decode_paged(q_abs, q_r, cache.kv, cache.table, p, o2, err, lse=lse2)
    else:
        api.mla_decode_paged_fp8(q_abs, q_r, cache.rows, cache.scales, cache.table, p, o2, err, lse=lse2)
    assert api.mla_check(err) == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)


def direct(api, plan):
    """The same plan with the smallest workspace: the FP8 pages are converted tile by tile."""
    plan.unpack = True                                       # the workspace is not judged again
    plan.workspace = plan.workspace[:max(16, api.mla_tree_workspace_size(plan.info, False))]
    return plan


@pytest.mark.parametrize("nodes", [[40, 17], [256, 3]])
def test_unpacked_pages_give_the_same_bits(api, nodes):
    cache = Cache(api, [2050 + nodes[0], 700 + nodes[1]], "fp8", 11)
    m = torch.from_numpy(masks([tree(b, n) for b, n in enumerate(nodes)], (max(nodes) + 63) // 64)).cuda()
    q_abs, q_r = queries(sum(nodes), 11)
    plans = [api.mla_tree_plan(cache.n, nodes) for _ in range(2)]
    small = api.mla_tree_workspace_size(plans[0].info, False)
    assert api.mla_tree_workspace_size(plans[0].info, True) == small + plans[0].info.total_pages * 64 * 1152
    o, lse, err = decode(api, cache, q_abs, q_r, m, plans[0])
    assert plans[0].workspace.numel() >= small + plans[0].info.total_pages * 64 * 1152
    o2, lse2, err2 = decode(api, cache, q_abs, q_r, m, direct(api, plans[1]))
    assert plans[1].workspace.numel() < plans[0].workspace.numel()
    assert api.mla_check(err) == 0 and api.mla_check(err2) == 0
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    check(cache, q_abs, q_r, m, o, lse, nodes, set(range(0, sum(nodes), 29)))
    plans[0] = api.mla_tree_plan([90], [2], into=plans[0])   # buffers kept, judged for the new lengths
    few = Cache(api, [90], "fp8", 12)
    m2 = torch.from_numpy(masks([tree(0, 2)], 1)).cuda()
    o3, lse3, err3 = decode(api, few, q_abs[:2], q_r[:2], m2, plans[0])
    assert api.mla_check(err3) == 0
    check(few, q_abs[:2], q_r[:2], m2, o3, lse3, [2])


@pytest.mark.parametrize("trees", [1, 31, 33, 1030])
def test_unpacked_pages_of_ragged_batches(api, trees):
    """Each page is found in the table of the trees: few and many of them, short ones beside a long one, some without nodes."""
    nodes = [0 if b % 7 == 3 else 4 + b % 5 for b in range(trees)] + [16]
    cache = Cache(api, [30 + 17 * (b % 9) for b in range(trees)] + [3000], "fp8", trees)
    m = torch.from_numpy(masks([tree(b, n) for b, n in enumerate(nodes)], 1)).cuda()
    q_abs, q_r = queries(sum(nodes), trees)
    plans = [api.mla_tree_plan(cache.n, nodes) for _ in range(2)]
    assert api.mla_tree_workspace_size(plans[0].info, True) > api.mla_tree_workspace_size(plans[0].info, False)
    o, lse, err = decode(api, cache, q_abs, q_r, m, plans[0])
    o2, lse2, err2 = decode(api, cache, q_abs, q_r, m, direct(api, plans[1]))
    assert api.mla_check(err) == 0 and api.mla_check(err2) == 0
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    check(cache, q_abs, q_r, m, o, lse, nodes, set(range(0, sum(nodes), max(1, sum(nodes) // 12))))


def test_a_captured_workspace_outlives_the_next(api):
    """A graph of the bf16 decode, then the same plan over an FP8 cache takes a larger workspace: the graph's stays."""
    n0, q = 3000, 20
    cache, eight = Cache(api, [n0 + q], "bf16", 31), Cache(api, [n0 + q], "fp8", 31)
    m = torch.from_numpy(masks([tree(0, q)], 1)).cuda()
    q_abs, q_r = queries(q, 31)
    plan = api.mla_tree_plan(cache.n, [q])
    plan.workspace = plan.workspace[:api.mla_tree_workspace_size(plan.info, False)].clone()   # none to spare
    want = decode(api, cache, q_abs, q_r, m, api.mla_tree_plan(cache.n, [q]))[0]
    wait = torch.cuda.Stream()
    o, err, graph = torch.zeros_like(want), word(), torch.cuda.CUDAGraph()
    lse = torch.zeros((q, 128), device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=wait):
        decode(api, cache, q_abs, q_r, m, plan, o=o, lse=lse, err=err)
        decode(api, cache, q_abs, q_r, m, plan, o=o, lse=lse, err=err, stream=wait)
    held = plan.workspace
    assert held.numel() > 0 and len(plan.captured) == 1 and plan.captured[0] is held
    e = decode(api, eight, q_abs, q_r, m, plan)[2]
    assert plan.workspace.data_ptr() != held.data_ptr() and plan.captured[0] is held
    graph.replay()
    torch.cuda.synchronize()
    assert int(e.item()) == 0 and int(err.item()) == 0 and torch.equal(o, want)
    with pytest.raises(TypeError):
        api.mla_tree_plan(cache.n, [q], into=api.mla_decode_plan(cache.n, [q]))


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("kind, n0, q", [("bf16", 200, 6), ("bf16", 3000, 100), ("fp8", 200, 6), ("fp8", 2000, 48)])
def test_inputs_written_just_before(api, kind, n0, q, captured):
    """The launch does not wait for the kernels before it, the kernel does: inputs written on the stream right before
    each call, by kernels and copies, on it and on another that it joins; the output taken right after."""
    cache = Cache(api, [n0 + q], kind, 61)
    m = torch.from_numpy(masks([tree(0, q)], 1 if q <= 64 else 2)).cuda()
    plan, rounds = api.mla_tree_plan(cache.n, [q]), 4
    qs = [queries(q, 62 + i) for i in range(rounds)]
    tables = [cache.table.clone() for _ in range(rounds)]
    for i in range(1, rounds):                               # the first pages in another order
        tables[i][0, :3] = tables[0][0, :3].roll(i)
    want = []
    for (a, r), t in zip(qs, tables):
        cache.table = t
        want.append(decode(api, cache, a, r, m, plan)[:2])
        torch.cuda.synchronize()
    cache.table = tables[0].clone()
    a, r, mm = (torch.zeros_like(x) for x in (*qs[0], m))
    o, lse, err = torch.empty_like(want[0][0]), torch.empty_like(want[0][1]), word()
    got = [(torch.zeros_like(o), torch.zeros_like(lse)) for _ in range(rounds)]
    busy = torch.randn((2048, 2048), device="cuda")
    main, other = torch.cuda.Stream(), torch.cuda.Stream()

    def work():
        for i in range(rounds):
            other.wait_stream(main)
            with torch.cuda.stream(other):
                busy.mul_(1.0)
                r.copy_(qs[i][1])
            torch.mul(m, 1, out=mm)
            cache.table.copy_(tables[i])
            busy.mul_(1.0)
            main.wait_stream(other)
            torch.mul(qs[i][0], 1, out=a)
            decode(api, cache, a, r, mm, plan, o=o, lse=lse, err=err)
            got[i][0].copy_(o)
            got[i][1].copy_(lse)
            a.zero_()

    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=main):
            work()
        for _ in range(3):
            graph.replay()
    else:
        with torch.cuda.stream(main):
            for _ in range(3):
                work()
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for (x, y), (wx, wy) in zip(got, want):
        assert torch.equal(x, wx) and torch.equal(y, wy)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_wider_masks_and_tables(api, kind):
    """Words that no tree needs, rows and columns of the table past the batch: the same bits, whatever they hold."""
    nodes = [20, 64, 3]
    cache = Cache(api, [300, 64, 1000], kind, 51)
    m = torch.from_numpy(masks([tree(b, n) for b, n in enumerate(nodes)], 1)).cuda()
    q_abs, q_r = queries(sum(nodes), 51)
    o, lse, err = decode(api, cache, q_abs, q_r, m, api.mla_tree_plan(cache.n, nodes))
    wide = torch.full((sum(nodes), 4), -1, dtype=torch.int64, device="cuda")
    wide[:, :1] = m
    table = torch.full((5, cache.table.shape[1] + 9), 1 << 30, dtype=torch.int32, device="cuda")
    table[:3, :cache.table.shape[1]] = cache.table
    cache.table = table
    o2, lse2, err2 = decode(api, cache, q_abs, q_r, wide, api.mla_tree_plan(cache.n, nodes))
    assert int(err.item()) == 0 and int(err2.item()) == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "nvfp4"])
def test_batches_without_nodes(api, kind):
    err, none = word(), torch.empty((0, 1), dtype=torch.int64, device="cuda")
    new = torch.zeros(2, dtype=torch.int32, device="cuda")
    raw = layered(kind, 2, 4, 2)
    want = [x.clone() for x in raw]
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    api.mla_tree_layout(i32([]), i32([0, 0, 0]), i32([70, 5]), none, err)
    call(api, "mla_tree_compact", kind, *views(kind, raw, 4), table, none, i32([0, 0, 0]), i32([70, 5]), i32([-1, -1]), new, err)
    assert int(err.item()) == 0 and new.tolist() == [70, 5]
    assert all(torch.equal(x, w) for x, w in zip(raw, want))
    if kind != "nvfp4":
        cache = Cache(api, [70, 5], kind, 52)
        q_abs, q_r = (torch.empty((0, 128, d), dtype=torch.bfloat16, device="cuda") for d in (512, 64))
        decode(api, cache, q_abs, q_r, none, api.mla_tree_plan([70, 5], [0, 0]), err=err)
        assert int(err.item()) == 0


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_longest_positions(api, kind):
    """2^31 - 1 tokens, all on one page but the last: its first node is NaN, which the second does not see."""
    n = 2 ** 31 - 1
    cache = Cache(api, [64, 64], kind, 41)
    table = torch.full((1, (n + 63) // 64), int(cache.bt[0, 0]), dtype=torch.int32, device="cuda")
    last = int(cache.bt[1, 0])
    table[0, -1] = last
    if kind == "bf16":
        cache.kv[last, 61] = float("nan")                    # position n - 2
    else:
        cache.rows[last, 61] = 0x7F
    m = torch.tensor([[1], [2]], dtype=torch.int64, device="cuda")
    plan = api.mla_tree_plan([n], [2])
    q_abs, q_r = queries(2, 41)
    cache.table = table
    o, lse, err = decode(api, cache, q_abs, q_r, m, plan)
    assert api.mla_check(err) == 0
    assert bool(torch.isnan(o[0]).all())
    assert bool(torch.isfinite(o[1]).all()) and bool(torch.isfinite(lse[1]).all())


def test_unpacked_decode_is_captured(api):
    """First use of a plan inside a capture, two graphs of one plan, replayed in turn after the cache has changed."""
    n0, q = 1200, 48
    caches = [Cache(api, [n0 + q], "fp8", s) for s in (21, 22)]
    m = torch.from_numpy(masks([tree(0, q)], 1)).cuda()
    q_abs, q_r = queries(q, 21)
    plan = api.mla_tree_plan(caches[0].n, [q])
    warm = api.mla_tree_plan(caches[0].n, [q])
    want = [decode(api, c, q_abs, q_r, m, warm)[0] for c in caches]
    rows, scales, table = caches[0].rows.clone(), caches[0].scales.clone(), caches[0].table.clone()
    live = Cache.__new__(Cache)
    live.kind, live.n, live.rows, live.scales, live.table = "fp8", caches[0].n, rows, scales, table
    outs, graphs, err = [torch.zeros_like(want[0]) for _ in range(2)], [], word()
    lse = torch.zeros((q, 128), dtype=torch.float32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for o in outs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            decode(api, live, q_abs, q_r, m, plan, o=o, lse=lse, err=err)
        graphs.append(graph)
    assert plan.workspace.numel() >= api.mla_tree_workspace_size(plan.info, True)
    for turn in (0, 1, 0):
        rows.copy_(caches[turn].rows)
        scales.copy_(caches[turn].scales)
        table.copy_(caches[turn].table)
        for o, graph in zip(outs, graphs):
            o.zero_()
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[turn]) and torch.equal(outs[1], want[turn]), turn
    assert int(err.item()) == 0


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_decodes_on_other_streams(api, kind):
    """One plan, uploaded on one stream, decoded on two others one after the other, dropped while queued."""
    cache = Cache(api, [700 + 40, 300 + 9], kind, 31)
    nodes = [40, 9]
    m = torch.from_numpy(masks([tree(b, n) for b, n in enumerate(nodes)], 1)).cuda()
    q_abs, q_r = queries(49, 31)
    want, want_lse, _ = decode(api, cache, q_abs, q_r, m, api.mla_tree_plan(cache.n, nodes))
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [(torch.zeros_like(want), torch.zeros_like(want_lse)) for _ in range(2)]
    err = word()
    torch.cuda.synchronize()
    plan = api.mla_tree_plan(cache.n, nodes, stream=a)
    decode(api, cache, q_abs, q_r, m, plan, stream=a, o=outs[0][0], lse=outs[0][1], err=err)
    b.wait_stream(a)
    with torch.cuda.stream(b):
        decode(api, cache, q_abs, q_r, m, plan, o=outs[1][0], lse=outs[1][1], err=err)
    del plan
    junk = [torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]  # blocks that are free again
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and len(junk) == 8
    for o, lse in outs:
        assert torch.equal(o, want) and torch.equal(lse, want_lse)


def test_two_plans_at_once(api):
    """Decodes of two plans in flight on two streams do not touch each other."""
    caches = [Cache(api, [900 + 24], "bf16", 41), Cache(api, [1500 + 40], "fp8", 42)]
    nodes = [24, 40]
    ms = [torch.from_numpy(masks([tree(5, n)], 1)).cuda() for n in nodes]
    qs = [queries(n, 50 + n) for n in nodes]
    want = [decode(api, c, *q, m, api.mla_tree_plan(c.n, [n])) for c, q, m, n in zip(caches, qs, ms, nodes)]
    streams = [torch.cuda.Stream() for _ in nodes]
    torch.cuda.synchronize()
    plans = [api.mla_tree_plan(c.n, [n], stream=s) for c, n, s in zip(caches, nodes, streams)]
    outs = [(torch.zeros_like(w[0]), torch.zeros_like(w[1]), word()) for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, q, m, p, s, (o, lse, err) in zip(caches, qs, ms, plans, streams, outs):
            decode(api, c, *q, m, p, stream=s, o=o, lse=lse, err=err)
    torch.cuda.synchronize()
    for w, (o, lse, err) in zip(want, outs):
        assert int(err.item()) == 0 and torch.equal(o, w[0]) and torch.equal(lse, w[1])


@pytest.mark.parametrize("unpack", [False, True])
def test_only_seen_scales_are_judged(api, unpack):
    n0, q = 1500, 64
    cache = Cache(api, [n0 + q], "fp8", 13)
    q_abs, q_r = queries(q, 13)
    full = masks([tree(0, q)], 1)
    free = full.copy()
    free[:, 0] &= ~(1 << 20)                                 # no row sees node 20
    plan = api.mla_tree_plan(cache.n, [q])
    assert api.mla_tree_workspace_size(plan.info, True) > api.mla_tree_workspace_size(plan.info, False)
    if not unpack:
        direct(api, plan)

    def word_after(position, scale, m):
        page, at = int(cache.bt[0, position // 64]), position % 64
        held = cache.scales[page, at].clone()
        cache.scales[page, at] = scale
        o, lse, err = decode(api, cache, q_abs, q_r, torch.from_numpy(m).cuda(), plan)
        cache.scales[page, at] = held
        return int(err.item())

    assert word_after(n0 + 20, 2.0 ** 20, free) == 0 and word_after(n0 + 20, float("nan"), free) == 0
    assert word_after(n0 + 20, 2.0 ** 20, full) == api.DEVERR_FP8_RANGE
    assert word_after(700, 2.0 ** -20, free) == api.DEVERR_FP8_RANGE
    assert word_after(n0 + 63, 2.0 ** 8, full) == api.DEVERR_FP8_RANGE
    o, lse, err = decode(api, cache, q_abs, q_r, torch.from_numpy(free).cuda(), plan)
    assert int(err.item()) == 0
    check(cache, q_abs, q_r, torch.from_numpy(free), o, lse, [q], {0, 19, 20, 21, 63})


@pytest.mark.parametrize("kind, unpack", [("bf16", False), ("fp8", False), ("fp8", True)])
def test_expired_wait_is_reported(api, kind, unpack):
    """A bound of 64 cycles makes waits run out: the word says so, and the next call on the same buffers is right."""
    cache = Cache(api, [1500 + 64], kind, 14)
    q_abs, q_r = queries(64, 14)
    m = torch.from_numpy(masks([tree(0, 64)], 1)).cuda()
    plan = api.mla_tree_plan(cache.n, [64])
    if kind == "fp8" and not unpack:
        direct(api, plan)
    o, lse, err = decode(api, cache, q_abs, q_r, m, plan)
    assert api.mla_check(err) == 0
    api.mla_debug_set_decode_wait_limit(64)
    try:
        late = decode(api, cache, q_abs, q_r, m, plan)[2]
        torch.cuda.synchronize()
    finally:
        api.mla_debug_set_decode_wait_limit(0)
    with pytest.raises(api.MlaError) as e:
        api.mla_check(late)
    assert e.value.status == 6
    again = decode(api, cache, q_abs, q_r, m, plan)
    assert api.mla_check(again[2]) == 0 and torch.equal(again[0], o) and torch.equal(again[1], lse)


def test_decode_tree_reports_bad_pages_and_refuses(api):
    cache = Cache(api, [200], "bf16", 1)
    q_abs, q_r = queries(3, 1)
    m = torch.from_numpy(masks([tree(0, 3)], 1)).cuda()
    plan = api.mla_tree_plan([200], [3])
    o, err = torch.zeros((3, 128, 512), dtype=torch.bfloat16, device="cuda"), word()
    kv = torch.zeros_like(cache.kv)
    table = cache.table.clone()
    table[0, 1] = 1000
    api.mla_decode_tree(q_abs, q_r, kv, table, m, plan, o, err)
    with pytest.raises(api.MlaError):
        api.mla_check(err)
    assert int(err.item()) == api.DEVERR_PAGE_OOB
    with pytest.raises(TypeError):
        api.mla_decode_tree(q_abs, q_r, kv, table, m, api.mla_decode_plan([200], [3]), o, err)
    with pytest.raises(ValueError):
        api.mla_decode_tree(q_abs[:2], q_r[:2], kv, table, m[:2], plan, o[:2], err)
    with pytest.raises(ValueError):
        api.mla_decode_tree(q_abs, q_r, kv, table, m[:2], plan, o, err)
    with pytest.raises(ValueError):
        api.mla_decode_tree(q_abs, q_r, kv, table[0], m, plan, o, err)
    with pytest.raises(TypeError):
        api.mla_decode_tree(q_abs, q_r, kv, table, m.to(torch.int32), plan, o, err)
    with pytest.raises(api.MlaError):                        # a tree of 70 nodes and masks of one word
        p70 = api.mla_tree_plan([200], [70])
        qa, qr = queries(70, 2)
        api.mla_decode_tree(qa, qr, kv, cache.table, torch.zeros((70, 1), dtype=torch.int64, device="cuda"), p70,
                            torch.zeros_like(qa), err)


# ------------------------------------------------------------------ caches of several layers
def layered(kind, layers, pages, seed, gap=0):
    """Caches with random bytes of every bit pattern; gap: pages between the layers that no call may touch."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    size = {"bf16": 1152, "fp8": 640, "nvfp4": 416}[kind]
    raw = torch.randint(0, 256, (layers, pages + gap, 64, size), generator=g, device="cuda", dtype=torch.uint8)
    out = [raw]
    if kind == "fp8":
        out.append(torch.randint(-2 ** 31, 2 ** 31, (layers, pages + gap, 64), generator=g, device="cuda",
                                 dtype=torch.int64).to(torch.int32))
    return out


def views(kind, raw, pages):
    """The tensors that the calls take, of the first `pages` pages of each layer."""
    if kind == "bf16":
        return [raw[0].view(torch.bfloat16)[:, :pages]]
    if kind == "fp8":
        return [raw[0][:, :pages], raw[1].view(torch.float32)[:, :pages]]
    return [raw[0][:, :pages]]


def call(api, name, kind, *args):
    return getattr(api, name + {"bf16": "", "fp8": "_fp8", "nvfp4": "_nvfp4"}[kind])(*args)


COMPACTS = [
    # tokens before the tree, nodes
    ([0], [1]),
    ([5, 60, 64, 127], [40, 64, 65, 256]),
    ([0, 63, 1, 300], [0, 10, 130, 33]),
]


@pytest.mark.parametrize("kind", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("layers, gap", [(1, 0), (3, 0), (2, 3)])
@pytest.mark.parametrize("case", range(len(COMPACTS)))
@pytest.mark.parametrize("which", ["last", "deep", "none", "dense"])
def test_compact(api, kind, layers, gap, case, which):
    ctx, nodes = COMPACTS[case]
    trees = [tree(b, n, 2, 3) for b, n in enumerate(nodes)]
    words = (max(nodes) + 63) // 64
    m = masks(trees, words)
    if which == "dense":                                     # any bits, many of them: sources that others move to
        rng = np.random.default_rng(case)
        m = np.array([words_of([k for k in range(n) if rng.random() < 0.8], words) for n in nodes for _ in range(n)], np.int64)
    acc = [n - 1 if which in ("last", "dense") else -1 if which == "none" or n == 0 else
           max(range(n), key=lambda i: len(path(t, i))) for n, t in zip(nodes, trees)]
    need = [(c + n + 63) // 64 for c, n in zip(ctx, nodes)]
    pages = sum(need) + 2
    perm = np.random.default_rng(case).permutation(pages)
    bt = np.full((len(ctx), max(max(need), 1)), -1, np.int32)
    for b, k in enumerate(need):
        bt[b, :k] = perm[sum(need[:b]):sum(need[:b]) + k]
    raw = layered(kind, layers, pages, case, gap)
    want = [x.cpu().clone() for x in raw]
    lens = []
    for b, (c, n) in enumerate(zip(ctx, nodes)):
        keep = kept(m[starts_of(nodes)[b] + acc[b]] if acc[b] >= 0 else [], acc[b])
        lens.append(c + len(keep))
        for k, i in enumerate(keep):                         # in order: no source is lost
            for x in want:
                x[:, bt[b, (c + k) // 64], (c + k) % 64] = x[:, bt[b, (c + i) // 64], (c + i) % 64].clone()
    new, err = torch.full((len(ctx) + 1,), -7, dtype=torch.int32, device="cuda"), word()
    call(api, "mla_tree_compact", kind, *views(kind, raw, pages), torch.from_numpy(bt).cuda(), torch.from_numpy(m.reshape(-1, words)).cuda(),
         i32(starts_of(nodes)), i32([c + n for c, n in zip(ctx, nodes)]), i32(acc), new[:-1], err)
    assert int(err.item()) == 0
    assert new.tolist() == lens + [-7]
    for x, w in zip(raw, want):
        assert torch.equal(x.cpu(), w)


def test_compact_judges_its_inputs(api):
    raw = layered("bf16", 2, 4, 0)
    want = raw[0].clone()
    kv = views("bf16", raw, 4)[0]
    nodes = [3, 3, 3, 3]
    m = torch.tensor([[1], [3], [5]] * 4, dtype=torch.int64, device="cuda")
    bt = torch.tensor([[0], [1], [4], [3]], dtype=torch.int32, device="cuda")
    new, err = torch.full((4,), -7, dtype=torch.int32, device="cuda"), word()
    api.mla_tree_compact(kv, bt, m, i32([0, 3, 6, 9, 12]), i32([3, 2, 10, 10]), i32([3, 2, 2, -2]), new, err)
    assert int(err.item()) == api.DEVERR_TREE | api.DEVERR_PAGE_OOB
    assert new.tolist() == [-7, -7, 9, -7] and torch.equal(raw[0], want)   # the third's page is not of the pool
    err.zero_()
    api.mla_tree_compact(kv, bt, m, i32([0, 3, 6, 9, 13]), i32([3, 3, 3, 3]), i32([2, -1, -1, 2]), new, err)
    assert int(err.item()) == api.DEVERR_TREE and new.tolist() == [2, 0, 0, -7]
    want[:, 0, 1] = want[:, 0, 2]
    assert torch.equal(raw[0], want)
    ok = (kv, bt, m, i32([0, 3, 6, 9, 12]), i32(nodes), i32([0] * 4), new, err)
    for at, bad, error in ((0, kv.transpose(1, 2), ValueError), (0, kv.float(), TypeError), (0, kv[0, 0], ValueError),
                           (1, bt[:3], ValueError), (2, m[:, 0], ValueError), (3, i32([0, 3]), ValueError),
                           (5, i32([0] * 3), ValueError), (6, ok[4], api.MlaError), (6, new.long(), TypeError)):
        args = list(ok)
        args[at] = bad
        with pytest.raises(error):
            api.mla_tree_compact(*args) if at != 6 or error is TypeError else api.mla_tree_compact(*args[:4], ok[4], *args[5:])
    with pytest.raises(ValueError):                          # every layer the same memory
        api.mla_tree_compact(kv.transpose(0, 1), *ok[1:])
    with pytest.raises(api.MlaError):
        api.mla_tree_compact(kv[:1].expand(2, 4, 64, 576), *ok[1:])


def test_compact_to_a_bad_page(api):
    """The kept row's page is good, the one that it would move to is not: nothing moves, and the word says so."""
    raw = layered("bf16", 2, 4, 1)
    want = raw[0].clone()
    m = torch.tensor([[1], [2]], dtype=torch.int64, device="cuda")
    bt = torch.tensor([[9, 1]], dtype=torch.int32, device="cuda")
    new, err = torch.full((1,), -7, dtype=torch.int32, device="cuda"), word()
    api.mla_tree_compact(views("bf16", raw, 4)[0], bt, m, i32([0, 2]), i32([65]), i32([1]), new, err)
    assert int(err.item()) == api.DEVERR_PAGE_OOB
    assert new.tolist() == [64] and torch.equal(raw[0], want)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("layers, gap, pages, pairs", [(1, 0, 2, 1), (3, 0, 50, 20), (2, 1, 200, 65), (1, 0, 30, 15)])
def test_copy_pages(api, kind, layers, gap, pages, pairs):
    rng = np.random.default_rng(pairs)
    ids = rng.permutation(pages).astype(np.int32)
    dst, src = ids[:pairs], rng.choice(ids[pairs:], pairs).astype(np.int32)
    raw = layered(kind, layers, pages, pairs, gap)
    want = [x.clone() for x in raw]
    for x in want:
        x[:, torch.from_numpy(dst).long().cuda()] = x[:, torch.from_numpy(src).long().cuda()]
    call(api, "mla_copy_pages", kind, *views(kind, raw, pages), src, dst)
    for x, w in zip(raw, want):
        assert torch.equal(x, w)
    one = [v[0] for v in views(kind, raw, pages)]            # a single layer's tensor
    call(api, "mla_copy_pages", kind, *one, list(map(int, dst[:1])), list(map(int, src[:1])))
    call(api, "mla_copy_pages", kind, *one, [], [])
    for x, w in zip(raw, want):
        w[0, int(src[0])] = w[0, int(dst[0])]
        assert torch.equal(x, w)


def test_copy_pages_of_more_than_a_launch(api):
    pages, n = 9000, 4001
    raw = torch.arange(pages, dtype=torch.int32, device="cuda").to(torch.uint8)[:, None, None].expand(pages, 64, 416).contiguous()
    raw[:, 0, :4] = torch.arange(pages, dtype=torch.int32, device="cuda").view(torch.uint8).view(pages, 4)
    src, dst = np.arange(4500, 4500 + n, dtype=np.int32), np.arange(n, dtype=np.int32)[::-1]
    want = raw.clone()
    want[torch.from_numpy(dst.copy()).long().cuda()] = raw[torch.from_numpy(src).long().cuda()]
    api.mla_copy_pages_nvfp4(raw, src, dst)
    assert torch.equal(raw, want)


@pytest.mark.parametrize("pairs", [3, 300])
def test_copies_and_compaction_are_captured(api, pairs):
    """A graph on a side stream, replayed after the caches, the accepted nodes and the lists of pages have changed."""
    kv = torch.randn((2, 2 * pairs + 2, 64, 576), device="cuda").to(torch.bfloat16)
    src, dst = np.arange(pairs, dtype=np.int32), np.arange(pairs, 2 * pairs, dtype=np.int32)
    t = tree(3, 9)
    m = torch.from_numpy(masks([t], 1)).cuda()
    table = torch.tensor([[2 * pairs, 2 * pairs + 1]], dtype=torch.int32, device="cuda")
    q, seq, acc, new, err = i32([0, 9]), i32([69]), i32([8]), i32([0]), word()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        api.mla_copy_pages(kv, src, dst)
        api.mla_tree_compact(kv, table, m, q, seq, acc, new, err)
    src[:], dst[:] = 0, 1                                    # they were read when the call was made
    for step in range(2):
        kv.normal_()
        last = 8 if step == 0 else 5
        acc.fill_(last)
        want = kv.clone()
        want[:, pairs:2 * pairs] = want[:, :pairs]
        keep = path(t, last)
        for r, k in enumerate(sorted(keep)):
            at, to = 60 + k, 60 + r
            want[:, 2 * pairs + to // 64, to % 64] = want[:, 2 * pairs + at // 64, at % 64].clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert int(err.item()) == 0 and new.tolist() == [60 + len(keep)] and torch.equal(kv, want)


def test_copy_pages_refusals(api):
    kv = torch.zeros((2, 8, 64, 576), dtype=torch.bfloat16, device="cuda")
    for src, dst, error in (([0, 1], [2, 2], api.MlaError), ([0, 1], [1, 2], api.MlaError), ([8], [0], api.MlaError),
                            ([0], [1, 2], ValueError), ([[0]], [[1]], ValueError), ([0.5], [1], ValueError),
                            ([2 ** 31], [1], (ValueError, OverflowError))):
        with pytest.raises(error):
            api.mla_copy_pages(kv, src, dst)
    rows, scales = torch.zeros((2, 8, 64, 640), dtype=torch.uint8, device="cuda"), torch.zeros((2, 8, 64), device="cuda")
    for r, s in ((rows, scales[0]), (rows, scales[:, :4]), (rows[0], scales), (rows[:, :4], scales[:, :4].half())):
        with pytest.raises((ValueError, TypeError)):
            api.mla_copy_pages_fp8(r, s, [0], [1])
    with pytest.raises(ValueError):
        api.mla_copy_pages(kv.cpu(), [0], [1])


# ------------------------------------------------------------------ together
def _verify(api, st):
    """One verification step over two layers: layout, appends, attention, compaction."""
    api.mla_tree_layout(st["parents"], st["q_starts"], st["seq_lens"], st["masks"], st["err"], positions=st["pos"],
                        slots=st["slots"], block_table=st["table"], num_pages=st["kv"].shape[1])
    for layer in range(2):
        api.mla_kv_append_rope(st["c"][layer], st["k"][layer], st["pos"], st["rope"], st["slots"], st["kv"][layer], st["err"])
        api.mla_rope_q(st["q_pe"], st["pos"], st["rope"], st["q_r"], st["err"])
        api.mla_decode_tree(st["q_abs"], st["q_r"], st["kv"][layer], st["table"], st["masks"], st["plan"], st["o"][layer],
                            st["err"])
    api.mla_tree_compact(st["kv"], st["table"], st["masks"], st["q_starts"], st["seq_lens"], st["accepted"], st["new_lens"],
                         st["err"])


@pytest.mark.parametrize("captured", [False, True])
def test_verification_step(api, captured):
    """Fork, draft, verify, keep: the next decode sees what a straight append of the accepted tokens gives."""
    rng = np.random.default_rng(3)
    pool = api.MlaPool(40)
    n0, nodes = 150, [20, 33]
    parent = pool.alloc(3)
    rows, src, dst = pool.fork(parent, n0, 2, max_pages=4)
    for b in range(2):
        rows[b, 3] = pool.alloc(1)[0]
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    kv = torch.randn((2, 40, 64, 576), generator=g, device="cuda").to(torch.bfloat16)
    api.mla_copy_pages(kv, src, dst)
    trees = [tree(b, n, 3, 5) for b, n in enumerate(nodes)]
    acc = [max(range(n), key=lambda i: len(path(t, i))) for n, t in zip(nodes, trees)]
    T = sum(nodes)
    rope = torch.empty((400, 32, 2), dtype=torch.float32, device="cuda")
    api.mla_rope_table(400, rope)
    q_abs, q_pe = queries(T, 4)
    st = dict(parents=i32([p for t in trees for p in t]), q_starts=i32(starts_of(nodes)), seq_lens=i32([n0 + n for n in nodes]),
              masks=torch.zeros((T, 1), dtype=torch.int64, device="cuda"), err=word(), pos=torch.zeros(T, dtype=torch.int32, device="cuda"),
              slots=torch.zeros(T, dtype=torch.int64, device="cuda"), table=torch.from_numpy(rows).cuda(), kv=kv, rope=rope,
              c=[to_bf16(bf16(rng, (T, 512)), "cuda") for _ in range(2)], k=[to_bf16(bf16(rng, (T, 64)), "cuda") for _ in range(2)],
              q_abs=q_abs, q_pe=q_pe, q_r=torch.zeros_like(q_pe), plan=api.mla_tree_plan([n0 + n for n in nodes], nodes),
              o=[torch.zeros((T, 128, 512), dtype=torch.bfloat16, device="cuda") for _ in range(2)], accepted=i32(acc),
              new_lens=torch.zeros(2, dtype=torch.int32, device="cuda"))
    want = kv.clone()
    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            _verify(api, st)                                 # warm-up: modules load outside the capture
            st["kv"].copy_(want)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                _verify(api, st)
        torch.cuda.current_stream().wait_stream(side)
        for _ in range(2):
            st["kv"].copy_(want)
            for x in (st["masks"], st["pos"], st["slots"], st["q_r"], *st["o"], st["new_lens"]):
                x.zero_()
            graph.replay()
    else:
        _verify(api, st)
    assert api.mla_check(st["err"]) == 0
    # the accepted tokens appended one after another
    paths = [path(t, a) for t, a in zip(trees, acc)]
    assert st["new_lens"].tolist() == [n0 + len(p) for p in paths]
    at = torch.tensor([starts_of(nodes)[b] + i for b, p in enumerate(paths) for i in p], device="cuda")
    seq = np.array([b for b, p in enumerate(paths) for _ in p], np.int32)
    pos = np.array([n0 + k for p in paths for k in range(len(p))], np.int32)
    slots = torch.from_numpy(api.mla_slot_mapping(rows, seq, pos)).cuda()
    for layer in range(2):
        api.mla_kv_append_rope(st["c"][layer][at], st["k"][layer][at], torch.from_numpy(pos).cuda(), rope, slots, want[layer], st["err"])
        for b, p in enumerate(paths):
            for j in range(n0 + len(p)):
                pg = int(rows[b, j // 64])
                if j >= n0 - 3 or j % 50 == 0:
                    assert torch.equal(st["kv"][layer, pg, j % 64], want[layer, pg, j % 64]), (layer, b, j)
        # each accepted node's output is the causal decode's of the straight sequence
        lens, m = [n0 + len(p) for p in paths], [len(p) for p in paths]
        o2 = torch.zeros((sum(m), 128, 512), dtype=torch.bfloat16, device="cuda")
        api.mla_decode_paged(q_abs[at], st["q_r"][at], want[layer], st["table"], api.mla_decode_plan(lens, m), o2, st["err"])
        assert api.mla_check(st["err"]) == 0
        r = 0
        for b, p in enumerate(paths):
            pages = torch.from_numpy(rows[b].copy()).long().cuda()
            for k in range(len(p)):                          # both are within the rounding of the same exact value
                j = torch.arange(n0 + k + 1, device="cuda")
                x = want[layer][pages[j // 64], j % 64].double()
                tol = decode_row(q_abs[at[r]].double(), st["q_r"][at[r]].double(), x[:, :512], x[:, 512:])[2]
                d = (st["o"][layer][at[r]].double() - o2[r].double()).abs()
                assert bool((d <= 2 * tol).all()), (layer, b, k)
                r += 1
    # the rest of the pool is untouched
    used = {int(x) for r in rows for x in r if x >= 0}
    rest = [p for p in range(40) if p not in used]
    assert torch.equal(st["kv"][:, rest], want[:, rest])


def test_pool_moves_with_its_sequences(api):
    """A pool brought together: copies, remapped tables, the same attention."""
    pool = api.MlaPool(30)
    rows = np.stack([pool.alloc(5) for _ in range(4)]).astype(np.int32)
    pool.free(rows[0])
    pool.free(rows[2])
    rows = rows[[1, 3]]
    kv = torch.randn((3, 30, 64, 576), device="cuda").to(torch.bfloat16)
    q_abs, q_r = queries(6, 9)
    nodes, seq = [3, 3], [300, 257]
    m = torch.from_numpy(masks([tree(b, 3) for b in range(2)], 1)).cuda()
    plan = api.mla_tree_plan(seq, nodes)
    o, p = [torch.zeros((6, 128, 512), dtype=torch.bfloat16, device="cuda") for _ in range(2)], word()
    api.mla_decode_tree(q_abs, q_r, kv[2], torch.from_numpy(rows).cuda(), m, plan, o[0], p)
    src, dst = pool.compact(100)
    assert len(src) == 10 - len([x for x in rows.reshape(-1) if x < 10])
    api.mla_copy_pages(kv, src, dst)
    new = api.mla_remap_pages(rows, src, dst)
    assert sorted(new.reshape(-1).tolist()) == list(range(10))
    api.mla_decode_tree(q_abs, q_r, kv[2], torch.from_numpy(new).cuda(), m, plan, o[1], p)
    assert api.mla_check(p) == 0 and torch.equal(o[0], o[1])
    pool.free(new[0])
    pool.free(new[1])
    assert pool.available() == 30
