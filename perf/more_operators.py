"""Cases and plain forms of the operators that verify a tree of drafted tokens.

A draft model proposes a tree of tokens after each sequence; all of its nodes
are appended to the paged latent cache and verified in one decode step, each
node seeing the sequence and its own ancestors.  Then the accepted path stays
and the other nodes go; sequences fork, share pages and move.  Four operators:

* ``layout``: a batch of trees, given as parents, turned into the nodes' masks
  (a bit for each ancestor), positions and cache slots;
* ``tree``: absorbed decode attention over the paged latent cache (bf16 or 8
  bits) in which a node sees the tokens before the tree and the nodes of its mask;
* ``compact``: in every layer's cache, the accepted path's rows moved to the
  places right after the sequence;
* ``copy``: pages copied in every layer's cache (a fork's last page, or the
  moves that bring a pool's used pages together).

``run`` computes them either with elementary torch operations (``own`` false)
or with this package's kernels (``own`` true).
"""
import math
import random

import numpy as np
import torch

own = False

H, D_C, D_R, PAGE = 128, 512, 64, 64
D_QK = D_C + D_R
SCALE = 1.0 / math.sqrt(128 + D_R)
DEV = "cuda"
TOKEN_BYTES = {"bf16": 1152, "fp8": 644, "nvfp4": 416}   # the FP8 cache has a scale beside each row


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one user, a small tree: the latency of a step
        {"name": "tree_b1_n8_1k", "op": "tree", "cache": "bf16", "batch": 1, "lo": 1024, "hi": 1024, "n_lo": 8, "n_hi": 8, "roots": 3},
        # a ragged batch of short conversations, trees of different sizes
        {"name": "tree_b16_n16_ragged", "op": "tree", "cache": "bf16", "batch": 16, "lo": 1024, "hi": 4096, "n_lo": 8, "n_hi": 24, "roots": 4},
        # one user with a long context in 8 bits and a large tree
        {"name": "tree_fp8_b1_n64_32k", "op": "tree", "cache": "fp8", "batch": 1, "lo": 32768, "hi": 32768, "n_lo": 64, "n_hi": 64, "roots": 8},
        # a large batch, the nodes of a short tree
        {"name": "tree_b64_n12_8k", "op": "tree", "cache": "bf16", "batch": 64, "lo": 8192, "hi": 8192, "n_lo": 12, "n_hi": 12, "roots": 4},
        # one user: the trees of a step before its layers run
        {"name": "layout_b1_n64", "op": "layout", "batch": 1, "lo": 1024, "hi": 1024, "n_lo": 64, "n_hi": 64, "roots": 8},
        # a large batch of the largest trees
        {"name": "layout_b256_n256", "op": "layout", "batch": 256, "lo": 100, "hi": 8192, "n_lo": 200, "n_hi": 256, "roots": 8},
        # one user, one model layer at a time
        {"name": "compact_b1_l1", "op": "compact", "cache": "bf16", "layers": 1, "batch": 1, "n_lo": 32, "n_hi": 32, "roots": 8, "accept": 5},
        # a ragged batch in 8 bits over all layers of a model
        {"name": "compact_fp8_b16_l60", "op": "compact", "cache": "fp8", "layers": 60, "batch": 16, "n_lo": 20, "n_hi": 64, "roots": 8, "accept": 6},
        # a large batch over all layers
        {"name": "compact_b64_l60", "op": "compact", "cache": "bf16", "layers": 60, "batch": 64, "n_lo": 32, "n_hi": 32, "roots": 10, "accept": 8},
        # one sequence forks: its last, partly filled page in every layer
        {"name": "copy_fork_b1_l60", "op": "copy", "cache": "bf16", "layers": 60, "pages": 16, "pairs": 1, "spread": "fork"},
        # sixteen sequences into four beams each, 8 bits
        {"name": "copy_fork_fp8_b48_l60", "op": "copy", "cache": "fp8", "layers": 60, "pages": 200, "pairs": 48, "spread": "fork"},
        # a pool brought together: two thousand pages a layer move down
        {"name": "copy_moves_l4", "op": "copy", "cache": "bf16", "layers": 4, "pages": 6000, "pairs": 2000, "spread": "moves"},
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "layout", "compact", "copy"])
    if op == "tree":
        n_hi = _spread(rng, 1, 256 if rng.random() < 0.3 else 64)
        n_lo = _spread(rng, max(1, n_hi // 4), n_hi)
        batch = _spread(rng, 1, max(1, min(64, 768 // n_hi)))
        lo = _spread(rng, 1, 16384) - 1
        hi = min(32768, _spread(rng, max(lo, 1), 4 * max(lo, 1)))
        while batch * n_hi * hi > 64 * 12 * 8192:            # the largest listed case's work
            hi //= 2
        return {"op": op, "cache": rng.choice(["bf16", "fp8"]), "batch": batch, "lo": min(lo, hi), "hi": hi, "n_lo": n_lo,
                "n_hi": n_hi, "roots": rng.randint(1, 10)}
    n_hi = _spread(rng, 1, 256)
    n_lo = _spread(rng, max(1, n_hi // 4), n_hi)
    if op == "layout":
        lo = _spread(rng, 1, 8192) - 1
        return {"op": op, "batch": _spread(rng, 1, 256), "lo": lo, "hi": _spread(rng, max(lo, 1), 8192), "n_lo": n_lo, "n_hi": n_hi,
                "roots": rng.randint(1, 10)}
    cache = rng.choice(["bf16", "fp8", "nvfp4"])
    if op == "compact":
        batch = _spread(rng, 1, 64)
        return {"op": op, "cache": cache, "layers": _spread(rng, 1, max(1, min(61, 3840 // batch))), "batch": batch, "n_lo": n_lo,
                "n_hi": n_hi, "roots": rng.randint(2, 12), "accept": rng.randint(1, 8)}
    layers = _spread(rng, 1, 61)
    pages = _spread(rng, 4, max(4, 12000 // layers))
    return {"op": op, "cache": cache, "layers": layers, "pages": pages, "pairs": _spread(rng, 1, max(1, pages // 3)),
            "spread": rng.choice(["fork", "moves"])}


def _lens(lo, hi, n):
    """n lengths spread over [lo, hi] in no order of size."""
    return [lo + int((hi - lo) * ((i * 0.6180339887498949 + 0.5) % 1.0) + 0.5) for i in range(n)]


def _tree(r, n, roots):
    """Parents of n nodes: the first `roots` follow the sequence, the others
    hang below one of the last few, as a draft grown level by level has them."""
    return [-1 if i < roots else r.randrange(max(0, i - 2 * roots), i) for i in range(n)]


def _path(parents, i):
    """The nodes from a root to node i."""
    p = []
    while i >= 0:
        p.append(i)
        i = parents[i]
    return p[::-1]


def _trees(case, seed=0):
    """(nodes, parents) of each sequence.  The trees of attention and
    compaction are the case's own, so that its work is known from the case."""
    r = random.Random(7919 * case["roots"] + 31 * case["n_hi"] + case["n_lo"] + (seed << 20))
    nodes = _lens(case["n_lo"], case["n_hi"], case["batch"])
    return nodes, [_tree(r, n, case["roots"]) for n in nodes]


def _ctx(case):
    """Tokens before the tree, for each sequence."""
    if case["op"] != "compact":
        return _lens(case["lo"], case["hi"], case["batch"])
    return _lens(0, PAGE - 1, case["batch"])                 # the pages before the tree's are not touched


def _accepted(parents, most):
    """The node with the longest path of at most `most` nodes of which none
    lies at a place that another one moves to (so that a pass can be repeated)."""
    best, length = -1, 0
    for i in range(len(parents)):
        p = _path(parents, i)
        if length < len(p) <= most and all(x == k or x >= len(p) for k, x in enumerate(p)):
            best, length = i, len(p)
    return best


def work(case):
    op = case["op"]
    if op == "copy":
        n = case["pairs"] * case["layers"] * PAGE * TOKEN_BYTES[case["cache"]]
        read = len({s for s, _ in _pairs(case, 0)}) * case["layers"] * PAGE * TOKEN_BYTES[case["cache"]]
        return {"bytes": n + read, "flops": 0}
    nodes, trees = _trees(case)
    T, words = sum(nodes), (max(nodes) + 63) // 64
    if op == "layout":
        # parents, offsets, lengths and table entries in; masks, positions and slots out
        pages = sum((c % PAGE + n - 1) // PAGE + 1 for c, n in zip(_ctx(case), nodes))
        return {"bytes": T * (4 + 8 * words + 4 + 8) + case["batch"] * 8 + 4 * pages, "flops": 0}
    if op == "compact":
        moved = 0
        for t in trees:
            a = _accepted(t, case["accept"])
            moved += sum(x != k for k, x in enumerate(_path(t, a)))
        return {"bytes": 2 * moved * case["layers"] * TOKEN_BYTES[case["cache"]] + case["batch"] * (8 * words + 16), "flops": 0}
    ctx = _ctx(case)
    token = TOKEN_BYTES[case["cache"]]
    pairs = sum(c * n + sum(len(_path(t, i)) for i in range(n)) for c, n, t in zip(ctx, nodes, trees))
    return {"bytes": (sum(ctx) + T) * token + T * H * (D_QK + D_C) * 2 + T * 8 * words, "flops": pairs * H * 2 * (D_QK + D_C)}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, std=1.0):
    """bf16 normal values, drawn a piece at a time."""
    n = math.prod(shape)
    out = torch.empty(n, dtype=torch.bfloat16, device=DEV)
    step = 1 << 28
    for i in range(0, n, step):
        m = min(step, n - i)
        out[i:i + m] = torch.randn(m, generator=g, device=DEV, dtype=torch.float32) * std
    return out.view(shape)


def _quantise(c):
    """E4M3 codes of latents [..., 512] and the power-of-two scale of each row."""
    amax = c.float().abs().amax(dim=-1)
    m, e = torch.frexp(amax / 448.0)                        # the smallest k with amax <= 448 * 2^k
    k = torch.where(m == 0.5, e - 1, e)
    k = torch.where(amax == 0, torch.zeros_like(k), k)
    codes = torch.ldexp(c.float(), -k.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return codes, torch.ldexp(torch.ones_like(amax), k)


def _cache(g, kind, lead):
    """A cache of `lead` = (pages,) or (layers, pages)."""
    if kind == "bf16":
        return {"kv": _normal(g, (*lead, PAGE, D_QK))}
    if kind == "nvfp4":
        rows = torch.randint(0, 256, (math.prod(lead), PAGE, 416), generator=g, device=DEV, dtype=torch.uint8)
        rows[..., 288:] = _normal(g, (math.prod(lead), PAGE, D_R)).view(torch.uint8)
        return {"rows": rows.view(*lead, PAGE, 416)}
    n = math.prod(lead)
    rows = torch.empty((n, PAGE, 640), dtype=torch.uint8, device=DEV)
    scales = torch.empty((n, PAGE), dtype=torch.float32, device=DEV)
    for i in range(0, n, 4096):
        c = _normal(g, (min(4096, n - i), PAGE, D_QK))
        codes, sc = _quantise(c[..., :D_C])
        rows[i:i + 4096, :, :D_C] = codes.view(torch.uint8)
        rows[i:i + 4096, :, D_C:] = c[..., D_C:].contiguous().view(torch.uint8)
        scales[i:i + 4096] = sc
    return {"rows": rows.view(*lead, PAGE, 640), "scales": scales.view(*lead, PAGE)}


def _table(seq, seed, from_page=None, spare=0):
    """A block table that hands out a random permutation of the pool, which
    holds `spare` pages more; with from_page the pages before it are of no
    interest and stay -1."""
    r = random.Random(seed)
    first = from_page or [0] * len(seq)
    held = [(n + PAGE - 1) // PAGE for n in seq]
    perm = list(range(sum(h - f for h, f in zip(held, first)) + spare))
    r.shuffle(perm)
    bt = torch.full((len(seq), max(held)), -1, dtype=torch.int32)
    k = 0
    for b, (h, f) in enumerate(zip(held, first)):
        bt[b, f:h] = torch.tensor(perm[k:k + h - f], dtype=torch.int32)
        k += h - f
    return bt.to(DEV), max(k + spare, 1)


def _words(trees, words):
    """Masks int64 [nodes, words]: a bit for each node of a node's path."""
    out = []
    for t in trees:
        m = []
        for i, p in enumerate(t):
            m.append((m[p] if p >= 0 else 0) | 1 << i)
        for x in m:
            for w in range(words):
                v = x >> (64 * w) & (1 << 64) - 1
                out.append(v - (1 << 64) if v >> 63 else v)
    return torch.tensor(out, dtype=torch.int64).view(-1, words).to(DEV)


def _pairs(case, seed):
    """Page copies (source, destination) of a case: forks may share a source,
    moves bring the highest used pages to the lowest free ones."""
    r = random.Random(seed + 1)
    ids = list(range(case["pages"]))
    n = case["pairs"]
    if case["spread"] == "moves":
        free = sorted(r.sample(ids[:len(ids) // 2], min(n, len(ids) // 2)))
        used = [i for i in ids[len(ids) // 2:]]
        return list(zip(used[::-1][:len(free)], free))
    r.shuffle(ids)
    src = ids[n:n + max(1, n // 3)]
    return [(src[i % len(src)], ids[i]) for i in range(n)]


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"op": op, "case": dict(case), "err": torch.zeros(1, dtype=torch.int32, device=DEV)}
    if op == "copy":
        st |= _cache(g, case["cache"], (case["layers"], case["pages"]))
        p = _pairs(case, seed)
        st["src"], st["dst"] = (np.array(x, dtype=np.int32) for x in zip(*p))
        st["src_dev"], st["dst_dev"] = (torch.from_numpy(x).long().to(DEV) for x in (st["src"], st["dst"]))
        return st
    nodes, trees = _trees(case, seed if op == "layout" else 0)
    ctx = _ctx(case)
    seq = [c + n for c, n in zip(ctx, nodes)]
    T, words = sum(nodes), (max(nodes) + 63) // 64
    starts = [sum(nodes[:i]) for i in range(len(nodes) + 1)]
    st["nodes"], st["seq"], st["starts"] = nodes, seq, starts
    st["q_starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
    st["seq_lens"] = torch.tensor(seq, dtype=torch.int32, device=DEV)
    if op == "layout":
        st["bt"], st["pages"] = _table(seq, seed, [c // PAGE for c in ctx], spare=4096)
        st["parents"] = torch.tensor([p for t in trees for p in t], dtype=torch.int32, device=DEV)
        st["masks"] = torch.zeros((T, words), dtype=torch.int64, device=DEV)
        st["positions"] = torch.zeros(T, dtype=torch.int32, device=DEV)
        st["slots"] = torch.zeros(T, dtype=torch.int64, device=DEV)
        return st
    st["masks"] = _words(trees, words)
    if op == "compact":
        st["bt"], pages = _table(seq, seed)
        st |= _cache(g, case["cache"], (case["layers"], pages))
        st["accepted"] = torch.tensor([_accepted(t, case["accept"]) for t in trees], dtype=torch.int32, device=DEV)
        st["new_lens"] = torch.zeros(len(seq), dtype=torch.int32, device=DEV)
        st["most"] = case["accept"]
        return st
    st["bt"], pages = _table(seq, seed)
    st |= _cache(g, case["cache"], (pages,))
    st["q_abs"] = _normal(g, (T, H, D_C), 0.5)
    st["q_r"] = _normal(g, (T, H, D_R))
    st["out"] = torch.zeros((T, H, D_C), dtype=torch.bfloat16, device=DEV)
    if own:                                                 # the step's plan, shared by a model's layers
        from mla_latent_kv_02_gb300 import api
        st["plan"] = api.mla_tree_plan(seq, nodes)
    return st


# ------------------------------------------------------------------ plain forms
def _rows(st, slots):
    """Cached rows [..., 576] of the given slots, in 32 bits."""
    if "kv" in st:
        return st["kv"].view(-1, D_QK)[slots].float()
    r = st["rows"].view(-1, 640)[slots]
    lat = r[..., :D_C].contiguous().view(torch.float8_e4m3fn).float() * st["scales"].view(-1)[slots].unsqueeze(-1)
    return torch.cat([lat, r[..., D_C:].contiguous().view(torch.bfloat16).float()], dim=-1)


def _slots(bt, b, pos):
    return bt[b, pos // PAGE].long() * PAGE + pos % PAGE


def _bits(masks):
    """Masks [n, words] as truth values [n, 64 words]."""
    return ((masks[:, :, None] >> torch.arange(64, device=DEV)) & 1).bool().flatten(1)


def _plain_tree(st):
    out = torch.empty_like(st["out"])
    bits = _bits(st["masks"])
    for b, (n, m) in enumerate(zip(st["seq"], st["nodes"])):
        t0 = st["starts"][b]
        kv = _rows(st, _slots(st["bt"], b, torch.arange(n, device=DEV)))
        step = max(1, (1 << 29) // (H * n))                 # score rows at a time
        for i in range(0, m, step):
            t = slice(t0 + i, t0 + min(m, i + step))
            q = torch.cat([st["q_abs"][t], st["q_r"][t]], dim=-1).float()
            x = torch.matmul(q, kv.T) * SCALE
            x[:, :, n - m:].masked_fill_(~bits[t, None, :m], -math.inf)
            p = torch.exp(x - x.amax(dim=-1, keepdim=True))
            out[t] = (torch.matmul(p, kv[:, :D_C]) / p.sum(dim=-1, keepdim=True)).to(torch.bfloat16)
    return out


def _plain_layout(st):
    B, T, words = len(st["seq"]), sum(st["nodes"]), st["masks"].shape[1]
    q0 = st["q_starts"].long()
    n = q0[1:] - q0[:-1]
    b = torch.repeat_interleave(torch.arange(B, device=DEV), n, output_size=T)
    own_at = torch.arange(T, device=DEV)
    i = own_at - q0[b]
    par = st["parents"].long()
    at = torch.where(par >= 0, q0[b] + par, torch.full_like(par, T))   # row T: above the roots
    at = torch.cat([at, at.new_tensor([T])])
    depth = torch.cat([torch.ones_like(par), par.new_zeros(1)])
    word = torch.arange(words, device=DEV)
    mask = torch.where(word == (i // 64)[:, None], torch.ones_like(i)[:, None] << (i % 64)[:, None], torch.zeros_like(i)[:, None])
    mask = torch.cat([mask, mask.new_zeros(1, words)])
    for _ in range(8):                                      # twice as far up in each round: 256 nodes at most
        mask = mask | mask[at]
        depth = depth + depth[at]
        at = at[at]
    st["masks"].copy_(mask[:T])
    ctx = st["seq_lens"].long() - n
    st["positions"].copy_(ctx[b] + depth[:T] - 1)
    st["slots"].copy_(_slots(st["bt"], b, ctx[b] + i))


def _plain_compact(st):
    q0 = st["q_starts"].long()
    n = q0[1:] - q0[:-1]
    ctx = st["seq_lens"].long() - n
    acc = st["accepted"].long()
    M = max(st["nodes"])
    bits = _bits(st["masks"][(q0[:-1] + acc.clamp(min=0))])[:, :M] & (acc >= 0)[:, None]
    bits &= torch.arange(M, device=DEV) <= acc[:, None]
    kept = bits.sum(dim=1)
    st["new_lens"].copy_(ctx + kept)
    # the kept nodes in order, `most` places for each sequence
    order = torch.sort(torch.where(bits, torch.arange(M, device=DEV), M), dim=1).values[:, :st["most"]]
    k = torch.arange(order.shape[1], device=DEV)
    order = torch.where(k < kept[:, None], order, k)        # the rest stays where it is
    order = torch.minimum(order, n[:, None] - 1)
    k = torch.minimum(k, n[:, None] - 1)
    b = torch.arange(len(st["seq"]), device=DEV)[:, None]
    src = _slots(st["bt"], b, ctx[:, None] + order).flatten()
    dst = _slots(st["bt"], b, ctx[:, None] + k).flatten()
    for x in _stores(st):
        v = x.view(x.shape[0], -1, *x.shape[3:])            # [layers, slots, ...]
        v[:, dst] = v[:, src]


def _stores(st):
    return [st[k] for k in ("kv", "rows", "scales") if k in st]


def _held(st):
    """A cache as the values that it stands for (4-bit rows as bytes)."""
    if "kv" in st:
        return {"kv": st["kv"]}
    if "scales" not in st:
        return {"rows": st["rows"]}
    return {"codes": st["rows"][..., :D_C].view(torch.float8_e4m3fn), "scales": st["scales"],
            "k_r": st["rows"][..., D_C:].view(torch.bfloat16)}


def run(st):
    op = st["op"]
    if own:
        from mla_latent_kv_02_gb300 import api
    if op == "tree":
        if not own:
            return _plain_tree(st)
        if "kv" in st:
            api.mla_decode_tree(st["q_abs"], st["q_r"], st["kv"], st["bt"], st["masks"], st["plan"], st["out"], st["err"],
                                scale=SCALE)
        else:
            api.mla_decode_tree_fp8(st["q_abs"], st["q_r"], st["rows"], st["scales"], st["bt"], st["masks"], st["plan"],
                                    st["out"], st["err"], scale=SCALE)
        return st["out"]
    if op == "layout":
        if own:
            api.mla_tree_layout(st["parents"], st["q_starts"], st["seq_lens"], st["masks"], st["err"], positions=st["positions"],
                                slots=st["slots"], block_table=st["bt"], num_pages=st["pages"])
        else:
            _plain_layout(st)
        return {"masks": st["masks"], "positions": st["positions"], "slots": st["slots"]}
    if op == "compact":
        rest = (st["bt"], st["masks"], st["q_starts"], st["seq_lens"], st["accepted"], st["new_lens"], st["err"])
        if not own:
            _plain_compact(st)
        elif "kv" in st:
            api.mla_tree_compact(st["kv"], *rest)
        elif "scales" in st:
            api.mla_tree_compact_fp8(st["rows"], st["scales"], *rest)
        else:
            api.mla_tree_compact_nvfp4(st["rows"], *rest)
        return {"new_lens": st["new_lens"], **_held(st)}
    if not own:
        for x in _stores(st):
            x[:, st["dst_dev"]] = x[:, st["src_dev"]]
    elif "kv" in st:
        api.mla_copy_pages(st["kv"], st["src"], st["dst"])
    elif "scales" in st:
        api.mla_copy_pages_fp8(st["rows"], st["scales"], st["src"], st["dst"])
    else:
        api.mla_copy_pages_nvfp4(st["rows"], st["src"], st["dst"])
    return _held(st)


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "tree":
        return None if work(case)["flops"] > 8e12 else _exact_tree(st)
    if op == "layout":
        return _exact_layout(st)
    bt = st["bt"].tolist() if op == "compact" else None
    if op == "copy":
        for s, d in zip(st["src"].tolist(), st["dst"].tolist()):
            for x in _stores(st):
                x[:, d].copy_(x[:, s])
        return _exact_held(st)
    lens = []
    for b, (n, m) in enumerate(zip(st["seq"], st["nodes"])):
        a = int(st["accepted"][b])
        word = [int(w) for w in st["masks"][st["starts"][b] + a]] if a >= 0 else []
        path = [i for i in range(a + 1) if word[i // 64] >> (i % 64) & 1]
        lens.append(n - m + len(path))
        for k, i in enumerate(path):
            s, d = n - m + i, n - m + k
            for x in _stores(st):
                x[:, bt[b][d // PAGE], d % PAGE].copy_(x[:, bt[b][s // PAGE], s % PAGE].clone())
    return {"new_lens": torch.tensor(lens, dtype=torch.int32, device=DEV), **_exact_held(st)}


def _exact_held(st):
    h = _held(st)
    return {k: v if v.dtype == torch.uint8 else v.double() for k, v in h.items()}


def _exact_layout(st):
    masks, positions, slots = [], [], []
    par, bt = st["parents"].tolist(), st["bt"].tolist()
    words = st["masks"].shape[1]
    for b, (n, m) in enumerate(zip(st["seq"], st["nodes"])):
        t = par[st["starts"][b]:st["starts"][b] + m]
        for i in range(m):
            p = _path(t, i)
            for w in range(words):
                v = sum(1 << (x % 64) for x in p if x // 64 == w)
                masks.append(v - (1 << 64) if v >> 63 else v)
            positions.append(n - m + len(p) - 1)
            s = n - m + i
            slots.append(bt[b][s // PAGE] * PAGE + s % PAGE)
    return {"masks": torch.tensor(masks, dtype=torch.int64, device=DEV).view(-1, words),
            "positions": torch.tensor(positions, dtype=torch.int32, device=DEV),
            "slots": torch.tensor(slots, dtype=torch.int64, device=DEV)}


def _exact_tree(st):
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
    masks = st["masks"].tolist()
    for b, (n, m) in enumerate(zip(st["seq"], st["nodes"])):
        at = torch.arange(n, device=DEV)
        pages, off = st["bt"][b].long()[at // PAGE], at % PAGE
        if "kv" in st:
            r = st["kv"][pages, off].double()
            lat, rope = r[:, :D_C], r[:, D_C:]
        else:
            r = st["rows"][pages, off]
            c = r[:, :D_C].int()
            e, f = (c >> 3) & 15, (c & 7).double()
            v = torch.where(e > 0, (8 + f) * torch.exp2(e.double() - 10), f * 2.0 ** -9)
            lat = torch.where(c >= 128, -v, v) * st["scales"][pages, off].double()[:, None]
            rope = r[:, D_C:].contiguous().view(torch.bfloat16).double()
        for i in range(m):
            t = st["starts"][b] + i
            path = [k for k in range(i + 1) if masks[t][k // 64] >> (k % 64) & 1]
            j = torch.cat([torch.arange(n - m, device=DEV), torch.tensor([n - m + k for k in path], device=DEV)])
            s = (st["q_abs"][t].double() @ lat[j].T + st["q_r"][t].double() @ rope[j].T) * SCALE
            out[t] = torch.softmax(s, dim=-1) @ lat[j]
    return out
