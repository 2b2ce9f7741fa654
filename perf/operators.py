"""Cases and plain forms of the bounded-memory serving operators.

A long-running sequence is served with a bounded share of the GPU's memory:
its latent cache is held in 8 bits, its attention sees a sliding window and
the first few tokens (the sinks), and the per-head projection weights are
held in 4 bits.  Four operators make up such a step:

* ``append``: the new tokens' latents quantised to E4M3 with one power-of-two
  scale each, their RoPE keys and queries rotated on the way;
* ``window``: absorbed decode attention over the paged latent cache (bf16 or
  8 bits) with a window and sinks;
* ``chunk``: the same attention for long query chunks, through the expanded
  per-head keys and values;
* ``absorb_w4`` / ``up_w4``: the per-head projections W_UK and W_UV with 4-bit
  weights and one bf16 scale per group of the contraction.

``run`` computes them either with elementary torch operations in 32 bits
(``own`` false) or with this package's kernels (``own`` true).
"""
import math

import torch

own = False

H, D_HC, D_C, D_R, PAGE = 128, 128, 512, 64, 64
D_QK = D_C + D_R
SCALE = 1.0 / math.sqrt(D_HC + D_R)
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 64 sequences with a two-token draft: 128 new tokens and their queries
        {"name": "append_mtp2_b64", "op": "append", "batch": 64, "new": 2, "ctx": 8192, "queries": True},
        # the context fill of a 64K prompt in 16 sequences: keys only
        {"name": "append_fill_b16_64k", "op": "append", "batch": 16, "new": 65536, "ctx": 0, "queries": False},
        # one sequence, one token: the latency of a single user
        {"name": "window_b1_ctx1k", "op": "window", "cache": "bf16", "batch": 1, "q_len": 1, "lo": 1024, "hi": 1024,
         "window": 512, "sinks": 4},
        # a ragged batch of short conversations over the 8-bit cache
        {"name": "window_fp8_b16_ragged", "op": "window", "cache": "fp8", "batch": 16, "q_len": 1, "lo": 1024,
         "hi": 4096, "window": 1000, "sinks": 4},
        # two-token drafts at a large batch
        {"name": "window_mtp2_b64_8k", "op": "window", "cache": "bf16", "batch": 64, "q_len": 2, "lo": 8194,
         "hi": 8194, "window": 2048, "sinks": 64},
        # long contexts in 8 bits: 65536 tokens held, 4112 of them seen
        {"name": "window_fp8_b16_64k", "op": "window", "cache": "fp8", "batch": 16, "q_len": 1, "lo": 65536,
         "hi": 65536, "window": 4096, "sinks": 16},
        # the last chunk of one prompt, just above the branch threshold
        {"name": "chunk_fp8_b1_300", "op": "chunk", "cache": "fp8", "batch": 1, "m_lo": 300, "m_hi": 300,
         "lo": 1000, "hi": 1000, "window": 511, "sinks": 4},
        # chunked prefill of four sequences after 16K cached tokens
        {"name": "chunk_b4_512_after_16k", "op": "chunk", "cache": "bf16", "batch": 4, "m_lo": 512, "m_hi": 512,
         "lo": 16896, "hi": 16896, "window": 4096, "sinks": 64},
        # one token's query absorption
        {"name": "absorb_w4_t1", "op": "absorb_w4", "tokens": 1, "group": 128},
        # the up-projection of a batch of sixteen, finer groups
        {"name": "up_w4_t16", "op": "up_w4", "tokens": 16, "group": 64},
        # a two-token step of 64 sequences
        {"name": "absorb_w4_t128", "op": "absorb_w4", "tokens": 128, "group": 64},
        # a chunk of 4 x 512 rows on the absorbed branch
        {"name": "up_w4_t2048", "op": "up_w4", "tokens": 2048, "group": 128},
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "window", "window", "chunk", "absorb_w4", "up_w4"])
    if op == "append":
        batch = _spread(rng, 1, 64)
        queries = rng.random() < 0.6
        new = _spread(rng, 1, max(1, (2048 if queries else 524288) // batch))
        return {"op": op, "batch": batch, "new": new, "ctx": _spread(rng, 1, 65536) - 1, "queries": queries}
    if op == "window":
        batch = _spread(rng, 1, 64)
        q_len = rng.choice([1, 1, 2, rng.randint(3, 8)])
        lo = _spread(rng, 16, 16384)
        hi = min(65536, _spread(rng, lo, 4 * lo))
        return {"op": op, "cache": rng.choice(["bf16", "fp8"]), "batch": batch, "q_len": q_len, "lo": lo, "hi": hi,
                "window": _spread(rng, 1, 4096 if q_len * batch <= 64 else 1024), "sinks": rng.choice([0, rng.randint(1, 64), 4])}
    if op == "chunk":
        batch = rng.randint(1, 4)
        m_lo = _spread(rng, 256, 512)
        m_hi = rng.randint(m_lo, 512)
        lo = _spread(rng, m_hi, 16384)
        return {"op": op, "cache": rng.choice(["bf16", "fp8"]), "batch": batch, "m_lo": m_lo, "m_hi": m_hi, "lo": lo,
                "hi": min(16896, _spread(rng, lo, 2 * lo)), "window": _spread(rng, 64, 4096),
                "sinks": rng.choice([0, rng.randint(1, 64), 4])}
    return {"op": op, "tokens": _spread(rng, 1, 2048), "group": rng.choice([32, 64, 128])}


def _lens(lo, hi, n):
    """n lengths spread over [lo, hi] in no order of size."""
    return [lo + int((hi - lo) * ((i * 0.6180339887498949 + 0.5) % 1.0) + 0.5) for i in range(n)]


def _shape(case):
    """(cached tokens, query rows) of each sequence of a window or chunk case."""
    seq = _lens(case["lo"], case["hi"], case["batch"])
    if case["op"] == "window":
        q = [min(case["q_len"], n) for n in seq]
    else:
        q = [min(m, n) for m, n in zip(_lens(case["m_lo"], case["m_hi"], case["batch"]), seq)]
    return seq, q


def _visible(p, window, sinks):
    """How many tokens a query at position p sees."""
    return min(p + 1, window) + min(max(p + 1 - window, 0), sinks)


def _kept(n, m, window, sinks):
    """How many cached tokens a chunk's m rows see, of n."""
    return min(n, min(sinks, n) + max(n - max(n - m + 1 - window, sinks), 0)) if n > sinks else n


def work(case):
    op = case["op"]
    if op == "append":
        n = case["batch"] * case["new"]
        b = n * (D_QK * 2 + 640 + 4 + 8 + 4)
        b += min(n, case["new"]) * 256                      # the positions' table rows
        b += 2 * n * H * D_R * 2 if case["queries"] else 0
        return {"bytes": b, "flops": n * (D_C * 2 + D_R * 3) + (n * H * D_R * 3 if case["queries"] else 0)}
    if op in ("absorb_w4", "up_w4"):
        K, N = (D_HC, D_C) if op == "absorb_w4" else (D_C, D_HC)
        t = case["tokens"]
        return {"bytes": H * K * N // 2 + H * (K // case["group"]) * N * 2 + t * H * (K + N) * 2,
                "flops": 2 * t * H * K * N}
    seq, q = _shape(case)
    w, s = case["window"], case["sinks"]
    token = 640 + 4 if case["cache"] == "fp8" else D_QK * 2
    pairs = sum(_visible(n - m + i, w, s) for n, m in zip(seq, q) for i in range(m))
    kept = sum(_kept(n, m, w, s) for n, m in zip(seq, q))
    if op == "window":
        return {"bytes": kept * token + sum(q) * H * (D_QK + D_C) * 2, "flops": pairs * H * 2 * (D_QK + D_C)}
    return {"bytes": kept * token + 2 * H * D_HC * D_C * 2 + sum(q) * H * (D_HC + D_R + D_HC) * 2,
            "flops": kept * H * 2 * D_C * 2 * D_HC + pairs * H * 2 * (D_HC + D_R + D_HC)}


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


def _pages(seq):
    return [(n + PAGE - 1) // PAGE for n in seq]


def _table(seq, seed):
    """A block table that hands out a random permutation of the pool."""
    r = torch.Generator()
    r.manual_seed(seed + 1)
    np_ = _pages(seq)
    perm = torch.randperm(sum(np_), generator=r).to(torch.int32)
    bt = torch.full((len(seq), max(np_)), -1, dtype=torch.int32)
    k = 0
    for b, n in enumerate(np_):
        bt[b, :n] = perm[k:k + n]
        k += n
    return bt, sum(np_)


def _cache(g, kind, num_pages):
    if kind == "bf16":
        return {"kv": _normal(g, (num_pages, PAGE, D_QK))}
    rows = torch.empty((num_pages, PAGE, 640), dtype=torch.uint8, device=DEV)
    scales = torch.empty((num_pages, PAGE), dtype=torch.float32, device=DEV)
    for i in range(0, num_pages, 4096):
        c = _normal(g, (min(4096, num_pages - i), PAGE, D_QK))
        codes, sc = _quantise(c[..., :D_C])
        rows[i:i + 4096, :, :D_C] = codes.view(torch.uint8)
        rows[i:i + 4096, :, D_C:] = c[..., D_C:].contiguous().view(torch.uint8)
        scales[i:i + 4096] = sc
    return {"rows": rows, "scales": scales}


def _rope_table(max_pos):
    i = torch.arange(D_R // 2, dtype=torch.float64, device=DEV)
    a = torch.arange(max_pos, dtype=torch.float64, device=DEV)[:, None] * torch.pow(10000.0, -2.0 * i / D_R)
    return torch.stack([a.cos(), a.sin()], dim=-1).float().contiguous()


def _codes4(g, K, N, group):
    """4-bit weights as a user's program keeps them: eight codes of the contraction to a word, and the groups' scales."""
    w = _normal(g, (H, K, N), math.sqrt(1.0 / D_C)).float()
    wg = w.view(H, K // group, group, N)
    sc = (wg.abs().amax(dim=2) / 7.0).to(torch.bfloat16)
    q = torch.round(wg / sc.float().unsqueeze(2)).clamp(-8, 7).to(torch.int64).view(H, K // 8, 8, N) & 15
    words = torch.zeros((H, K // 8, N), dtype=torch.int64, device=DEV)
    for i in range(8):
        words |= q[:, :, i] << (4 * i)
    words = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
    return words.contiguous(), sc.contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"op": op, "case": dict(case), "err": torch.zeros(1, dtype=torch.int32, device=DEV)}
    if op == "append":
        B, new, ctx = case["batch"], case["new"], case["ctx"]
        n = B * new
        first = ctx // PAGE
        held = (ctx + new - 1) // PAGE - first + 1          # the pages that the new tokens touch
        perm = torch.randperm(B * held, generator=g, device=DEV).view(B, held)
        pos = ctx + torch.arange(new, device=DEV)
        st["slots"] = (perm[:, pos // PAGE - first] * PAGE + pos % PAGE).reshape(-1).contiguous()
        st["positions"] = pos.to(torch.int32).repeat(B)
        st["table"] = _rope_table(ctx + new)
        st["c"] = _normal(g, (n, D_C))
        st["k"] = _normal(g, (n, D_R))
        st["rows"] = torch.zeros((B * held, PAGE, 640), dtype=torch.uint8, device=DEV)
        st["scales"] = torch.ones((B * held, PAGE), dtype=torch.float32, device=DEV)
        st["q"] = _normal(g, (n, H, D_R)) if case["queries"] else None
        st["q_out"] = torch.zeros_like(st["q"]) if case["queries"] else None
        return st
    if op in ("absorb_w4", "up_w4"):
        K, N = (D_HC, D_C) if op == "absorb_w4" else (D_C, D_HC)
        st["words"], st["wscale"] = _codes4(g, K, N, case["group"])
        st["x"] = _normal(g, (case["tokens"], H, K))
        st["out"] = torch.zeros((case["tokens"], H, N), dtype=torch.bfloat16, device=DEV)
        return st
    seq, q = _shape(case)
    bt, num_pages = _table(seq, seed)
    T = sum(q)
    st["seq"], st["q_lens"] = seq, q
    st["bt"] = bt.to(DEV)
    st |= _cache(g, case["cache"], num_pages)
    st["row_seq"] = torch.tensor([b for b, m in enumerate(q) for _ in range(m)], device=DEV)
    st["row_pos"] = torch.tensor([n - m + i for n, m in zip(seq, q) for i in range(m)], device=DEV)
    st["q_r"] = _normal(g, (T, H, D_R))
    if op == "window":
        st["q_abs"] = _normal(g, (T, H, D_C), 0.5)
        st["out"] = torch.zeros((T, H, D_C), dtype=torch.bfloat16, device=DEV)
        if own:                                             # the step's plan, shared by a model's layers
            from mla_latent_kv_02_gb300 import api
            st["plan"] = api.mla_window_plan(seq, q, case["window"], case["sinks"])
        return st
    st["q_c"] = _normal(g, (T, H, D_HC))
    st["w_uk"] = _normal(g, (H, D_HC, D_C), math.sqrt(1.0 / D_C))
    st["w_uv"] = _normal(g, (H, D_C, D_HC), math.sqrt(1.0 / D_C))
    st["out"] = torch.zeros((T, H, D_HC), dtype=torch.bfloat16, device=DEV)
    st["starts"] = [sum(q[:i]) for i in range(len(q))]
    if own:                                                 # the workspace that a serving program keeps
        from mla_latent_kv_02_gb300 import api
        nbytes = api.mla_prefill_window_workspace_size(q, seq, case["window"], case["sinks"])
        st["ws"] = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------------ plain forms
def _rotate(x, cs):
    """Pairs (x[2i], x[2i+1]) of [..., 64] turned by (cos, sin) [..., 32, 2]."""
    x = x.float().unflatten(-1, (D_R // 2, 2))
    a, b, c, s = x[..., 0], x[..., 1], cs[..., 0], cs[..., 1]
    return torch.stack([a * c - b * s, a * s + b * c], dim=-1).flatten(-2)


def _plain_append(st):
    cs = st["table"][st["positions"].long()]
    codes, sc = _quantise(st["c"])
    rows = st["rows"].view(-1, 640)
    row = torch.cat([codes.view(torch.uint8), _rotate(st["k"], cs).to(torch.bfloat16).view(torch.uint8)], dim=1)
    rows[st["slots"]] = row
    st["scales"].view(-1)[st["slots"]] = sc
    if st["q"] is not None:
        st["q_out"].copy_(_rotate(st["q"], cs[:, None]))


def _rows(st, slots):
    """Cached rows [..., 576] of the given slots, in 32 bits."""
    if "kv" in st:
        return st["kv"].view(-1, D_QK)[slots].float()
    r = st["rows"].view(-1, 640)[slots]
    lat = r[..., :D_C].contiguous().view(torch.float8_e4m3fn).float() * st["scales"].view(-1)[slots].unsqueeze(-1)
    return torch.cat([lat, r[..., D_C:].contiguous().view(torch.bfloat16).float()], dim=-1)


def _slots(bt, b, pos):
    return bt[b, pos // PAGE].long() * PAGE + pos % PAGE


def _plain_window(st):
    w, s = st["case"]["window"], st["case"]["sinks"]
    pos = st["row_pos"][:, None]
    w = min(w, max(st["seq"]))
    sink = torch.arange(s, device=DEV)[None].expand(pos.shape[0], -1)
    win = pos - torch.arange(w, device=DEV)[None]
    at = torch.cat([sink, win], dim=1)
    seen = torch.cat([sink <= pos - w, win >= 0], dim=1)    # a sink inside the window counts there
    kv = _rows(st, _slots(st["bt"], st["row_seq"][:, None], torch.where(seen, at, torch.zeros_like(at))))
    q = torch.cat([st["q_abs"], st["q_r"]], dim=-1).float()
    x = torch.matmul(q, kv.transpose(1, 2)) * SCALE
    x = x.masked_fill(~seen[:, None], -math.inf)
    p = torch.exp(x - x.amax(dim=-1, keepdim=True))
    o = torch.matmul(p, kv[..., :D_C]) / p.sum(dim=-1, keepdim=True)
    return o.to(torch.bfloat16)


def _plain_chunk(st):
    w, s = st["case"]["window"], st["case"]["sinks"]
    n = torch.tensor(st["seq"], device=DEV)[:, None]
    m = torch.tensor(st["q_lens"], device=DEV)[:, None]
    start = torch.tensor(st["starts"], device=DEV)[:, None]
    M = max(st["q_lens"])
    lead = torch.clamp(n - m + 1 - w, min=s)                # the first token after the sinks that a row sees
    tail = max(max(a - max(a - b + 1 - w, s), 0) for a, b in zip(st["seq"], st["q_lens"]))
    at = torch.cat([torch.arange(s, device=DEV)[None].expand(n.shape[0], -1), lead + torch.arange(tail, device=DEV)], dim=1)
    held = at < n                                           # [sequences, kept tokens]
    kv = _rows(st, _slots(st["bt"], torch.arange(n.shape[0], device=DEV)[:, None], torch.where(held, at, torch.zeros_like(at))))
    k = torch.einsum("blc,hdc->bhld", kv[..., :D_C], st["w_uk"].float())
    v = torch.einsum("blc,hcd->bhld", kv[..., :D_C], st["w_uv"].float())
    i = torch.arange(M, device=DEV)[None]
    row = start + torch.minimum(i, m - 1)                   # rows past a chunk's end repeat its last one
    pos = n - m + torch.minimum(i, m - 1)
    seen = held[:, None] & (at[:, None] <= pos[..., None]) & ((at[:, None] < s) | (at[:, None] > pos[..., None] - w))
    qc, qr = st["q_c"][row].float().transpose(1, 2), st["q_r"][row].float().transpose(1, 2)
    x = torch.matmul(qc, k.transpose(2, 3)) + torch.matmul(qr, kv[:, None, :, D_C:].transpose(2, 3))
    x = (x * SCALE).masked_fill(~seen[:, None], -math.inf)
    p = torch.exp(x - x.amax(dim=-1, keepdim=True))
    o = (torch.matmul(p, v) / p.sum(dim=-1, keepdim=True)).transpose(1, 2)
    out = torch.empty_like(st["out"])
    out[row.reshape(-1)] = o.reshape(-1, H, D_HC).to(torch.bfloat16)
    return out


def _plain_w4(st):
    words, sc = st["words"], st["wscale"].float()
    K, N = words.shape[1] * 8, words.shape[2]
    shift = torch.arange(0, 32, 4, device=DEV, dtype=torch.int32)
    code = (((words[:, :, None] >> shift[:, None]) & 15) ^ 8) - 8
    w = code.view(H, sc.shape[1], K // sc.shape[1], N).float() * sc[:, :, None]
    y = torch.matmul(st["x"].float().transpose(0, 1), w.view(H, K, N))
    return y.transpose(0, 1).to(torch.bfloat16).contiguous()


def run(st):
    op = st["op"]
    if op == "append":
        if own:
            from mla_latent_kv_02_gb300 import api
            api.mla_kv_append_rope_fp8(st["c"], st["k"], st["positions"], st["table"], st["slots"], st["rows"],
                                       st["scales"], st["err"], q_pe=st["q"], q_r=st["q_out"])
        else:
            _plain_append(st)
        out = {"codes": st["rows"][..., :D_C].view(torch.float8_e4m3fn), "scales": st["scales"],
               "k_r": st["rows"][..., D_C:].view(torch.bfloat16)}
        if st["q"] is not None:
            out["q_r"] = st["q_out"]
        return out
    if op == "window":
        if own:
            from mla_latent_kv_02_gb300 import api
            if "kv" in st:
                api.mla_decode_window(st["q_abs"], st["q_r"], st["kv"], st["bt"], st["plan"], st["out"], st["err"],
                                      scale=SCALE)
            else:
                api.mla_decode_window_fp8(st["q_abs"], st["q_r"], st["rows"], st["scales"], st["bt"], st["plan"],
                                          st["out"], st["err"], scale=SCALE)
            return st["out"]
        return _plain_window(st)
    if op == "chunk":
        if own:
            from mla_latent_kv_02_gb300 import api
            c = st["case"]
            ids = range(len(st["seq"]))
            if "kv" in st:
                api.mla_prefill_window_batch(st["q_c"], st["q_r"], st["kv"], st["bt"], ids, st["starts"], st["q_lens"],
                                             st["seq"], c["window"], c["sinks"], st["w_uk"], st["w_uv"], st["ws"],
                                             st["out"], st["err"], scale=SCALE)
            else:
                api.mla_prefill_window_batch_fp8(st["q_c"], st["q_r"], st["rows"], st["scales"], st["bt"], ids,
                                                 st["starts"], st["q_lens"], st["seq"], c["window"], c["sinks"],
                                                 st["w_uk"], st["w_uv"], st["ws"], st["out"], st["err"], scale=SCALE)
            return st["out"]
        return _plain_chunk(st)
    if own:
        from mla_latent_kv_02_gb300 import api
        f = api.mla_absorb_q_w4 if op == "absorb_w4" else api.mla_up_v_w4
        f(st["x"], st["words"], st["wscale"], st["out"], st["err"])
        return st["out"]
    return _plain_w4(st)


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "append":
        return _exact_append(st)
    if op == "window":
        return _exact_window(st, case)
    if op == "chunk":
        return _exact_chunk(st, case)
    x, words, sc = st["x"].double(), st["words"].long(), st["wscale"].double()
    t, K, N, group = case["tokens"], words.shape[1] * 8, words.shape[2], case["group"]
    y = torch.zeros((t, H, N), dtype=torch.float64, device=DEV)
    for k in range(K):                                      # one row of every head's weights at a time
        nib = torch.bitwise_and(torch.bitwise_right_shift(words[:, k // 8], 4 * (k % 8)), 15)
        val = torch.where(nib > 7, nib - 16, nib).double() * sc[:, k // group]
        y += x[:, :, k, None] * val
    return y


def _exact_append(st):
    c = st["c"].double()
    n = c.shape[0]
    codes = torch.zeros((st["rows"].shape[0] * PAGE, D_C), dtype=torch.float64, device=DEV)
    keys = torch.zeros((st["rows"].shape[0] * PAGE, D_R), dtype=torch.float64, device=DEV)
    scales = torch.ones(st["rows"].shape[0] * PAGE, dtype=torch.float64, device=DEV)
    big = c.abs().max(dim=1).values
    k = torch.ceil(torch.log2(big.clamp(min=1e-300) / 448.0))
    k = torch.where(big > 448.0 * torch.exp2(k), k + 1, k)  # the logarithm may round across a power of two
    k = torch.where(big <= 448.0 * torch.exp2(k - 1), k - 1, k)
    k = torch.where(big == 0, torch.zeros_like(k), k)
    codes[st["slots"]] = c * torch.exp2(-k)[:, None]
    scales[st["slots"]] = torch.exp2(k)
    z = torch.view_as_complex(st["table"].double())[st["positions"].long()]
    turn = lambda x, z: torch.view_as_real(torch.view_as_complex(x.double().reshape(*x.shape[:-1], D_R // 2, 2)) * z).flatten(-2)  # noqa: E731
    keys[st["slots"]] = turn(st["k"], z)
    out = {"codes": codes.view(-1, PAGE, D_C), "scales": scales.view(-1, PAGE), "k_r": keys.view(-1, PAGE, D_R)}
    if st["q"] is not None:
        out["q_r"] = turn(st["q"], z[:, None])
    return out


def _exact_tokens(st, b, positions):
    """Latents and RoPE keys of a sequence's tokens, in 64 bits."""
    pages = st["bt"][b].long()[positions // PAGE]
    if "kv" in st:
        r = st["kv"][pages, positions % PAGE].double()
        return r[:, :D_C], r[:, D_C:]
    r = st["rows"][pages, positions % PAGE]
    c = r[:, :D_C].int()
    e, f = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e > 0, (8 + f) * torch.exp2(e.double() - 10), f * 2.0 ** -9)
    v = torch.where(c >= 128, -v, v) * st["scales"][pages, positions % PAGE].double()[:, None]
    return v, r[:, D_C:].contiguous().view(torch.bfloat16).double()


def _seen_positions(p, window, sinks):
    j = torch.arange(p + 1, device=DEV)
    return j[(j < sinks) | (j > p - window)]


def _exact_window(st, case):
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
    t = 0
    for b, (n, m) in enumerate(zip(st["seq"], st["q_lens"])):
        for i in range(m):
            c, r = _exact_tokens(st, b, _seen_positions(n - m + i, case["window"], case["sinks"]))
            s = (st["q_abs"][t].double() @ c.T + st["q_r"][t].double() @ r.T) * SCALE
            out[t] = torch.softmax(s, dim=-1) @ c
            t += 1
    return out


def _exact_chunk(st, case):
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
    uk, uv = st["w_uk"].double(), st["w_uv"].double()
    for b, (n, m, t0) in enumerate(zip(st["seq"], st["q_lens"], st["starts"])):
        first = max(0, n - m + 1 - case["window"])
        j = torch.arange(n, device=DEV)
        j = j[(j < case["sinks"]) | (j >= first)]
        c, r = _exact_tokens(st, b, j)
        p = torch.arange(n - m, n, device=DEV)[:, None]
        hide = (j > p) | ((j >= case["sinks"]) & (j <= p - case["window"]))
        for h in range(H):
            s = st["q_c"][t0:t0 + m, h].double() @ (c @ uk[h].T).T + st["q_r"][t0:t0 + m, h].double() @ r.T
            a = torch.softmax((s * SCALE).masked_fill(hide, -math.inf), dim=-1)
            out[t0:t0 + m, h] = a @ (c @ uv[h])
    return out
