"""A sequence served in bounded memory, the new operators together as a server runs them.

Prompt chunk, then two-token steps over the FP8 cache: rotating append, 4-bit
query absorption, windowed decode, 4-bit up-projection; pages that slid out of
the window go back to the pool and are handed out again.  The 64-bit reference
keeps every token (the dequantised latents and the keys as cached), so it is
right only if the cache holds what each row may see.

Bound of the difference, in the 2-norm: the steps round four times at half a
bf16 step or better (absorbed queries or expanded keys, probabilities, the
latent output or expanded values, the result), each at most 2^-8 relative, and
scores of unit variance pass a relative error on with a factor of at most two:
8 * 2^-8.
"""
import math

import numpy as np
import pytest

import oracle
from mla_latent_kv_02_gb300 import workloads as wl

from _helpers import to_bf16
from _window_ref import SCALE, bf16, seen_positions

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
f8 = oracle.fp8_cache


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from mla_latent_kv_02_gb300 import api as a
    a.mla_version()
    return a


def _w4_values(words, scales):
    w = words.to(torch.int64) & 0xFFFFFFFF
    nib = torch.stack([(w >> (4 * i)) & 15 for i in range(8)], dim=2)
    code = torch.where(nib > 7, nib - 16, nib).reshape(128, -1, words.shape[2])
    return code.double() * scales.double().repeat_interleave(code.shape[1] // scales.shape[1], dim=1)


class Server:
    """One or more sequences over a small pool, window and sinks fixed."""

    def __init__(self, api, batch, window, sinks, pages, seed):
        self.api, self.window, self.sinks = api, window, sinks
        self.rng = np.random.default_rng(seed)
        self.pool = api.MlaPool(pages)
        self.rows = torch.full((pages, 64, 640), 0x55, dtype=torch.uint8, device="cuda")
        self.scales = torch.ones((pages, 64), dtype=torch.float32, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.table = torch.empty((4096, 32, 2), dtype=torch.float32, device="cuda")
        api.mla_rope_table(4096, self.table)
        self.bt = np.full((batch, 64), -1, np.int32)
        self.n = [0] * batch
        self.lat = [np.zeros((0, 512)) for _ in range(batch)]
        self.key = [np.zeros((0, 64)) for _ in range(batch)]
        std = 512 ** -0.5
        self.w_uk = to_bf16(bf16(self.rng, (128, 128, 512), std), "cuda")
        self.w_uv = to_bf16(bf16(self.rng, (128, 512, 128), std), "cuda")
        self.uk4, self.uv4 = api.mla_pack_w4(self.w_uk, 64), api.mla_pack_w4(self.w_uv, 128)

    def append(self, counts):
        """New tokens of every sequence, with their queries; returns (q_c, rotated q_r) on the GPU."""
        T = sum(counts)
        c, k = bf16(self.rng, (T, 512)), bf16(self.rng, (T, 64))
        q_c, q_pe = to_bf16(bf16(self.rng, (T, 128, 128)), "cuda"), to_bf16(bf16(self.rng, (T, 128, 64)), "cuda")
        seq, pos = [], []
        for b, m in enumerate(counts):
            for p in range(self.n[b], self.n[b] + m):
                if self.bt[b, p // 64] < 0:
                    self.bt[b, p // 64] = int(self.pool.alloc(1)[0])
                seq.append(b)
                pos.append(p)
            self.n[b] += m
        slots = self.api.mla_slot_mapping(self.bt, np.array(seq, np.int32), np.array(pos, np.int32))
        tpos = torch.tensor(pos, dtype=torch.int32, device="cuda")
        q_r = torch.empty_like(q_pe)
        self.api.mla_kv_append_rope_fp8(to_bf16(c, "cuda"), to_bf16(k, "cuda"), tpos, self.table,
                                        torch.from_numpy(slots).cuda(), self.rows, self.scales, self.err, q_pe=q_pe, q_r=q_r)
        codes, sc = f8.quantize_rows(c)
        lat = f8.dequantize_rows(codes, sc)
        stored = self.rows.view(-1, 640)[torch.from_numpy(slots).cuda(), 512:].contiguous().view(torch.bfloat16)
        key = stored.float().cpu().numpy()
        t = 0
        for b, m in enumerate(counts):
            self.lat[b] = np.concatenate([self.lat[b], lat[t:t + m]])
            self.key[b] = np.concatenate([self.key[b], key[t:t + m]])
            t += m
        return q_c, q_r

    def evict(self):
        """Pages that no later row can see go back to the pool."""
        for b, n in enumerate(self.n):
            for pg in range(self.bt.shape[1]):
                last = pg * 64 + 63
                if self.bt[b, pg] >= 0 and pg * 64 >= self.sinks and last < n - self.window + 1:
                    self.rows[int(self.bt[b, pg])] = 0x7F            # NaN codes: a later read would show
                    self.pool.free([int(self.bt[b, pg])])
                    self.bt[b, pg] = -1

    def check(self, out, q_c, q_r, counts, w_uk, w_uv):
        t = 0
        for b, m in enumerate(counts):
            for i in range(m):
                if m <= 4 or i % 37 == 0 or i == m - 1:
                    at = seen_positions(self.n[b] - m + i, self.window, self.sinks)
                    c = torch.from_numpy(self.lat[b][at].astype(np.float64)).cuda()
                    r = torch.from_numpy(self.key[b][at].astype(np.float64)).cuda()
                    qa = torch.einsum("hd,hdc->hc", q_c[t].double(), w_uk)
                    s = (qa @ c.T + q_r[t].double() @ r.T) * SCALE
                    want = torch.einsum("hc,hcd->hd", torch.softmax(s, dim=-1) @ c, w_uv)
                    rel = float((out[t].double() - want).norm() / want.norm())
                    assert rel <= 8 * 2.0 ** -8, (b, i, rel)
                t += 1

    def chunk(self, counts):
        q_c, q_r = self.append(counts)
        out = torch.empty((sum(counts), 128, 128), dtype=torch.bfloat16, device="cuda")
        starts = [sum(counts[:b]) for b in range(len(counts))]
        ws = torch.empty(self.api.mla_prefill_window_workspace_size(counts, self.n, self.window, self.sinks),
                         dtype=torch.uint8, device="cuda")
        self.api.mla_prefill_window_batch_fp8(q_c, q_r, self.rows, self.scales, torch.from_numpy(self.bt).cuda(),
                                              range(len(counts)), starts, counts, self.n, self.window, self.sinks,
                                              self.w_uk, self.w_uv, ws, out, self.err)
        assert self.api.mla_check(self.err) == 0
        self.check(out, q_c, q_r, counts, self.w_uk.double(), self.w_uv.double())

    def step(self, counts):
        api = self.api
        q_c, q_r = self.append(counts)
        T = sum(counts)
        q_abs, o = (torch.empty((T, 128, 512), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        out = torch.empty((T, 128, 128), dtype=torch.bfloat16, device="cuda")
        plan = api.mla_window_plan(self.n, counts, self.window, self.sinks)
        api.mla_absorb_q_w4(q_c, *self.uk4, q_abs, self.err)
        api.mla_decode_window_fp8(q_abs, q_r, self.rows, self.scales, torch.from_numpy(self.bt).cuda(), plan, o, self.err)
        api.mla_up_v_w4(o, *self.uv4, out, self.err)
        assert api.mla_check(self.err) == 0
        self.check(out, q_c, q_r, counts, _w4_values(*self.uk4), _w4_values(*self.uv4))


def test_served_in_bounded_memory(api):
    s = Server(api, batch=3, window=200, sinks=4, pages=36, seed=5)
    s.chunk([300, 270, 257])                                 # prompts, first chunk
    s.evict()
    s.chunk([301, 290, 511])                                 # and second: pages of the first handed out again
    s.evict()
    for counts in ([2, 2, 2], [1, 0, 3], [1, 1, 1], [16, 1, 16], [40, 40, 40], [2, 2, 2]):
        s.step(counts)
        s.evict()
    held = int((s.bt >= 0).sum())
    assert held == 36 - s.pool.available() and held <= 3 * (1 + (200 + 62) // 64 + 1), "more pages held than the window needs"


def test_a_long_stream_holds_the_pool(api):
    """A sequence that outgrows its pool many times over."""
    s = Server(api, batch=1, window=130, sinks=70, pages=6, seed=6)
    s.step([1])
    while s.n[0] < 1400:
        s.step([37 if s.n[0] < 1200 else 64])
        s.evict()
    assert s.n[0] >= 1400 and s.pool.available() >= 0
