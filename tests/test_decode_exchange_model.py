"""Model check of the decode's score exchange in parts, each buffer as byte ranges (CPU only).

test_decode_model.py gives every warp one block of an exchange buffer, for scores and
finished rows alike.  Where a tile's scores cross in two parts a warp's share is two
blocks, and what a finished row takes on its way to memory is a question of bytes.
Here the ranges are those of csrc/exchange.h, asked of the header itself, for the forms
of the decode whose softmax warps store the rows (bf16 and windowed: two parts; over the
FP8 cache: one), with the roles as they issue and wait now: scores leave TMEM and free
it before any is staged, part after part is pushed, part after part is received and its
barrier armed again, QK^T waits for its page last.  Under random interleavings of every
role, of the four warps of both softmax warpgroups and of every asynchronous completion:
  * no byte is staged, received or used by a finished row while it holds scores not yet
    read, a copy's source, or another warp's row;
  * every parity wait passes only when its own phase is complete, and nothing deadlocks;
  * after an abort no CTA exits with a copy in flight.
"""
import random
import shutil
import subprocess

import pytest

from mla_latent_kv_02_gb300 import _build
from test_decode_model import Barrier, ProtocolError, _layouts

STAGES, XBUFS, WARPS = 4, 4, 4
GRAIN = 1024                                                 # bytes that the model tells apart

PROGRAM = r"""
#include <cstdio>
#include "exchange.h"
template <int kParts> void print() {
  using X = mla::decode::Exchange<kParts>;
  for (unsigned w = 0; w < 4; ++w) {
    for (unsigned p = 0; p < kParts; ++p) std::printf("share %d %u %u %u %d\n", kParts, w, p, p * X::kBytes + X::share(w), X::kWarp);
    for (unsigned r = 0; r < 32; ++r) {
      for (unsigned p = 0; p < kParts; ++p)
        for (unsigned k = 0; k < X::kPieces; ++k) std::printf("scores %d %u %u %u\n", kParts, w, p, X::scores(32 * w + r, p, k));
      for (unsigned k = 0; k < 8; ++k) std::printf("row %d %u %u %u %u\n", kParts, w, r, k, X::finished(w, r, k));
    }
  }
}
int main() { std::printf("buffer %d\n", mla::decode::kXBytes); print<1>(); print<2>(); }
"""


@pytest.fixture(scope="module")
def header(tmp_path_factory):
    """The lines that the header's arithmetic prints."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("needs a host compiler")
    d = tmp_path_factory.mktemp("exchange")
    (d / "x.cpp").write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-Wall", "-Werror", "-I", _build.CSRC, str(d / "x.cpp"), "-o", str(d / "x")], check=True)
    lines = subprocess.run([str(d / "x")], check=True, capture_output=True, text=True).stdout.split("\n")
    return [[x if i == 0 else int(x) for i, x in enumerate(line.split())] for line in lines if line]


class Places:
    """Grains of a buffer: share[w][p], what warp w stages, sends and receives of part p; room[w], what its rows take."""

    def __init__(self, header, parts):
        self.parts = parts
        self.buffer = next(x[1] for x in header if x[0] == "buffer") // GRAIN
        self.share = [[None] * parts for _ in range(WARPS)]
        self.room = [set() for _ in range(WARPS)]
        for x in header:
            if x[0] == "share" and x[1] == parts:
                assert x[4] % GRAIN == 0 and x[5] % GRAIN == 0
                self.share[x[2]][x[3]] = set(range(x[4] // GRAIN, (x[4] + x[5]) // GRAIN))
            if x[0] == "row" and x[1] == parts:
                self.room[x[2]] |= {x[5] // GRAIN, (x[5] + 15) // GRAIN}


def contiguous(places):
    """A quarter of the buffer for each warp's rows, whatever the parts."""
    n = places.buffer // WARPS
    places.room = [set(range(w * n, (w + 1) * n)) for w in range(WARPS)]
    return places


@pytest.mark.parametrize("parts", [1, 2])
def test_places_of_scores_and_rows(header, parts):
    """The scores fill a buffer, a warp's all within its shares; its row pieces too, each in a place of its own, and the
    eight lanes that write or read at one time touch every bank once."""
    shares = {(x[2], x[3]): range(x[4], x[4] + x[5]) for x in header if x[0] == "share" and x[1] == parts}
    scores = [x[2:] for x in header if x[0] == "scores" and x[1] == parts]
    assert sorted(at for _, _, at in scores) == list(range(0, next(x[1] for x in header if x[0] == "buffer"), 16))
    assert all(at in shares[w, p] and at + 15 in shares[w, p] for w, p, at in scores)
    rows = {(x[2], x[3], x[4]): x[5] for x in header if x[0] == "row" and x[1] == parts}
    assert len(rows) == WARPS * 32 * 8
    for w in range(WARPS):
        mine = [rows[w, r, k] for r in range(32) for k in range(8)]
        assert len(set(mine)) == 256
        assert all(any(at in shares[w, p] and at + 15 in shares[w, p] for p in range(parts)) for at in mine)
        for i in range(0, 32, 8):                            # written: a lane a row; read: eight lanes a row
            for k in range(8):
                assert len({rows[w, i + j, k] // 16 % 8 for j in range(8)}) == 8
        for r in range(32):
            assert len({rows[w, r, k] // 16 % 8 for k in range(8)}) == 8


def run_model(segs, seed, places, xlead=2, epi_shift=0, early_push=False, abort_at=None, drain=True):
    """Parameters as in test_decode_model.py; places: where scores and rows lie."""
    rnd = random.Random(seed)
    parts = places.parts
    tiles = [(si, i == 0, i == n - 1) for si, n in enumerate(segs) for i in range(n)]
    G = len(tiles)
    ctas = [dict(kv_full=[Barrier(1) for _ in range(STAGES)], kv_empty=[Barrier(1) for _ in range(STAGES)],
                 s_full=[Barrier(1), Barrier(1)], s_free=Barrier(WARPS), p_full=Barrier(WARPS),
                 o_done=[Barrier(1), Barrier(1)], q_ready=Barrier(WARPS), o_free=Barrier(WARPS),
                 x_full=[[Barrier(1) for _ in range(XBUFS)] for _ in range(parts)],
                 armed=[[-1] * XBUFS for _ in range(parts)],
                 bytes=[[None] * places.buffer for _ in range(XBUFS)], reading=[[False] * places.buffer for _ in range(XBUFS)],
                 slot=[[None] * WARPS for _ in range(4)], slot_unread=[[False] * WARPS for _ in range(4)],
                 abort=False, pushes=[0] * (2 * WARPS), peer_pushes=None, peer_abort=None, exited=False, arrived=False)
            for _ in range(2)]
    events = []

    def wait(c, cond):
        n = 0
        while not cond():
            if c["abort"]:
                return False
            n += 1
            if n > 200 and any(x["abort"] for x in ctas):    # the kernel's waits are bounded
                c["abort"] = True
                return False
            yield
        return True

    def take_bytes(c, b, grains, what, who):
        """`who` writes `what` into these grains: nothing else may live there."""
        for i in grains:
            held = c["bytes"][b][i]
            if held is not None and held[0] in ("data", "row"):
                raise ProtocolError(f"{who} over {held}")
            if c["reading"][b][i]:
                raise ProtocolError(f"{who} over a copy in flight")
            c["bytes"][b][i] = what

    def setup(ci):
        for _ in range(rnd.randrange(60)):
            yield
        ctas[ci]["arrived"] = True

    def producer(ci):
        c = ctas[ci]
        while not c["arrived"]:
            yield
        for t in range(G):
            if t >= STAGES and not (yield from wait(c, lambda: c["kv_empty"][t % STAGES].test(t // STAGES - 1))):
                return
            events.append(("kv", ci, t))

    def qk(ci):
        c = ctas[ci]
        for t, (seg, first, _) in enumerate(tiles):
            if first and not (yield from wait(c, lambda: c["q_ready"].test(seg))):
                return
            if t > 0 and not (yield from wait(c, lambda: c["s_free"].test(t - 1))):
                return
            if not (yield from wait(c, lambda: c["kv_full"][t % STAGES].test(t // STAGES))):
                return
            events.append(("s", ci, t))

    def pv(ci):
        c = ctas[ci]
        for t, (seg, first, _) in enumerate(tiles):
            if not (yield from wait(c, lambda: c["p_full"].test(t))):
                return
            if first and not (yield from wait(c, lambda: c["o_free"].test(seg))):
                return
            events.append(("o", ci, t))

    def softmax_warp(ci, wg, w):
        c = ctas[ci]
        while not c["arrived"]:
            yield
        if wg == 0:
            c["o_free"].arrive()
            c["q_ready"].arrive()
            if w == 0:
                for t in range(min(G, XBUFS)):
                    for p in range(parts):
                        c["x_full"][p][t].arrive(1, expect_tx=WARPS)
                        c["armed"][p][t] = t
        for t in range(wg, G, 2):
            seg, first, last = tiles[t]
            if not (yield from wait(c, lambda: c["s_full"][t & 1].test(t >> 1))):
                return
            c["s_free"].arrive()                             # the scores are in registers
            sb, b = (t + xlead) % XBUFS, t % XBUFS
            for p in range(parts):
                if rnd.random() < 0.5:
                    yield
                take_bytes(c, sb, places.share[w][p], ("stage", t, w, p), f"staging tile {t} part {p} by warp {w}")
                yield
                if not early_push:
                    while not ctas[1 - ci]["arrived"]:
                        yield
                if not ctas[1 - ci]["arrived"]:
                    raise ProtocolError("scores pushed before the peer was set up")
                for i in places.share[w][p]:
                    if c["bytes"][sb][i] != ("stage", t, w, p):
                        raise ProtocolError(f"tile {t} part {p} pushed by warp {w} holds {c['bytes'][sb][i]}")
                    c["reading"][sb][i] = True
                events.append(("x", ci, (t, w, p, sb)))
            c["pushes"][wg * WARPS + w] += 1
            if last and seg + 1 < len(segs):
                c["q_ready"].arrive()
            yield
            for p in range(parts):
                bar = c["x_full"][p][b]
                if not (yield from wait(c, lambda: bar.test(t // XBUFS))):
                    return
                if w == 0 and t + XBUFS < G:
                    bar.arrive(1, expect_tx=WARPS)
                    c["armed"][p][b] = t + XBUFS
                yield
                for i in places.share[w][p]:
                    if c["bytes"][b][i] != ("data", t, w, p):
                        raise ProtocolError(f"tile {t} part {p} reads {c['bytes'][b][i]}")
                    c["bytes"][b][i] = None
            if not first:
                sl = (t - 1) % 4
                if not (yield from wait(c, lambda: c["slot"][sl][w] == t - 1)):
                    return
                c["slot_unread"][sl][w] = False
            sl = t % 4
            if c["slot_unread"][sl][w]:
                raise ProtocolError(f"tile {t} overwrites tile {c['slot'][sl][w]}'s max before it was read")
            c["slot"][sl][w] = t
            c["slot_unread"][sl][w] = t + 1 < G and not tiles[t + 1][1]
            yield
            if t > 0 and not (yield from wait(c, lambda: c["o_done"][(t - 1) & 1].test((t - 1) >> 1))):
                return
            c["p_full"].arrive()
            if last:
                if not (yield from wait(c, lambda: c["o_done"][t & 1].test(t >> 1))):
                    return
                eb = (t + epi_shift) % XBUFS
                for rnd_ in range(4):                        # the finished row, a round at a time
                    what = ("row", t, w, rnd_)
                    take_bytes(c, eb, places.room[w], what, f"warp {w}'s row of tile {t}")
                    for _ in range(rnd.randrange(1, 12)):
                        yield
                    for i in places.room[w]:
                        if c["bytes"][eb][i] != what:
                            raise ProtocolError(f"warp {w} stores {c['bytes'][eb][i]} as its row of tile {t}")
                        c["bytes"][eb][i] = None
                c["o_free"].arrive()

    def exit_sequence(ci):
        c, peer = ctas[ci], ctas[1 - ci]
        peer["peer_pushes"] = list(c["pushes"])
        peer["peer_abort"] = c["abort"]
        c["at_barrier"] = 1
        while peer.get("at_barrier", 0) < 1:
            yield
        if drain and (c["abort"] or c["peer_abort"]):
            for p in range(parts):
                for b in range(XBUFS):
                    t, bar = c["armed"][p][b], c["x_full"][p][b]
                    if t < 0 or bar.phase >= t // XBUFS + 1:
                        continue
                    issued = sum(1 for q in range(WARPS) if c["peer_pushes"][(t & 1) * WARPS + q] > t >> 1)
                    if issued < WARPS:
                        bar.complete_tx(WARPS - issued)
                    while bar.phase < t // XBUFS + 1:
                        yield
            c["at_barrier"] = 2
            while peer.get("at_barrier", 0) < 2 and not peer["exited"]:
                yield
        c["exited"] = True
        if any(kind == "x" for kind, _, _ in events):
            raise ProtocolError(f"CTA {ci} exits with a score copy in flight")

    roles = {}
    for ci in range(2):
        roles["setup", ci], roles["prod", ci], roles["qk", ci], roles["pv", ci] = setup(ci), producer(ci), qk(ci), pv(ci)
        for wg in range(2):
            for w in range(WARPS):
                roles["sm", ci, wg, w] = softmax_warp(ci, wg, w)
    idle, steps, pending_exit = 0, 0, {0, 1}
    while roles or events:
        steps += 1
        if abort_at is not None and steps == abort_at[1]:
            ctas[abort_at[0]]["abort"] = True
        for ci in list(pending_exit):
            if not any(key[1] == ci for key in roles):
                pending_exit.discard(ci)
                roles["exit", ci] = exit_sequence(ci)
        pick = rnd.randrange(len(roles) + len(events))
        if pick >= len(roles) and events[pick - len(roles)][0] == "x" and any(x["abort"] for x in ctas):
            working = [k for k in roles if k[0] != "exit"]   # after an abort, copies linger until every role has left
            if working:
                pick = list(roles).index(rnd.choice(working))
        if pick >= len(roles):
            kind, ci, t = events.pop(pick - len(roles))
            c = ctas[ci]
            if kind == "kv":
                c["kv_full"][t % STAGES].arrive()
            elif kind == "s":
                c["s_full"][t & 1].arrive()
            elif kind == "o":
                c["kv_empty"][t % STAGES].arrive()
                c["o_done"][t & 1].arrive()
            else:                                            # a warp's part lands in the peer's buffer t mod XBUFS
                tile, w, p, sb = t
                peer = ctas[1 - ci]
                if peer["exited"] or c["exited"]:
                    raise ProtocolError(f"a copy of tile {tile} lands after a CTA exited")
                take_bytes(peer, tile % XBUFS, places.share[w][p], ("data", tile, w, p), f"tile {tile} part {p} landing")
                for i in places.share[w][p]:
                    c["reading"][sb][i] = False
                peer["x_full"][p][tile % XBUFS].complete_tx(1)
            idle = 0
            continue
        key = list(roles)[pick]
        try:
            next(roles[key])
            idle += 1
        except StopIteration:
            del roles[key]
            idle = 0
        if idle > 50000:
            raise ProtocolError(f"deadlock; roles still running: {sorted(map(str, roles))}")
    assert abort_at is not None or all(c["exited"] for c in ctas)


@pytest.mark.parametrize("parts", [1, 2])
def test_exchange_holds_on_random_interleavings(header, parts):
    places = Places(header, parts)
    for i, segs in enumerate(_layouts(80, 71)):
        run_model(segs, i, places)
    for seed in range(40):
        run_model([1, 1, 1, 2, 2, 3, 3, 7], seed, places)


@pytest.mark.parametrize("parts", [1, 2])
def test_abort_drains_every_part_before_exit(header, parts):
    rng, places = random.Random(72), Places(header, parts)
    for i, segs in enumerate(_layouts(60, 73)):
        run_model(segs, i, places, abort_at=(rng.randrange(2), rng.randrange(1, 4000)))


def _caught(header, parts, places=lambda p: p, **kw):
    n = 0
    for i, segs in enumerate(_layouts(40, 74)):
        try:
            run_model(segs + [3, 5], i, places(Places(header, parts)), **kw)
        except ProtocolError:
            n += 1
    return n


def test_rows_in_a_quarter_of_the_buffer_are_caught(header):
    """Two parts: a warp's quarter holds the scores of other warps.  One part: it is the warp's own share."""
    assert _caught(header, 2, contiguous) > 30
    assert _caught(header, 1, contiguous) == 0


@pytest.mark.parametrize("parts", [1, 2])
@pytest.mark.parametrize("mistake", [dict(xlead=1), dict(xlead=3), dict(epi_shift=1), dict(epi_shift=2), dict(epi_shift=3),
                                     dict(early_push=True)])
def test_planted_mistakes_are_caught(header, parts, mistake):
    assert _caught(header, parts, **mistake) > 0, f"the model did not catch {mistake}"


def test_exit_without_drain_is_caught(header):
    rng, caught, places = random.Random(75), 0, Places(header, 2)
    for i, segs in enumerate(_layouts(100, 76)):
        try:
            run_model(segs + [3, 5], i, places, abort_at=(rng.randrange(2), rng.randrange(1, 4000)), drain=False)
        except ProtocolError:
            caught += 1
    assert caught > 0, "the model did not catch an exit with copies in flight"
