"""Model check of what the decode kernels' protocol has gained since its first model.

The model of test_decode_protocol.py is extended where the kernels differ:
  * FP8: P·V of a tile is issued as soon as its own inputs are ready;
  * a row's epilogue crosses through the tile's own exchange buffer, between
    its last P·V and the warpgroup's next staging: nothing may land there;
  * windowed: the P·V warp clears masked tokens in the page stage once the
    tile's scores are complete, before it issues P·V; a softmax warpgroup
    publishes the last tile whose scores it has seen complete, since a phase of
    the score barriers may be two behind there;
  * the set-up's cluster barrier is split: a CTA pushes scores only after both
    CTAs have arrived.
Each part comes with a planted mistake that must be caught.
"""
import os
import random

import pytest

import test_decode_protocol as base
from test_decode_protocol import ProtocolError, _layouts


def _model():
    """run_model of the first model with the differences put in."""
    src = open(os.path.splitext(base.__file__)[0] + ".py").read()
    src = src[src.index("STAGES = 4"):src.index("def _layouts(")]

    def put(old, new):
        nonlocal src
        assert src.count(old) == 1, (src.count(old), old)
        src = src.replace(old, new)

    put("abort_at=None, drain=True):", "abort_at=None, drain=True, epi_shift=0, clear=False, clear_waits=True, "
        "clear_by_phase=False, early_push=False):")
    put("            if fp8 and t + 2 < G:\n", "            if False:\n")
    # the epilogue through the exchange buffer
    put("                if not (yield from wait(c, lambda: bar.test(k))):\n"
        "                    return\n"
        "                c[\"o_free\"].arrive(per_warp)\n",
        "                if not (yield from wait(c, lambda: bar.test(k))):\n"
        "                    return\n"
        "                eb = (t + epi_shift) % XBUFS\n"
        "                for _ in range(4):\n"
        "                    if c['xbuf'][eb][w] is not None and c['xbuf'][eb][w][0] == 'data':\n"
        "                        raise ProtocolError(f'epilogue of tile {t} over scores of {c[\"xbuf\"][eb][w]}')\n"
        "                    if c['reading'][eb][w]:\n"
        "                        raise ProtocolError(f'epilogue of tile {t} over a copy in flight')\n"
        "                    yield\n"
        "                c[\"o_free\"].arrive(per_warp)\n")
    # the clearing of masked tokens
    put("    def pv(ci):\n        c = ctas[ci]\n        for t in range(G):\n",
        "    def pv(ci):\n        c = ctas[ci]\n        for t in range(G):\n"
        "            if clear:\n"
        "                if clear_by_phase:\n"
        "                    b_, k_ = s_full_bar(c, t)\n"
        "                    if not (yield from wait(c, lambda: b_.test(k_))):\n"
        "                        return\n"
        "                elif clear_waits:\n"
        "                    if not (yield from wait(c, lambda: c['scored'][t & 1] >= t)):\n"
        "                        return\n"
        "                if s_full_bar(c, t)[0].phase < s_full_bar(c, t)[1] + 1:\n"
        "                    raise ProtocolError(f'tile {t} cleared while QK^T may read it')\n"
        "                if c['kv_empty'][t % n_stages].phase > t // n_stages:\n"
        "                    raise ProtocolError(f'tile {t} cleared after its stage was handed back')\n"
        "                yield\n")
    put("            c[\"s_free\"].arrive(per_warp)\n            # stage this",
        "            if w == 0:\n                c['scored'][wg] = t\n"
        "            c[\"s_free\"].arrive(per_warp)\n            # stage this")
    put("qk_issued=-1,\n", "qk_issued=-1, scored=[-1, -1], arrived=False,\n")
    # the split set-up barrier
    put("    def producer(ci):\n        c = ctas[ci]\n",
        "    def setup(ci):\n        for _ in range(rnd.randrange(60)):\n            yield\n        ctas[ci]['arrived'] = True\n\n"
        "    def producer(ci):\n        c = ctas[ci]\n        while not c['arrived']:\n            yield\n")
    put("        if wg == 0:\n            c[\"o_free\"].arrive(per_warp)\n",
        "        while not c['arrived']:\n            yield\n        if wg == 0:\n            c[\"o_free\"].arrive(per_warp)\n")
    put("            # stage this row block's scores and push them to the peer\n",
        "            if not early_push:\n                while not ctas[1 - ci]['arrived']:\n                    yield\n"
        "            if not ctas[1 - ci]['arrived']:\n                raise ProtocolError('scores pushed before the peer was set up')\n"
        "            # stage this row block's scores and push them to the peer\n")
    put("        roles[(\"prod\", ci)] = producer(ci)\n", "        roles[(\"setup\", ci)] = setup(ci)\n        roles[(\"prod\", ci)] = producer(ci)\n")
    space = {"random": random}
    exec(compile(src, "window_model", "exec"), space)
    return space["run_model"], space["ProtocolError"]


run_model, ModelError = _model()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("clear", [False, True])
def test_protocol_holds_on_random_interleavings(fp8, clear):
    for i, segs in enumerate(_layouts(120, 51)):
        run_model(segs, seed=i, fp8=fp8, clear=clear)
    for seed in range(60):
        run_model([1, 1, 1, 1, 2, 2, 3, 3, 11], seed, fp8=fp8, clear=clear)


@pytest.mark.parametrize("fp8", [False, True])
def test_abort_drains_every_copy_before_exit(fp8):
    rng = random.Random(52)
    for i, segs in enumerate(_layouts(120, 53)):
        run_model(segs, seed=i, fp8=fp8, clear=True, abort_at=(rng.randrange(2), rng.randrange(200, 3000)))


@pytest.mark.parametrize("mistake", [dict(epi_shift=1), dict(epi_shift=2), dict(epi_shift=3), dict(clear=True, clear_waits=False),
                                     dict(clear=True, clear_by_phase=True), dict(early_push=True)])
def test_planted_mistakes_are_caught(mistake):
    caught = 0
    for i, segs in enumerate(_layouts(80, 54)):
        try:
            run_model(segs + [1, 1, 3], seed=i, **mistake)
        except ModelError:
            caught += 1
    assert caught > 0, f"the model did not catch {mistake}"
