"""Plain forms of the draft-tree operators, written row by row."""
import random

import numpy as np


def tree(seed, n, roots=3, reach=6):
    """Parents of n nodes in topological order."""
    r = random.Random(seed)
    return [-1 if i < roots or i == 0 else r.randrange(max(0, i - reach), i) for i in range(n)]


def path(parents, i):
    p = []
    while i >= 0:
        p.append(i)
        i = parents[i]
    return p[::-1]


def words_of(nodes, words):
    """The mask words (as int64 values) of a set of nodes."""
    out = [0] * words
    for k in nodes:
        out[k // 64] |= 1 << (k % 64)
    return [x - (1 << 64) if x >> 63 else x for x in out]


def masks(trees, words):
    rows = [words_of(path(t, i), words) for t in trees for i in range(len(t))]
    return np.array(rows, dtype=np.int64).reshape(len(rows), words)


def seen(n0, i, row):
    """The positions that node i (mask words `row`) sees, of a sequence of n0 tokens and its nodes."""
    return list(range(n0)) + [n0 + k for k in range(min(i + 1, 64 * len(row))) if int(row[k // 64]) >> (k % 64) & 1]


def kept(row, accepted):
    return [k for k in range(accepted + 1) if int(row[k // 64]) >> (k % 64) & 1] if accepted >= 0 else []
