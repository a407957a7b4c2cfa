"""CPU oracle of eviction by accumulated attention weight -- test infrastructure only.

``block_weights``: the softmax weight that a decode query gives to every selected block and its
own block, summed over tokens and heads, in fp64.  ``kept_blocks``: which blocks of a sequence
stay, in the order of the definition (sort by weight, the lower block among equals).

parity pins: tests/test_oracle_evict.py.
"""
from __future__ import annotations

import numpy as np

BLOCK = 4


def block_weights(q, keys, length, blocks):
    """q [24][128]; keys [2][length][128] (one sequence); blocks: the selected blocks, all before
    the own block (length - 1) // 4.  Returns fp64 weights of blocks + [own block], in order."""
    q = np.asarray(q, dtype=np.float64)
    keys = np.asarray(keys, dtype=np.float64)
    own = (length - 1) // BLOCK
    blocks = [int(x) for x in blocks] + [own]
    w = np.zeros(len(blocks))
    group = q.shape[0] // keys.shape[0]
    for h in range(q.shape[0]):
        kh = keys[h // group]
        x = [kh[BLOCK * b: min(BLOCK * b + BLOCK, length)] @ q[h] / np.sqrt(q.shape[1])
             for b in blocks]
        top = max(y.max() for y in x)
        e = [np.exp(y - top).sum() for y in x]
        w += np.array(e) / sum(e)
    return w


def kept_blocks(mass, nb, keep, sinks, recent):
    """Old indices, ascending, of the blocks that a sequence of nb complete blocks keeps."""
    if nb <= keep:
        return list(range(nb))

    def weight(i):
        x = float(mass[i])
        return -np.inf if np.isnan(x) else x + 0.0

    middle = sorted(range(sinks, nb - recent), key=lambda i: (-weight(i), i))
    return sorted(list(range(sinks)) + middle[: keep - sinks - recent]
                  + list(range(nb - recent, nb)))
