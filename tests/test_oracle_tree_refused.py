"""The definitions of a step in which the plan has no pages for a sequence: with what was granted as its tree's
length, the sequence stays as it was."""
import numpy as np

from oracle import tree

PARENTS = [-1, 0, 1, 1, 2, 3, 4, 5]


def refused_step():
    """Two sequences of 30 and 5 positions, pages of 16, 8 drafted tokens each; the ring is empty."""
    table, held, kv = [[0, 1, -1], [2, -1, -1]], [2, 1], [30, 5]
    return kv, tree.plan(table, [9, 9, 9, 9], held, [0, 0], kv, [8, 8], 16, 16, [PARENTS] * 2)


def test_granted():
    kv, got = refused_step()
    assert got[4] == [30, 13] and got[8] == [0, 8]
    assert got[6] == [-1] * 8 + [2 * 16 + 5 + t for t in range(8)]
    # enough for all, and what is no longer needed given back
    got = tree.plan([[0, 1, -1], [2, 3, -1]], [3, 9, 9, 3], [2, 2], [3, 1], [30, 5], [8, 0], 8, 16)
    assert got[4] == [38, 5] and got[8] == [8, 0]


def test_a_refused_sequence_keeps_its_context():
    kv, p = refused_step()
    rng = np.random.default_rng(1)
    kp, vp = rng.standard_normal((4, 2, 16, 8)), rng.standard_normal((4, 2, 16, 8))
    q = rng.standard_normal((2, 8, 4, 8))
    o, lse, _, _ = tree.decode_tree(q, None, kp, vp, p[0], p[4], [PARENTS] * 2, p[8], 1e4)
    assert (o[0] == 0).all() and np.isneginf(lse[0]).all() and np.isfinite(lse[1]).all()
    for path, m in (([0, 3], 2), ([0, 0], 0), ([7, 1], 2)):
        k2, v2, n = tree.keep(kp, vp, p[0], p[4], p[8], [path, [0, 1]], [m, 2], 16)
        assert n == [30, 7] and (k2 == kp).all() and (v2 == vp).all()
