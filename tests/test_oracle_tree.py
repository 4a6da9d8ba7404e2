"""Pins of the definitions in oracle/tree.py: by hand, and a chain of tokens against the pinned decode."""
import numpy as np

from oracle import paged, tree


def test_ancestors():
    parents = [-1, 0, 0, 1, -1, 4, 9, -5]
    assert [tree.ancestors(parents, t) for t in range(8)] == [[0], [1, 0], [2, 0], [3, 1, 0], [4], [5, 4], [6], [7]]


def test_plan_by_hand():
    table = [[7, 0, 0], [1, 2, 3], [0, 0, 0], [0, 0, 0]]
    ring = [9, 8, 4, 5]
    # sequence 0 needs one page more, 1 gives two back, 2 needs two (the ring has one left), 3 none of its own
    got = tree.plan(table, ring, [1, 3, 0, 0], [3, 2], [3, 2, 0, 0], [3, 1, 5, 0], 11, 4, [[-1, 0, 0, 1, 1]] * 4)
    assert got[0] == [[7, 5, 0], [1, 2, 3], [0, 0, 0], [0, 0, 0]]
    assert got[1] == [9, 2, 3, 5]               # the free page 9 stays, 2 and 3 follow it
    assert got[2] == [2, 1, 0, 0] and got[3] == [0, 3]
    assert got[4] == [6, 3, 0, 0] and got[5] == [0, 3, 4, 9, 9]
    assert got[6] == [31, 20, 21, 6] + [-1] * 7
    assert got[7] == [3, 4, 4, 2, 0, 1, 1, 2, 2, 0, 0]


def test_a_chain_is_the_causal_decode():
    rng = np.random.default_rng(1)
    kp, vp = rng.standard_normal((8, 2, 16, 8)), rng.standard_normal((8, 2, 16, 8))
    table, lens = [[3, 1, 5], [0, 7, 2]], [40, 5]
    q = rng.standard_normal((2, 5, 4, 8))
    o, lse, _, _ = tree.decode_tree(q, None, kp, vp, table, lens, [[-1, 0, 1, 2, 3]] * 2, [5, 5], 1e4)
    ro, rl = paged.decode_paged(q, None, kp, vp, table, lens, 1e4)
    assert np.max(np.abs(o - ro)) <= 1e-14 and np.max(np.abs(lse - rl)) <= 1e-14


def test_siblings_do_not_see_each_other():
    """Every path of a tree is the chain of its own tokens, moved behind the context by keep."""
    rng = np.random.default_rng(2)
    page, D, ctx, parents = 4, 8, 6, [-1, 0, 0, 1, 2, 2]
    kp, vp = rng.standard_normal((5, 2, page, D)), rng.standard_normal((5, 2, page, D))
    table, q = [[4, 0, 3]], rng.standard_normal((1, 6, 4, D))
    o, lse, _, _ = tree.decode_tree(q, None, kp, vp, table, [ctx + 6], [parents], [6], 1e4)
    for t in range(6):
        line = tree.ancestors(parents, t)[::-1]
        k2, v2, n = tree.keep(kp, vp, table, [ctx + 6], [6], [line], [len(line)], page)
        assert n == [ctx + len(line)]
        ro, rl = paged.decode_paged(q[:, t:t + 1], None, k2, v2, table, n, 1e4)
        assert np.max(np.abs(o[:, t] - ro[:, 0])) <= 1e-14 and np.max(np.abs(lse[:, :, t] - rl[:, :, 0])) <= 1e-14


def test_rows_without_keys():
    rng = np.random.default_rng(3)
    kp, vp = rng.standard_normal((2, 1, 4, 8)), rng.standard_normal((2, 1, 4, 8))
    q = rng.standard_normal((3, 3, 1, 8))
    o, lse, _, _ = tree.decode_tree(q, None, kp, vp, [[0, 1]] * 3, [0, 2, 1], [[-1, 0, 0]] * 3, [3, 3, 1], 1e4)
    assert (o[:2] == 0).all() and np.isneginf(lse[:2]).all()       # idle, and shorter than its tree
    assert np.allclose(o[2, 0, 0], vp[0, 0, 0]) and (o[2, 1:] == 0).all()
