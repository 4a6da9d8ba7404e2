"""Pins of the fp64 definitions in oracle/paged.py: against the pinned attention
oracle, against each other, and the norm's gradient against central differences."""
import numpy as np
import pytest

from oracle import paged


def test_norm_gradient_against_differences():
    rng = np.random.default_rng(1)
    x, w, g = rng.standard_normal((5, 3, 8)), 1 + 0.3 * rng.standard_normal(8), rng.standard_normal((5, 3, 8))
    x[2, 1] *= 1e-3  # a row where eps matters
    eps = 1e-4
    dx, dw = paged.rms_heads_bwd(x, w, g, eps)
    f = lambda a, b: float((g * paged.rms_heads(a, b, eps)).sum())
    for idx in np.ndindex(*x.shape):
        h = 1e-6 * max(1e-3, abs(x[idx]))
        xp, xm = x.copy(), x.copy()
        xp[idx] += h
        xm[idx] -= h
        fd = (f(xp, w) - f(xm, w)) / (2 * h)
        assert abs(fd - dx[idx]) <= 1e-5 * (1 + abs(dx[idx]))
    for i in range(8):
        wp, wm = w.copy(), w.copy()
        wp[i] += 1e-5
        wm[i] -= 1e-5
        assert abs((f(x, wp) - f(x, wm)) / 2e-5 - dw[i]) <= 1e-7 * (1 + abs(dw[i]))


@pytest.mark.parametrize("half", [False, True])
def test_rotation_against_the_oracle(oracle_mod, half):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((1, 9, 3, 16))
    ref = oracle_mod.rope(x, 10000.0, half=half)[0]
    got = paged.rope_at(x[0], np.arange(9), 10000.0, half)
    if half:  # the oracle keeps the features' own order
        ref = np.stack((ref[..., :8], ref[..., 8:]), -1).reshape(ref.shape)
    assert np.max(np.abs(got - ref)) <= 1e-12


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("prefix", [0, 2])
def test_decode_against_the_oracle(oracle_mod, half, prefix):
    """Pages in any order, with or without a shared prefix: rows of the whole-sequence attention."""
    rng = np.random.default_rng(3)
    B, Tq, Hq, Hkv, D, page, base = 3, 2, 4, 2, 8, 4, 10000.0
    lens = [11, 2 + prefix * page, 17]
    P = 16
    perm = rng.permutation(P)
    table = np.full((B, 5), -7)
    shared, at = list(perm[:prefix]), prefix
    kp, vp = rng.standard_normal((P, Hkv, page, D)), rng.standard_normal((P, Hkv, page, D))
    ks, vs = rng.standard_normal((B, 17, Hkv, D)), rng.standard_normal((B, 17, Hkv, D))
    ks[:, :prefix * page], vs[:, :prefix * page] = ks[:1, :prefix * page], vs[:1, :prefix * page]
    for b in range(B):
        need = -(-lens[b] // page)
        table[b, prefix:need] = perm[at:at + need - prefix]
        at += need - prefix
        pages = shared + list(table[b, prefix:need])
        kr = paged.rope_at(ks[b, :lens[b]], np.arange(lens[b]), base, half)
        for j in range(lens[b]):
            kp[pages[j // page], :, j % page] = kr[j]
            vp[pages[j // page], :, j % page] = vs[b, j]
    q = rng.standard_normal((B, Tq, Hq, D))
    o, lse = paged.decode_paged(q, None, kp, vp, table, lens, base, half=half, prefix_pages=shared)
    for b in range(B):
        ro, rl = oracle_mod.decode_fwd(q[b:b + 1], ks[b:b + 1, :lens[b]], vs[b:b + 1, :lens[b]], base, half=half)
        assert np.max(np.abs(o[b] - ro[0])) <= 1e-12 and np.max(np.abs(lse[b] - rl[0])) <= 1e-12


def test_empty_rows():
    rng = np.random.default_rng(4)
    kp, vp = rng.standard_normal((2, 1, 4, 8)), rng.standard_normal((2, 1, 4, 8))
    q = rng.standard_normal((3, 3, 1, 8))
    o, lse = paged.decode_paged(q, None, kp, vp, [[0, 1]] * 3, [0, 1, 5], 100.0)
    assert (o[0] == 0).all() and np.isneginf(lse[0]).all()      # idle slot
    assert (o[1, :2] == 0).all() and np.isneginf(lse[1, 0, :2]).all()
    assert np.allclose(o[1, 2, 0], vp[0, 0, 0])                 # one visible key: its value
    assert np.isfinite(lse[2]).all()


def test_places_of_a_ragged_append():
    assert paged.places([[5, 6], [7, 8], [9, 1]], [3, 0, 2], [0, 2, 2, 3], 4) == [(0, 5, 3, 3), (1, 6, 0, 4), (2, 9, 2, 2)]
