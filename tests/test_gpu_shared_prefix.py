"""Decode over a shared prefix held to the precision of the same call without one, and with row
maxima that keep growing from key tile to key tile.

Bounds: those of the decode without a prefix (test_gpu_paged: q as two fp16 parts, the weights as
two bf16 parts, so 2^-17 of each) with one more term: a tensor-core sum of the weights times the values
takes 16 keys of one part at a time, at most prefix / 8 products into one fp32 accumulator, each
of them off by at most one unit 2^-23 of sum_j p_j |v_j|:
  |o error| <= (2 d + 2^-14 + 2^-23 prefix / 8) A.
One bf16 part alone is off by up to 2^-9 of a weight: ten times as much where one or two keys hold most
of a row's weight, as they do with logits of standard deviation 4.
"""
import numpy as np
import pytest

import _harness as H
from oracle import paged
from test_gpu_paged import BASE, EPS, nb, setup  # noqa: F401  (nb is a fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def hold(nb, s, got, prefix, norm=False, half=False):
    o, lse = got
    nb.check_status()
    ro, rl, A, M = paged.decode_paged(s["fq"], s["fqw"] if norm else None, s["fk"], s["fv"], s["ftable"], s["flens"], BASE,
                                      EPS, half, s["fptable"], bounds=True)
    d = M * (2.0 ** -18 + 2.0 ** -21)
    tol = (2 * d[..., None] + 2.0 ** -14 + 2.0 ** -23 * prefix / 8) * A
    err = np.abs(H.to_f64(o) - ro)
    assert (err <= tol + 1e-37).all(), float((err / (tol + 1e-37)).max())
    gl = lse.cpu().numpy().astype(np.float64)
    empty = np.isneginf(rl)
    assert (np.isneginf(gl) == empty).all()
    ltol = np.moveaxis(d, 1, 2) + 2.0 ** -14 + 2.0 ** -22 * np.abs(np.where(empty, 0, rl))
    assert (np.abs(np.where(empty, 0, gl) - np.where(empty, 0, rl)) <= ltol).all()


def decode(nb, s, prefix, **kw):
    return nb.attn_decode_paged(s["q"], s["kp"], s["vp"], s["table"], s["lens"], eps=EPS, rope_base=BASE,
                                o_dtype=torch.float32, prefix_table=s["ptable"], prefix_len=prefix, **kw)


CASES = [
    # own lengths past the prefix (None: idle), prefix, Tq, Hq, Hkv, D, page, norm, half
    ([1, 1], 16, 1, 4, 2, 32, 16, False, False),
    ([1, None, 17, 129], 256, 1, 12, 4, 64, 64, False, False),
    ([5, 2, 70], 128, 2, 6, 3, 64, 32, True, True),
    ([2, 40, 9, 8], 80, 1, 12, 4, 64, 16, False, True),
    ([(i * 13) % 90 + 1 for i in range(70)], 1024, 1, 12, 4, 64, 16, False, False),
    ([3, 4, 500, 9], 768, 3, 8, 1, 32, 256, False, False),
    ([600, 12, 77], 128, 12, 8, 2, 64, 16, False, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "b%d_p%d_t%d_%dx%dx%d" % (len(c[0]), c[1], c[2], c[3], c[4], c[5]))
def test_precision(nb, case):
    """Logits of standard deviation 4: a few keys hold most of a row's weight."""
    own, prefix, Tq, Hq, Hkv, D, page, norm, half = case
    lens = [0 if x is None else prefix + x for x in own]
    s = setup(lens, Tq, Hq, Hkv, D, page, seed=prefix + Tq, prefix=prefix, scale=2.0)
    got = decode(nb, s, prefix, q_weight=s["qw"] if norm else None, rope_half=half)
    hold(nb, s, got, prefix, norm, half)


@pytest.mark.parametrize("shape", [(20, 4, 16, 8, 64, 4096), (9, 1, 32, 8, 32, 8192), (3, 5, 4, 4, 64, 1024)],
                         ids=lambda c: "b%d_t%d_%dx%dx%d_p%d" % c)
def test_growing_maxima(nb, shape):
    """Keys of seven times 3 more standard deviations from tile to tile, over and over: a row's maximum
    grows by more than 2^8 inside nearly every block's stretch, and O is rescaled."""
    B, Tq, Hq, Hkv, D, prefix = shape
    page = 64
    s = setup([prefix + 3 + 7 * b for b in range(B)], Tq, Hq, Hkv, D, page, seed=77, prefix=prefix)
    fk = s["fk"]
    for i, pg in enumerate(s["fptable"]):
        fk[pg] *= 1 + 3 * ((i * page // 128) % 8)
    k16 = fk.astype(np.float16)
    s["kp"], s["fk"] = torch.from_numpy(k16).cuda(), k16.astype(np.float64)
    got = decode(nb, s, prefix)
    hold(nb, s, got, prefix)
    again = decode(nb, s, prefix)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def test_same_with_and_without(nb):
    """The same pages in every sequence's own table: one bound holds both calls."""
    prefix, page = 512, 64
    s = setup([prefix + 1 + 3 * i for i in range(40)], 1, 12, 4, 64, page, seed=4, prefix=prefix, scale=2.0)
    one = decode(nb, s, prefix)
    table = s["table"].clone()
    table[:, :prefix // page] = s["ptable"]
    two = nb.attn_decode_paged(s["q"], s["kp"], s["vp"], table, s["lens"], eps=EPS, rope_base=BASE, o_dtype=torch.float32)
    hold(nb, s, one, prefix)
    hold(nb, s, two, prefix)


MANY = [
    # own lengths, prefix, Tq, Hq, Hkv, D, page: more (head, pair of row tiles)s than blocks take the prefix
    ([3, 70, 900], 640, 1, 200, 200, 32, 64),
    ([5, 1], 400, 2, 180, 180, 64, 16),
    ([(i * 7) % 60 + 4 for i in range(70)], 256, 4, 80, 40, 32, 128),     # 560 rows a head: 5 row tiles
    ([4000, 3900, 17], 128, 1, 48, 24, 64, 64),
]


@pytest.mark.parametrize("case", MANY, ids=lambda c: "b%d_p%d_t%d_%dx%dx%d" % (len(c[0]), *c[1:6]))
def test_many_heads(nb, case):
    """The prefix's tiles of all heads lie in one line: a block has parts of several heads and row tiles."""
    own, prefix, Tq, Hq, Hkv, D, page = case
    s = setup([prefix + x for x in own], Tq, Hq, Hkv, D, page, seed=prefix, prefix=prefix, scale=1.5)
    got = decode(nb, s, prefix)
    hold(nb, s, got, prefix)
    for _ in range(3):
        again = decode(nb, s, prefix)
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
