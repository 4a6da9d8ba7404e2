"""A NaN in a query of the paged decode: its row's o and lse are NaN (an lse of -infinity would say that it
saw no key), the other rows keep their results bit by bit."""
import pytest

from test_gpu_paged import BASE, nb, setup  # noqa: F401  (nb is a fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

CASES = [
    # lens, prefix, Tq, Hq, Hkv, D: 3, 12, 40 and 16 query rows a sequence; one cut among blocks; shared prefixes
    ([300, 33, 0], 0, 1, 12, 4, 64),
    ([300, 6000], 0, 3, 8, 2, 32),
    ([300, 70], 0, 10, 8, 2, 64),
    ([9000, 17], 0, 4, 4, 1, 64),
    ([300, 257, 0], 256, 1, 12, 4, 64),
    ([700, 520], 512, 6, 8, 2, 32),
]


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "b%d_p%d_t%d_%dx%dx%d" % (len(c[0]), *c[1:]))
def test_nan_in_a_query(nb, case, norm):
    lens, prefix, Tq, Hq, Hkv, D = case
    s = setup(lens, Tq, Hq, Hkv, D, 32, seed=3, prefix=prefix)
    call = lambda q: nb.attn_decode_paged(q, s["kp"], s["vp"], s["table"], s["lens"], q_weight=s["qw"] if norm else None,
                                          rope_base=BASE, prefix_table=s["ptable"], prefix_len=prefix)
    want = call(s["q"])
    q = s["q"].clone()
    q[1, Tq - 1, Hq - 2, 5] = float("nan")
    o, lse = call(q)
    nb.check_status()
    assert torch.isnan(o[1, Tq - 1, Hq - 2]).all() and torch.isnan(lse[1, Hq - 2, Tq - 1])
    o[1, Tq - 1, Hq - 2], lse[1, Hq - 2, Tq - 1] = want[0][1, Tq - 1, Hq - 2], want[1][1, Hq - 2, Tq - 1]
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
