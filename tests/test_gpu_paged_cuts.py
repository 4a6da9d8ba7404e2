"""Sequences that the paged sweep cuts among blocks, with every number of query rows: their parts go through
the workspace, the counters and the joins of the blocks that finish last (a sequence of at most 8 key
tiles, 16 with D = 32, is never cut). Bounds as in test_gpu_paged, without the allowance for the prefix."""
import pytest

from test_gpu_paged import BASE, EPS, check, nb, setup  # noqa: F401  (nb is a fixture)
from test_gpu_shared_prefix import hold

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

CUTS = [
    # lens, Tq, Hq, Hkv, D, page, norm, half
    ([6000, 17, 2500], 3, 12, 4, 64, 16, True, False),              # 9 rows
    ([4100, 900], 4, 16, 4, 64, 64, False, True),                   # 16 rows
    ([9000, 3, 2700, 5000], 8, 4, 2, 32, 32, True, False),          # 16 rows
    ([5000, 40, 0, 1300], 5, 16, 4, 64, 16, False, False),          # 20 rows
    ([7001, 2600], 16, 4, 2, 32, 128, False, True),                 # 32 rows
    ([4500, 1500, 33], 16, 8, 2, 64, 32, True, False),              # 64 rows
    ([8200, 60, 2400], 33, 2, 2, 32, 64, False, False),             # 33 rows
    ([2900, 4000, 127], 32, 12, 4, 64, 256, False, False),          # 96 rows
    ([6500, 2222], 128, 2, 2, 32, 16, True, True),                  # 128 rows
    ([30000], 128, 1, 1, 64, 64, False, False),                     # 128 rows, more than a tile a block
    ([25000, 12345, 700, 9], 4, 8, 4, 64, 64, True, False),         # 8 rows, several tiles a block
    ([30000, 11000, 400, 0, 5], 10, 8, 4, 64, 16, False, False),    # 20 rows, several tiles a block
]


@pytest.mark.parametrize("case", CUTS, ids=lambda c: "b%d_t%d_%dx%dx%d_p%d" % (len(c[0]), *c[1:6]))
def test_cut_sequences(nb, case):
    lens, Tq, Hq, Hkv, D, page, norm, half = case
    s = setup(lens, Tq, Hq, Hkv, D, page, seed=lens[0] + Tq)
    n = nb.decode_paged_workspace_size(len(lens), Tq, Hq, Hkv, D)
    own = torch.full((n + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    for ws in (None, own):
        call = lambda: nb.attn_decode_paged(s["q"], s["kp"], s["vp"], s["table"], s["lens"],
                                            q_weight=s["qw"] if norm else None, eps=EPS, rope_base=BASE,
                                            o_dtype=torch.float32, rope_half=half, workspace=ws)
        got = call()
        check(nb, s, got, norm, half)
        for _ in range(3):
            again = call()
            assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    assert (own[n:] == 0xFF).all()


PREFIXED = [
    # own lengths past the prefix (None: idle), prefix, Tq, Hq, Hkv, D, page, norm, half
    ([5000, 7, 2600, None], 256, 1, 12, 4, 64, 64, True, False),    # 3 rows
    ([6001, 2900, 40], 512, 2, 8, 2, 32, 32, False, True),          # 8 rows
    ([4000, 1500], 128, 3, 12, 4, 64, 16, False, False),            # 9 rows
    ([3500, 20, 1600], 1024, 5, 8, 2, 64, 128, True, False),        # 20 rows
    ([5200, 2500], 384, 12, 8, 2, 32, 64, False, False),            # 48 rows
    ([3300, 1400], 256, 100, 2, 2, 64, 64, False, False),           # 100 rows
]


@pytest.mark.parametrize("case", PREFIXED, ids=lambda c: "b%d_p%d_t%d_%dx%dx%d" % (len(c[0]), *c[1:6]))
def test_cut_own_parts(nb, case):
    """The sequences' own parts behind a shared prefix are cut too, and joined before the prefix's."""
    own, prefix, Tq, Hq, Hkv, D, page, norm, half = case
    s = setup([0 if x is None else prefix + x for x in own], Tq, Hq, Hkv, D, page, seed=own[0], prefix=prefix)
    call = lambda: nb.attn_decode_paged(s["q"], s["kp"], s["vp"], s["table"], s["lens"], q_weight=s["qw"] if norm else None,
                                        eps=EPS, rope_base=BASE, rope_half=half, o_dtype=torch.float32,
                                        prefix_table=s["ptable"], prefix_len=prefix)
    got = call()
    hold(nb, s, got, prefix, norm, half)
    for _ in range(3):
        again = call()
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
