"""Sequences without a tree in a call (tree_len 0): no key of theirs is read, the others are as they would be."""
import numpy as np
import pytest

from test_gpu_tree import BASE, check, i32, nb, setup  # noqa: F401 (nb is a fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Tq,Hq,D,fp32", [(9, 12, 64, False), (32, 16, 64, False), (64, 16, 64, True), (5, 4, 32, True)])
def test_nothing_is_read(nb, Tq, Hq, D, fp32):
    """Contexts of many tiles, every second one without a tree and with a table of wild entries."""
    ctx = [(i * 331) % 3000 for i in range(24)]
    nodes = [0 if i % 2 else 1 + (i * 5) % Tq for i in range(24)]
    s = setup(ctx, nodes, Tq, Hq, 4, D, 16, seed=Tq)
    s["table"][1::2] = i32(np.resize([-1, 2 ** 31 - 1, -2 ** 31, 10 ** 6], (12, s["table"].shape[1])))
    got = nb.attn_decode_tree(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["parents"], tree_len=s["nodes"], rope_base=BASE,
                              o_dtype=torch.float32 if fp32 else torch.bfloat16)
    # the definition gives zeros and -infinity to tokens past tree_len; a bad page that was met would be reported
    check(nb, s, got, False, False)
    assert not got[0][1::2].any() and torch.isneginf(got[1][1::2]).all()


def test_nobody_has_a_tree(nb):
    s = setup([500, 20, 3000], [0, 0, 0], 8, 12, 4, 64, 16, seed=2)
    got = nb.attn_decode_tree(s["q"], s["kp"], s["vp"], torch.full_like(s["table"], -1), s["lens"], s["parents"], tree_len=s["nodes"])
    nb.check_status()
    assert not got[0].any() and torch.isneginf(got[1]).all()
    # a length that is too large is reported all the same
    s["lens"][1] = s["table"].shape[1] * 16 + 1
    nb.attn_decode_tree(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["parents"], tree_len=s["nodes"])
    assert nb.status_of_last_kernels() == -8
