"""The persistent forward on many short sequences: a head of one query tile whose group
has no partner for it is an item of its own, and a block then runs several such
items one after another, where only one of its two units reads the key/value stages.
"""
import pytest

import _harness as H
from causal_gqa_attention_flashattention_gb300 import inputs

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# B, T, Hq, Hkv, D: 800 to 1,536 lone items, 5 to 10 to a block of 152
SHAPES = [(160, 100, 5, 5, 64), (128, 128, 12, 12, 32), (260, 40, 12, 4, 64)]


@pytest.fixture(scope="module")
def nb():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_gqa_attention_flashattention_gb300 import binding
    binding.lib()
    return binding


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_items_of_one_unit(nb, oracle_mod, shape):
    B, T, Hq, Hkv, D = shape
    lists = nb.fwd_schedule(B, Hkv, Hq // Hkv, (T + 127) // 128, 152)
    assert max(sum(u1 is None for _, _, u1 in l) for l in lists) > 4
    x = H.make(*shape, seed=sum(shape))
    q, k, v = (H.to_device(x[n + "_bits"]) for n in ("q", "k", "v"))
    ref_o, ref_l = oracle_mod.attn_fwd(x["q"], x["k"], x["v"])
    o, lse = nb.attn_fwd(q, k, v)
    nb.check_status()
    rel, mx = H.errors(H.to_f64(o), ref_o)
    assert rel <= H.REL_L2_TOL and mx <= H.MAX_ABS_TOL, (rel, mx)
    assert H.errors(lse.double().cpu().numpy(), ref_l)[1] <= H.LSE_ABS_TOL
    again = nb.attn_fwd(q, k, v)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


def test_items_of_one_unit_fp8(nb, oracle_mod):
    shape = (160, 100, 5, 5, 64)
    x = H.make(*shape, seed=17)
    q, k, v = (H.to_device(x[n + "_bits"]) for n in ("q", "k", "v"))
    o, lse = nb.attn_fwd(q, k, v, fp8=True)
    nb.check_status()
    floor, ref_o, ref_l = H.fp8_floor(oracle_mod, x, inputs.ROPE_BASE)
    b_rel, b_mx, b_lse = H.fp8_bounds(floor)
    rel, mx = H.errors(H.to_f64(o), ref_o)
    assert rel <= b_rel and mx <= b_mx and H.errors(lse.double().cpu().numpy(), ref_l)[1] <= b_lse
