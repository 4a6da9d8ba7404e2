"""CPU checks: lengths that the plan and keep write may not lie on what their kernels still read."""
import pytest

from test_abi_tree import KEEP, call, libne, mem  # noqa: F401 (fixtures)
from test_abi_tree_refused import PLAN


def test_keep(libne, mem):
    """B = 4: the arrays read, each in a place of its own, of 4, 4, 4, 4 x 5 and 4 x 3 entries."""
    p = mem[1]
    n = dict(len=4, nodes=4, count=4, path=20, table=12)
    at = {name: p + 1024 * (i + 1) for i, name in enumerate(n)}
    good = dict(at, kp=p, vp=p, out=p + 8192, B=4, tokens=0, width=5, Hkv=2, D=32, page=16, P=4, tw=3, stride=1024, stream=None)
    f = lambda **c: call(libne.ne_attn_kv_keep_paged, KEEP, good, **c)
    for name, k in n.items():
        for out in (at[name], at[name] + 4 * (k - 1), at[name] - 12):
            assert f(out=out) == -1, name
    assert f(out=at["nodes"], nodes=None, tokens=5) != -1  # no array there


@pytest.mark.parametrize("which", ["len_o", "new_o"])
def test_plan(libne, mem, which):
    p = mem[1]
    n = dict(len=4, ring=7, table=12, parents=4 * 6)
    at = {name: p + 1024 * (i + 1) for i, name in enumerate(n)}
    good = dict(at, new=p + 16384, held=p + 17408, span=p + 18432, held_o=p + 20480, span_o=p + 20544, len_o=p + 8192, new_o=p + 8256, cu=p + 24576, slots=p + 28672,
                pos=p + 32768, N=5, B=4, Tq=6, page=16, P=7, width=3, pstride=6, stream=None)
    f = lambda **c: call(libne.ne_attn_paged_plan_ex, PLAN, good, **c)
    for name, k in n.items():
        for out in (at[name], at[name] + 4 * (k - 1), at[name] - 12):
            assert f(**{which: out}) == -1, name
    assert f(new_o=p + 8192 + 4) == -1                 # one output on the other
    assert f(**{which: at["parents"]}, parents=None) != -1
    for fine in (p + 16384, p + 17408):                # the requested lengths, the pages held: read before
        assert f(**{which: fine}) != -1
    assert f(new_o=None) != -1
