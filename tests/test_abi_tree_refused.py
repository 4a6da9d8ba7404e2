"""CPU checks of ne_attn_paged_plan_ex: the plan's refusals with the output of what was granted, which may be missing
or the requested lengths themselves."""
from test_abi_tree import call, libne, mem  # noqa: F401 (fixtures)

PLAN = "table ring held span len new parents held_o span_o len_o new_o cu slots pos N B Tq page P width pstride stream"


def test_plan_ex(libne, mem):
    p = mem[1]
    good = dict(table=p, ring=p, held=p, span=p, len=p, new=p + 128, parents=p, held_o=p, span_o=p, len_o=p + 64, new_o=p + 256, cu=p,
                slots=p, pos=p, N=5, B=2, Tq=4, page=16, P=4, width=3, pstride=4, stream=None)
    f = lambda **c: call(libne.ne_attn_paged_plan_ex, PLAN, good, **c)
    for name in "table ring held span len new held_o span_o len_o cu slots pos".split():
        assert f(**{name: None}) == -1
    assert f(new_o=p + 258) == -2
    for new_o in (None, p + 128):  # what follows is found all the same
        assert f(new_o=new_o, page=8) == -3 and f(new_o=new_o, B=0) == -1 and f(new_o=new_o, slots=p + 2) == -2
