"""Steps of drafted trees on the GPU with a ring that runs short: a sequence that the plan has no pages for sits the step
out, and no bit of any context changes."""
import numpy as np
import pytest

from oracle import tree
from test_gpu_tree import BASE, PLANS, grow, i32, nb, plan_inputs, setup  # noqa: F401 (nb is a fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", PLANS, ids=lambda c: "b%d_p%d_%s" % (len(c[0]), c[2], "tree" if c[6] else "rows"))
def test_granted(nb, case):
    table, ring, held, span, kv, new, rows, page, parents = plan_inputs(case)
    want = tree.plan(table.tolist(), ring.tolist(), held, span, kv, new, rows, page, parents)
    kw = dict(parents=None if parents is None else i32(parents))
    p = nb.paged_plan(i32(table), i32(ring), i32(held), i32(span), i32(kv), i32(new), rows, page, **kw)
    assert p.new_len.tolist() == want[8] and len(p) == 6
    own, same = i32([-7] * len(kv)), i32(new)  # a buffer of the caller's, and the requested lengths themselves
    p = nb.paged_plan(i32(table), i32(ring), i32(held), i32(span), i32(kv), i32(new), rows, page, new_len_out=own, **kw)
    assert p.new_len is own and own.tolist() == want[8]
    p = nb.paged_plan(i32(table), i32(ring), i32(held), i32(span), i32(kv), same, rows, page, new_len_out=same, **kw)
    assert same.tolist() == want[8]
    for g, w in zip((p.held, p.span, p.kv_len, p.cu_new, p.slots, p.positions), want[2:8]):
        assert g.tolist() == w
    nb.check_status()


def test_granted_where_the_plan_reports(nb):
    """Sequences that cannot be, rows that are not all there, a ring that is none: nothing is granted."""
    def go(kv=(5, 5, 5), new=(20, 20, 20), span=(3, 4), rows=80):
        p = nb.paged_plan(i32([[0, -1], [1, -1], [2, -1]]), i32([9, 9, 9, 3, 4, 5, 6, 9]), i32([1, 1, 1]), i32(span), i32(kv), i32(new),
                          rows, 16)
        return p.new_len.tolist(), nb.status_of_last_kernels()
    assert go() == ([20, 20, 20], 0)
    assert go(kv=(5, -1, 5)) == ([20, 0, 20], -8) and go(new=(20, -3, 20)) == ([20, 0, 20], -8)
    assert go(rows=50) == ([20, 20, 0], -8) and go(span=(8, 1)) == ([0, 0, 0], -8)
    with pytest.raises(ValueError):
        nb.paged_plan(i32([[0]]), i32([0]), i32([1]), i32([0, 0]), i32([3]), i32([1]), 1, 16, new_len_out=i32([0, 0]))


def test_keep_without_a_tree(nb):
    """A tree of no tokens keeps its length and every row, whatever its path holds; the others keep theirs."""
    s = setup([30, 40], [0, 8], 8, 2, 2, 64, 16, seed=7)
    for path, m in (([0, 3], 2), ([0, 0], 0), ([3, 1], 2), ([-5, 2 ** 31 - 1], 2), ([0, 1], -1), ([0, 1], 2 ** 31 - 1)):
        kp, vp = s["kp"].clone(), s["vp"].clone()
        n = nb.kv_keep_paged(kp, vp, s["table"], s["lens"], s["nodes"], i32([path, [0, 1]]), i32([m, 2]))
        nb.check_status()
        assert n.tolist() == [30, 42]
        assert torch.equal(kp.view(torch.int16), s["kp"].view(torch.int16)) and torch.equal(vp.view(torch.int16), s["vp"].view(torch.int16))


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_steps_that_run_short(nb, graph, in_place):
    """Ten steps on a ring that is refilled now and then (a sequence ends): who is refused changes from step to step.  The
    contexts' bits are compared with a copy kept on the host."""
    B, Tq, P, width, page, Hkv, Hq, D = 6, 12, 17, 9, 16, 2, 4, 64
    rng = np.random.default_rng(11)
    g = torch.Generator(device="cuda").manual_seed(11)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    kp = torch.zeros((P, Hkv, page, D), dtype=torch.float16, device="cuda")
    vp = torch.zeros((P, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
    table, held, span = torch.full((B, width), -1, dtype=torch.int32, device="cuda"), i32([0] * B), i32([0, P])
    ring, n, total = torch.randperm(P, generator=g, device="cuda").to(torch.int32), i32([0] * B), i32([0] * B)
    prompt = [int(x) for x in rng.integers(20, 48, B)]
    p = nb.paged_plan(table, ring, held, span, n, i32(prompt), sum(prompt), page, held_out=held, span_out=span)
    assert p.new_len.tolist() == prompt
    nb.kv_append_slots(r(sum(prompt), Hkv, D), r(sum(prompt), Hkv, D), kp, vp, p.slots, p.positions, width * page, rope_base=BASE)
    n.copy_(p.kv_len)
    q, k, v = r(B, Tq, Hq, D), r(B * Tq, Hkv, D), r(B * Tq, Hkv, D)
    parents, new, path, m = i32([[-1] * Tq] * B), i32([0] * B), i32([[0] * Tq] * B), i32([0] * B)
    granted = new if in_place else i32([0] * B)

    def front():
        p = nb.paged_plan(table, ring, held, span, n, new, B * Tq, page, parents=parents, kv_len_out=total, held_out=held, span_out=span,
                          new_len_out=granted)
        nb.kv_append_slots(k, v, kp, vp, p.slots, p.positions, width * page, rope_base=BASE)
        return nb.attn_decode_tree(q, kp, vp, table, total, parents, tree_len=granted, rope_base=BASE)

    back = lambda: nb.kv_keep_paged(kp, vp, table, total, granted, path, m, kv_len_out=n)
    if graph:
        front(), back()  # nothing is added: tables of the shape exist before the capture
        gf, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(gf):
            out = front()
        with torch.cuda.graph(gb):
            back()

    def rows(b, lo, hi):
        t = table.tolist()[b]
        at = [(t[j // page], j % page) for j in range(lo, hi)]
        pg, of = torch.tensor([a[0] for a in at], device="cuda"), torch.tensor([a[1] for a in at], device="cuda")
        return [x.view(torch.int16)[pg, :, of].cpu() if at else torch.zeros((0, Hkv, D), dtype=torch.int16) for x in (kp, vp)]

    lens = list(prompt)
    mine = [rows(b, 0, lens[b]) for b in range(B)]
    refused = both = 0
    for step in range(10):
        if step in (5, 8):  # a sequence ends, its pages are free with the next plan
            b = step % B
            lens[b], mine[b] = 0, rows(b, 0, 0)
            n[b] = 0
        size = [int(x) for x in rng.integers(1, Tq + 1, B)]
        trees = [grow(rng, Tq) for _ in range(B)]
        new.copy_(i32(size))
        parents.copy_(i32(trees))
        for x in (q, k, v):
            x.copy_(r(*x.shape))
        want = tree.plan(table.tolist(), ring.tolist(), held.tolist(), span.tolist(), lens, size, B * Tq, page, trees)
        if graph:
            gf.replay()
        else:
            out = front()
        nb.check_status()
        got = granted.tolist()
        assert got == want[8] and total.tolist() == want[4]
        for b in range(B):  # no tree: no output
            if got[b] == 0:
                assert (out[0][b] == 0).all() and torch.isneginf(out[1][b]).all()
            else:
                assert torch.isfinite(out[1][b, :, :got[b]]).all()
        # a program that accepts without a look at what was granted: paths by the requested sizes, one of them empty
        lines = [tree.ancestors(t, int(rng.integers(0, s)))[::-1] for t, s in zip(trees, size)]
        lines[step % B] = []
        moved = [[x[lines[b]] for x in rows(b, lens[b], lens[b] + got[b])] if got[b] else None for b in range(B)]
        path.copy_(i32([x + [0] * (Tq - len(x)) for x in lines]))
        m.copy_(i32([len(x) for x in lines]))
        if graph:
            gb.replay()
        else:
            back()
        nb.check_status()
        for b in range(B):
            if got[b]:
                lens[b] += len(lines[b])
                mine[b] = [torch.cat(x) for x in zip(mine[b], moved[b])]
        assert n.tolist() == lens
        for b in range(B):
            for x, y in zip(rows(b, 0, lens[b]), mine[b]):
                assert torch.equal(x, y)
        refused += got.count(0)
        both += 0 < got.count(0) < B
        first, count = span.tolist()
        free, ring_now, tables, helds = [], ring.tolist(), table.tolist(), held.tolist()
        assert sorted([ring_now[(first + j) % P] for j in range(count)] + [x for b in range(B) for x in tables[b][:helds[b]]]) == list(range(P))
    assert refused >= 5 and both >= 3
