"""The drafted trees' calls at the ends of their ranges, together, captured, and on shared buffers; definitions and
bounds as in test_gpu_tree.py."""
import numpy as np
import pytest

from oracle import tree
from test_gpu_tree import BASE, check, i32, nb, plan_inputs, setup  # noqa: F401 (nb is a fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def run_plan(nb, case):
    table, ring, held, span, kv, new, rows, page, parents = plan_inputs(case)
    want = tree.plan(table.tolist(), ring.tolist(), held, span, kv, new, rows, page, parents)
    t, r = i32(table), i32(ring)
    got = nb.paged_plan(t, r, i32(held), i32(span), i32(kv), i32(new), rows, page, parents=None if parents is None else i32(parents))
    nb.check_status()
    for g, w in zip((t, r, got.held, got.span, got.kv_len, got.cu_new, got.slots, got.positions), want):
        assert g.tolist() == w


def test_plan_without_rows(nb):
    """Nothing new: the pages that were given too many come back."""
    run_plan(nb, ([40, 0, 16, 17], [0] * 4, 16, 1, 2, 0, False))
    t, r = i32([[0, 1, 2]]), i32([9, 9, 9, 9])
    p = nb.paged_plan(t, r, i32([3]), i32([2, 0]), i32([0]), i32([0]), 0, 16)
    nb.check_status()
    assert r.tolist() == [2, 9, 0, 1] and p.span.tolist() == [2, 3] and p.held.tolist() == [0] and p.slots.numel() == 0
    # a row that has no room is refused
    p = nb.paged_plan(i32([[0]]), i32([0]), i32([1]), i32([0, 0]), i32([3]), i32([1]), 0, 16)
    assert nb.status_of_last_kernels() == -8 and p.kv_len.tolist() == [3]
    with pytest.raises(ValueError):
        nb.paged_plan(i32([[0]]), i32([0]), i32([1]), i32([0, 0]), i32([3]), i32([1]), -1, 16)


@pytest.mark.parametrize("rows", [4096, 4097])
def test_plan_on_both_sides_of_the_second_launch(nb, rows):
    """The same plan with its rows written by one block and by many: refused sequences, trees, padding."""
    kv = [(i * 13) % 90 for i in range(70)]
    run_plan(nb, (kv, [64 - i % 30 if i % 7 else 0 for i in range(70)], 16, -9, 1, rows - sum(64 - i % 30 if i % 7 else 0 for i in range(70)), True))


def test_most_sequences(nb):
    """2048 sequences, the most there may be, idle ones and empty trees among them."""
    ctx = [None if i % 11 == 5 else (i * 7) % 150 for i in range(2048)]
    for D in (32, 64):
        s = setup(ctx, [i % 4 for i in range(2048)], 3, 2, 1, D, 16, seed=D)
        check(nb, s, nb.attn_decode_tree(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["parents"], tree_len=s["nodes"],
                                         rope_base=BASE), False, False)


@pytest.mark.parametrize("fp32", [False, True])
def test_many_row_tiles(nb, fp32):
    """64 tokens of 13 heads on one: 832 rows, pairs of row tiles and a last one of a single tile; sequences of a tile or
    two, so that a block's segments follow each other at once with one and two row tiles in turn."""
    ctx = [(i * 5) % 120 for i in range(40)]
    s = setup(ctx, [64 - (i * 9) % 40 for i in range(40)], 64, 13, 1, 64, 32, seed=21)
    check(nb, s, nb.attn_decode_tree(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["parents"], tree_len=s["nodes"], rope_base=BASE,
                                     o_dtype=torch.float32 if fp32 else torch.bfloat16), False, False)
    s = setup(ctx, [20 - i % 10 for i in range(40)], 20, 13, 1, 64, 32, seed=22)  # 260 rows: two tiles and four rows
    check(nb, s, nb.attn_decode_tree(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["parents"], tree_len=s["nodes"], rope_base=BASE,
                                     o_dtype=torch.float32 if fp32 else torch.bfloat16), False, False)


@pytest.mark.parametrize("Tq,Hq", [(3, 4), (20, 16), (33, 12)])
def test_short_sequences_in_a_row(nb, Tq, Hq):
    """Many sequences of one or two tiles for every block: slots, barriers and the groups' turns over many segments."""
    ctx = [(i * 29) % 230 for i in range(700)]
    s = setup(ctx, [Tq - i % min(Tq, 5) for i in range(700)], Tq, Hq, 4, 64, 16, seed=Tq)
    check(nb, s, nb.attn_decode_tree(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["parents"], tree_len=s["nodes"], rope_base=BASE), False,
          False)


def test_no_page_of_its_own(nb):
    """Two sequences that share their context's pages, and one table row given twice."""
    s = setup([96, 96], [4, 4], 4, 4, 2, 64, 32, seed=31)
    table = s["table"].clone()
    s["table"] = table[:1].repeat(2, 1)
    for name in ("q", "parents", "nodes", "lens"):
        s[name] = s[name][:1].repeat(2, *[1] * (s[name].dim() - 1))
    o, lse = nb.attn_decode_tree(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["parents"], rope_base=BASE)
    nb.check_status()
    assert torch.equal(o[0], o[1]) and torch.equal(lse[0], lse[1])


def test_outputs_on_the_queries(nb):
    """Queries are read while rows of others are written: o may not lie on them."""
    s = setup([40, 3], [4, 4], 4, 4, 2, 64, 16, seed=32)
    args = (s["kp"], s["vp"], s["table"], s["lens"], s["parents"])
    want = nb.attn_decode_tree(s["q"], *args, rope_base=BASE)[0]
    with pytest.raises(nb.NeAttnError) as e:
        nb.attn_decode_tree(s["q"], *args, rope_base=BASE, o=s["q"])
    assert e.value.status == -1
    room = torch.empty(2 * s["q"].numel(), dtype=torch.bfloat16, device="cuda")
    q, o = room[:s["q"].numel()].view_as(s["q"]), room[s["q"].numel():].view_as(s["q"])
    q.copy_(s["q"])
    assert torch.equal(nb.attn_decode_tree(q, *args, rope_base=BASE, o=o)[0], want)  # side by side is fine
    with pytest.raises(nb.NeAttnError):
        nb.attn_decode_tree(q, *args, rope_base=BASE, o=room[8:8 + q.numel()].view_as(q))


def test_graphs_share_a_workspace(nb):
    """Two captured calls of different shapes on one workspace, replayed in turn with new lengths, trees and queries."""
    a = setup([3000, 10], [16, 9], 16, 12, 4, 64, 64, seed=41)
    b = setup([500, 77, 0], [60, 64, 1], 64, 16, 4, 64, 32, seed=42)
    n = max(nb.decode_tree_workspace_size(2, 16, 12, 4, 64), nb.decode_tree_workspace_size(3, 64, 16, 4, 64))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for s in (a, b):
        call = lambda s=s: nb.attn_decode_tree(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["parents"], tree_len=s["nodes"],
                                               rope_base=BASE, workspace=ws)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call())
        graphs.append(g)
    for i in range(6):
        graphs[i & 1].replay()
    for s, got in ((a, outs[0]), (b, outs[1])):
        check(nb, s, got, False, False)
    a["lens"].copy_(i32([700, 0]))  # shorter, and an idle slot
    graphs[0].replay()
    want = nb.attn_decode_tree(a["q"], a["kp"], a["vp"], a["table"], a["lens"], a["parents"], tree_len=a["nodes"], rope_base=BASE)
    nb.check_status()
    assert torch.equal(outs[0][0], want[0]) and torch.equal(outs[0][1], want[1]) and not outs[0][0][1].any()


def test_capture_without_a_workspace(nb):
    s = setup([900, 31], [8, 5], 8, 12, 4, 64, 16, seed=43)
    call = lambda: nb.attn_decode_tree(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["parents"], tree_len=s["nodes"], rope_base=BASE)
    want = call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call()
        more = call()
    g.replay()
    nb.check_status()
    for x, y, z in zip(want, got, more):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_keep_a_whole_tree_and_none(nb):
    """Paths of 64 and of 0 tokens: everything stays where it is, nothing stays; a second call on the new lengths' trees."""
    s = setup([50, 7], [64, 64], 64, 4, 4, 64, 16, seed=44)
    bits = lambda: torch.stack([s["kp"].view(torch.int16), s["vp"].view(torch.int16)])  # unreached rows are NaN
    before = bits()
    path = i32([list(range(64))] * 2)
    n = nb.kv_keep_paged(s["kp"], s["vp"], s["table"], s["lens"], 64, path, i32([64, 0]))
    nb.check_status()
    assert n.tolist() == [114, 7] and torch.equal(bits(), before)
    n = nb.kv_keep_paged(s["kp"], s["vp"], s["table"], n, i32([0, 0]), path, i32([0, 0]))
    nb.check_status()
    assert n.tolist() == [114, 7] and torch.equal(bits(), before)


def test_longest_table(nb):
    """Positions up to 2^20 - 1: the largest table, rotated at its end."""
    top = 1 << 20
    page, pages = 256, 40
    kp = torch.zeros((pages, 1, page, 32), dtype=torch.float16, device="cuda")
    vp = torch.zeros((pages, 1, page, 32), dtype=torch.bfloat16, device="cuda")
    vp[:] = torch.randn_like(vp)
    table = i32(np.arange(top // page) % pages)[None]
    q = torch.randn((1, 3, 2, 32), device="cuda").bfloat16()
    o, lse = nb.attn_decode_tree(q, kp, vp, table, i32([top]), i32([-1, 0, 0]), rope_base=BASE, o_dtype=torch.float32)
    nb.check_status()
    # keys of zeros: every visible value has the same weight
    n = top - 3
    per = vp[table[0].long(), 0].reshape(top, 32).double()
    ctx = per[:n].sum(0)
    for t, see in enumerate(([0], [0, 1], [0, 2])):
        want = (ctx + per[[n + u for u in see]].sum(0)) / (n + len(see))
        # the bound of check with M = 0 and A, the mean of |v|, below 1
        assert float((o[0, t, 0].double() - want).abs().max()) <= 2.0 ** -14
        assert abs(float(lse[0, 0, t]) - np.log(n + len(see))) <= 2.0 ** -14 + 2.0 ** -22 * 14


@pytest.mark.parametrize("front", ["nothing", "memset", "copy", "host", "kernel", "join"])
def test_captured_behind_other_work(nb, front):
    """The calls' kernels are dependent launches: a step captured behind every kind of node, which writes what it reads."""
    s = setup([300, 20], [8, 6], 8, 12, 4, 64, 16, seed=45)
    q, lens, path = s["q"].clone(), s["lens"].clone(), i32([[0, 1], [0, 2]])
    host = s["q"].cpu().pin_memory()
    side = torch.cuda.Stream()

    def step():
        if front == "memset":
            s["q"].zero_()
        elif front == "copy":
            s["q"].copy_(q)
        elif front == "host":
            s["q"].copy_(host, non_blocking=True)
        elif front == "kernel":
            torch.mul(q, 2, out=s["q"])
        elif front == "join":
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                torch.mul(q, 2, out=s["q"])
            torch.add(lens, 0, out=s["lens"])
            torch.cuda.current_stream().wait_stream(side)
        got = nb.attn_decode_tree(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["parents"], tree_len=s["nodes"], rope_base=BASE)
        kp, vp = s["kp"].clone(), s["vp"].clone()
        n = nb.kv_keep_paged(kp, vp, s["table"], s["lens"], s["nodes"], path, i32two)
        return (*got, n, kp.view(torch.int16), vp.view(torch.int16))
    i32two = i32([2, 1])
    want = [x.clone() for x in step()]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(3):
        if front not in ("nothing",):
            s["q"].fill_(7)
        for x in got:
            x.zero_()
        g.replay()
        nb.check_status()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
