"""Trees of drafted tokens over the paged cache on the GPU, against the definitions in oracle/tree.py: the plan
(whole numbers, equal), the append to slots (bit by bit the same as the paged append's), the tree's attention, the
kept path (bit by bit), and a step of them all.

Bounds of the attention: q as two fp16 parts (2^-22), the weights as two bf16 parts (2^-17), sums in fp32, as in the
paged decode: with M = max_j sum_i |q_i k_ji| / sqrt(D) a logit is off by at most d = M (2^-18 for the norm
and rotation + 2^-21 for the parts and the fp32 sum of D terms), a weight by 2 d + 2^-16 (exp2, parts) relative, so
  |o error| <= (2 d + 2^-14) A + the output's rounding (2^-8 for bf16: half a step),  A = sum_j p_j |v_j|
(2^-14: the weights' 2^-16 and the fp32 sums over thousands of keys), and |lse error| <= d + 2^-14 + 2^-22 |lse|.
"""
import numpy as np
import pytest

import _harness as H
from causal_gqa_attention_flashattention_gb300 import inputs
from oracle import tree

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

EPS = 1e-6
BASE = 10000.0


@pytest.fixture(scope="module")
def nb():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_gqa_attention_flashattention_gb300 import binding
    binding.lib()
    return binding


def bf16(x):
    bits = inputs.bf16_round_bits(np.asarray(x, dtype=np.float32))
    return H.to_device(bits), inputs.bf16_bits_to_f64(bits)


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int64), dtype=torch.int32, device="cuda")


def grow(rng, n, wide=5):
    """Parents of a tree of n tokens; now and then a second root."""
    return [-1 if t == 0 or rng.random() < 0.05 else int(rng.integers(max(0, t - wide), t)) for t in range(n)]


# ------------------------------------------------------------------ plan
PLANS = [
    # kv, new, page, free pages past the need, surplus pages held, pad, tree
    ([0], [1], 16, 1, 0, 0, False),
    ([15, 16, 17, 0, 100], [1, 1, 1, 1, 0], 16, 0, 1, 3, False),
    ([0, 5, 31, 200, 7], [300, 0, 1, 33, 250], 32, -8, 2, 9, False),        # the ring runs short
    ([(i * 37) % 300 for i in range(150)], [1 + i % 13 for i in range(150)], 64, 4, 3, 0, True),
    ([10, 20, 30], [64, 1, 7], 16, 3, 0, 40, True),
    ([i % 97 for i in range(2048)], [i % 3 for i in range(2048)], 16, -100, 1, 5, False),
    ([0, 0, 0], [9000, 1, 70000], 256, 1, 0, 100, False),                   # rows of a second launch
    ([3] * 500, [16] * 500, 128, -2, 0, 0, True),
]


def plan_inputs(case, seed=0):
    kv, new, page, spare, surplus, pad, drafted = case
    rng = np.random.default_rng(seed)
    held = [-(-k // page) + (surplus if i % 3 == 1 else 0) for i, k in enumerate(kv)]
    want = [-(-(k + n) // page) for k, n in zip(kv, new)]
    free = max(1, sum(max(0, w - h) for w, h in zip(want, held)) + spare)
    P = sum(held) + free
    order = rng.permutation(P)
    table = np.full((len(kv), max(max(want), max(held)) + 1), -5)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
    first = P - 1 - free // 2 if P > free // 2 else 0
    ring = np.full(P, -9)
    ring[(first + np.arange(free)) % P] = order[at:]
    parents = [grow(rng, max(new)) for _ in kv] if drafted else None
    return table, ring, held, [first, free], kv, new, sum(new) + pad, page, parents


@pytest.mark.parametrize("case", PLANS, ids=lambda c: "b%d_p%d_%s" % (len(c[0]), c[2], "tree" if c[6] else "rows"))
def test_plan(nb, case):
    table, ring, held, span, kv, new, rows, page, parents = plan_inputs(case)
    want = tree.plan(table.tolist(), ring.tolist(), held, span, kv, new, rows, page, parents)
    t, r = i32(table), i32(ring)
    args = (i32(held), i32(span), i32(kv), i32(new), rows, page)
    kw = dict(parents=None if parents is None else i32(parents))
    for _ in range(2):  # a second call with the same inputs has the same outputs: the taken pages are still in the ring
        got = nb.paged_plan(t, r, *args, **kw)
        nb.check_status()
        for g, w in zip((t, r, got.held, got.span, got.kv_len, got.cu_new, got.slots, got.positions), want):
            assert g.tolist() == w
    # in place
    t, r, h, s = i32(table), i32(ring), i32(held), i32(span)
    got = nb.paged_plan(t, r, h, s, *args[2:], held_out=h, span_out=s, **kw)
    assert got.held is h and h.tolist() == want[2] and s.tolist() == want[3] and got.slots.tolist() == want[6]


def test_plan_one_tree_for_all(nb):
    parents = [-1, 0, 0, 1, 1, 2]
    table, ring = i32([[0], [1], [2]]), i32([0, 0, 0, 3])
    a = nb.paged_plan(table, ring, i32([1, 1, 1]), i32([3, 1]), i32([0, 3, 9]), i32([6, 2, 5]), 14, 16, parents=i32(parents))
    assert a.positions.tolist() == [0, 1, 1, 2, 2, 2, 3, 4, 9, 10, 10, 11, 11, 0]
    assert a.slots.tolist() == [0, 1, 2, 3, 4, 5, 19, 20, 41, 42, 43, 44, 45, -1]
    nb.check_status()


def test_plan_refusals(nb):
    """Lengths, counts and rings that cannot be: the sequence (the whole call) keeps what it has, and it is reported."""
    def go(kv=(5, 5, 5), new=(20, 20, 20), held=(1, 1, 1), span=(3, 4), rows=80, parents=None):
        table = [[0, -1], [1, -1], [2, -1]]
        t, r = i32(table), i32([9, 9, 9, 3, 4, 5, 6, 9])
        p = nb.paged_plan(t, r, i32(held), i32(span), i32(kv), i32(new), rows, 16, parents=parents)
        return p, t.tolist(), r.tolist(), nb.status_of_last_kernels()
    p, t, r, st = go()
    assert st == 0 and t == [[0, 3], [1, 4], [2, 5]] and p.span.tolist() == [6, 1]
    for bad in (dict(kv=(5, -1, 5)), dict(kv=(5, 33, 5)), dict(new=(20, 28, 20)), dict(kv=(5, 2 ** 31 - 1, 5)),
                dict(held=(1, -1, 1)), dict(held=(1, 3, 1))):
        p, t, r, st = go(**bad)
        assert st == -8 and t == [[0, 3], [1, -1], [2, 4]] and p.span.tolist() == [5, 2]
        assert p.held.tolist() == [2, bad.get("held", (1, 1, 1))[1], 2]
        assert p.kv_len.tolist() == [25, bad.get("kv", (5, 5, 5))[1], 25]
        n = p.cu_new.tolist()
        assert n[:2] == [0, 20] and p.slots.tolist()[n[1]:n[2]] == [-1] * (n[2] - n[1])
    p, t, r, st = go(new=(20, -3, 20))
    assert st == -8 and p.cu_new.tolist() == [0, 20, 20, 40] and p.kv_len.tolist() == [25, 5, 25]
    for span in ((-1, 4), (8, 1), (0, 9), (0, -1)):
        p, t, r, st = go(span=span)
        assert st == -8 and t == [[0, -1], [1, -1], [2, -1]] and p.span.tolist() == list(span)
        assert p.kv_len.tolist() == [5, 5, 5] and p.held.tolist() == [1, 1, 1] and set(p.slots.tolist()) == {-1}
    # rows that are not all there
    p, t, r, st = go(rows=50)
    assert st == -8 and p.cu_new.tolist() == [0, 20, 40, 50] and p.kv_len.tolist() == [25, 25, 5]
    # more tokens than the tree has, and a parent after its child
    p, t, r, st = go(new=(2, 3, 2), parents=i32([-1, 0]))
    assert st == -8 and p.kv_len.tolist() == [7, 5, 7]
    p, t, r, st = go(new=(3, 3, 3), parents=i32([[-1, 0, 1], [-1, 1, 0], [-1, 0, -2]]))
    assert st == -9 and p.positions.tolist()[:9] == [5, 6, 7, 5, 5, 6, 5, 6, 5]
    # a bad page in the ring: handed out, its rows get no slot
    t, r = i32([[-1]]), i32([7])
    p = nb.paged_plan(t, r, i32([0]), i32([0, 1]), i32([0]), i32([3]), 3, 16)
    assert nb.status_of_last_kernels() == -8 and p.slots.tolist() == [-1] * 3


# ------------------------------------------------------------------ append to slots
@pytest.mark.parametrize("case", [(1, 1, 32, 16, False, False), (37, 4, 64, 32, True, False), (300, 3, 32, 256, True, True),
                                  (5, 2, 64, 128, False, True)], ids=lambda c: "n%d_%dx%d_p%d" % c[:4])
def test_append_slots(nb, case):
    """The same bits as the paged append writes for the same places and positions."""
    N, Hkv, D, page, norm, half = case
    g = torch.Generator(device="cuda").manual_seed(N)
    kv = torch.randn((N, 2 * Hkv, D), generator=g, device="cuda").bfloat16()
    k, v = kv[:, :Hkv], kv[:, Hkv:]
    kw = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).bfloat16() if norm else None
    P = N // page + 3
    pools = [torch.full((P, 2, Hkv, page, D), 7.0, dtype=t, device="cuda") for t in (torch.float16, torch.bfloat16) * 2]
    table = torch.randperm(P, generator=g, device="cuda").to(torch.int32).view(1, P)
    first = 5
    kw_ = dict(k_weight=kw, eps=EPS, rope_base=BASE, rope_half=half)
    nb.kv_append_paged(k, v, pools[0][:, 1], pools[1][:, 1], table, i32([first]), **kw_)
    at = torch.arange(N, device="cuda") + first
    slots = (table[0, at // page] * page + at % page).to(torch.int32)
    order = torch.randperm(N, generator=g, device="cuda")  # rows in any order, some without a place
    k2, v2 = torch.cat((kv[order], kv[:4] * float("nan"))).split(Hkv, 1)
    nb.kv_append_slots(k2, v2, pools[2][:, 1], pools[3][:, 1], torch.cat((slots[order], i32([-1, -7, -2 ** 31, -1])[:len(kv[:4])])),
                       torch.cat((at.to(torch.int32)[order], i32([0, 2 ** 31 - 1, -1, 3])[:len(kv[:4])])), N + first, **kw_)
    nb.check_status()
    assert torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])


def test_append_bad_slots(nb):
    k = torch.ones((2, 1, 32), device="cuda").bfloat16()
    kp, vp = nb.paged_cache(4, 16, 1, 32, "cuda")
    for slots, pos in (([64, 1], [0, 0]), ([2 ** 31 - 1, 1], [0, 0]), ([3, 1], [10, 0]), ([3, 1], [-1, 0])):
        vp.zero_()
        nb.kv_append_slots(k, k, kp, vp, i32(slots), i32(pos), 10)
        assert nb.status_of_last_kernels() == -8
        assert (vp[0, :, 1] == 1).all() and float(vp.float().sum()) == 32.0
    nb.kv_append_slots(k[:0], k[:0], kp, vp, i32([]), i32([]), 10)
    nb.check_status()


# ------------------------------------------------------------------ attention
def setup(ctx, nodes, Tq, Hq, Hkv, D, page, seed, scale=1.0, wide=5):
    """Pools whose unreached rows and pages are NaN, and tables whose unreached entries are wild.  ctx None: idle."""
    rng = np.random.default_rng(seed)
    B = len(ctx)
    lens = [0 if c is None else c + n for c, n in zip(ctx, nodes)]
    need = [-(-n // page) for n in lens]
    P = sum(need) + 2
    perm = rng.permutation(P)
    table = np.full((B, max(need) + 1), -2 ** 31)
    kp, vp = np.full((P, Hkv, page, D), np.nan), np.full((P, Hkv, page, D), np.nan)
    at = 0
    for b in range(B):
        table[b, :need[b]] = perm[at:at + need[b]]
        for i in range(need[b]):
            n = min(page, lens[b] - i * page)
            kp[perm[at + i], :, :n] = rng.standard_normal((Hkv, n, D)) * scale
            vp[perm[at + i], :, :n] = rng.standard_normal((Hkv, n, D))
        at += need[b]
    k16 = kp.astype(np.float16)
    dvp = torch.from_numpy(vp.astype(np.float32)).cuda().bfloat16()
    q, fq = bf16(rng.standard_normal((B, Tq, Hq, D)) * scale)
    qw, fqw = bf16(1 + 0.3 * rng.standard_normal(D))
    parents = [grow(rng, Tq, wide) for _ in range(B)]
    return dict(q=q, qw=qw, kp=torch.from_numpy(k16).cuda(), vp=dvp, table=i32(table), lens=i32(lens), parents=i32(parents),
                nodes=i32(nodes), fq=fq, fqw=fqw, fk=k16.astype(np.float64), fv=dvp.float().cpu().numpy().astype(np.float64),
                ftable=table, flens=lens, fparents=parents, fnodes=nodes)


def check(nb, s, got, norm, half):
    o, lse = got
    nb.check_status()
    ro, rl, A, M = tree.decode_tree(s["fq"], s["fqw"] if norm else None, s["fk"], s["fv"], s["ftable"], s["flens"],
                                    s["fparents"], s["fnodes"], BASE, EPS, half)
    d = M * (2.0 ** -18 + 2.0 ** -21)
    go, gl = H.to_f64(o), lse.cpu().numpy().astype(np.float64)
    tol = (2 * d[..., None] + 2.0 ** -14) * A
    if o.dtype == torch.bfloat16:
        tol = tol + (np.abs(ro) + tol) * 2.0 ** -8
    err = np.abs(go - ro)
    assert (err <= tol + 1e-37).all(), float((err / (tol + 1e-37)).max())
    empty = np.isneginf(rl)
    assert (np.isneginf(gl) == empty).all() and np.isfinite(gl[~empty]).all()
    ltol = np.moveaxis(d, 1, 2) + 2.0 ** -14 + 2.0 ** -22 * np.abs(np.where(empty, 0, rl))
    assert (np.abs(np.where(empty, 0, gl) - np.where(empty, 0, rl)) <= ltol).all()


TREES = [
    # ctx, nodes, Tq, Hq, Hkv, D, page, norm, half, fp32 o
    ([0], [1], 1, 1, 1, 32, 16, False, False, False),
    ([129], [8], 8, 12, 4, 64, 16, False, False, True),                              # 24 rows
    ([0, 1, 120, 127, 128, 129, None, 250, 1000], [8] * 9, 8, 12, 4, 64, 16, True, False, False),
    ([0, 17, 63, 64, None, 5000], [13, 1, 0, 7, 13, 12], 13, 4, 2, 32, 16, True, True, True),      # 26 rows
    ([700, 3, 64, 65], [2, 3, 1, 3], 3, 8, 8, 64, 64, False, True, False),           # 3 rows
    ([900, 100, 0], [16, 9, 16], 16, 12, 4, 64, 32, True, False, True),              # 48 rows
    ([1111, 5, 300], [32] * 3, 32, 16, 4, 64, 128, True, False, False),              # 128 rows
    ([515, 40, 0], [64, 63, 64], 64, 4, 2, 64, 256, False, True, True),              # 128 rows
    ([300, 60], [64, 30], 64, 12, 4, 64, 16, True, False, False),                    # 192 rows
    ([257, 1], [64, 64], 64, 16, 4, 32, 64, False, False, True),                     # 256 rows
    ([200, None, 0], [64, 64, 40], 64, 6, 1, 64, 32, True, True, True),              # 384 rows
    ([333], [61], 61, 8, 1, 32, 16, True, False, False),                             # 488 rows
    ([40000], [20], 20, 16, 4, 64, 128, False, False, True),                         # one long context over every SM
    ([30000, 7], [64, 64], 64, 16, 4, 64, 64, False, False, True),
    ([(i * 37) % 400 for i in range(200)], [1 + i % 6 for i in range(200)], 6, 6, 3, 64, 16, True, False, False),
    ([(i * 61) % 900 for i in range(90)], [24 - i % 20 for i in range(90)], 24, 4, 4, 32, 32, False, False, True),
    ([6000, 20, 3000, 2500], [17, 16, 15, 2], 17, 12, 4, 64, 16, True, False, True),   # 51 rows, cut among blocks
    ([5000, 4000, 300], [32, 30, 31], 32, 8, 2, 32, 64, True, False, True),           # 128 rows, cut among blocks
]


@pytest.mark.parametrize("case", TREES, ids=lambda c: "b%d_t%d_%dx%dx%d_p%d" % (len(c[0]), c[2], c[3], c[4], c[5], c[6]))
def test_tree(nb, case):
    ctx, nodes, Tq, Hq, Hkv, D, page, norm, half, o32 = case
    s = setup(ctx, nodes, Tq, Hq, Hkv, D, page, seed=len(ctx) + Tq)
    n = nb.decode_tree_workspace_size(len(ctx), Tq, Hq, Hkv, D)
    ws = torch.full((n + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    kw = dict(q_weight=s["qw"] if norm else None, eps=EPS, rope_base=BASE, rope_half=half,
              o_dtype=torch.float32 if o32 else torch.bfloat16)
    call = lambda **x: nb.attn_decode_tree(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["parents"], tree_len=s["nodes"], **kw, **x)
    got = call(workspace=ws)
    check(nb, s, got, norm, half)
    assert (ws[n:] == 0xFF).all()
    for again in (call(workspace=ws), call()):  # on the used workspace and the library's, bit by bit
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def test_chain_is_the_decode(nb):
    """A tree without branches, whole and with one tree for all, against the paged decode of the same tokens."""
    s = setup([300, 33, 1000], [10] * 3, 10, 12, 4, 64, 32, seed=3)
    chain = i32([t - 1 for t in range(10)])
    want = nb.attn_decode_paged(s["q"], s["kp"], s["vp"], s["table"], s["lens"], rope_base=BASE, o_dtype=torch.float32)
    s["fparents"] = [list(range(-1, 9))] * 3
    for parents in (chain, chain.expand(3, 10), chain.repeat(3, 1)):
        got = nb.attn_decode_tree(s["q"], s["kp"], s["vp"], s["table"], s["lens"], parents, rope_base=BASE, o_dtype=torch.float32)
        check(nb, s, got, False, False)
        # both are off by at most the bound of check, with |v| below 5
        assert float((got[0] - want[0]).abs().max()) <= 2e-3 and float((got[1] - want[1]).abs().max()) <= 1e-3


def test_tokens_off_the_path_do_not_matter(nb):
    """Infinite and NaN keys of tokens that a token does not descend from."""
    s = setup([200, 60], [9, 9], 9, 4, 2, 64, 16, seed=15)
    s["parents"] = i32([[-1, 0, 0, 1, 1, 2, 2, 5, 3]] * 2)
    call = lambda kp: nb.attn_decode_tree(s["q"], kp, s["vp"], s["table"], s["lens"], s["parents"], rope_base=BASE)
    want, kp = call(s["kp"]), s["kp"].clone()
    for b, c in enumerate((200, 60)):  # token 2
        kp[int(s["table"][b, (c + 2) // 16]), :, (c + 2) % 16] = float("nan") if b else float("inf")
    got, off = call(kp), [0, 1, 3, 4, 8]
    assert torch.equal(got[0][:, off], want[0][:, off]) and torch.equal(got[1][:, :, off], want[1][:, :, off])


def test_nan_query(nb):
    """A NaN in a query gives a NaN o and lse for that row alone."""
    s = setup([500, 3], [20, 20], 20, 12, 4, 64, 16, seed=16)
    call = lambda q: nb.attn_decode_tree(q, s["kp"], s["vp"], s["table"], s["lens"], s["parents"], rope_base=BASE)
    want, q = call(s["q"]), s["q"].clone()
    q[1, 7, 5, 3] = float("nan")
    o, lse = call(q)
    assert torch.isnan(o[1, 7, 5].float()).all() and torch.isnan(lse[1, 5, 7])
    o[1, 7, 5], lse[1, 5, 7] = want[0][1, 7, 5], want[1][1, 5, 7]
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("Tq", [2, 40])
def test_large_logits(nb, Tq):
    """Logits of a few hundred: one key takes the whole weight, the maximum moves a lot."""
    s = setup([700, 129, 2], [Tq] * 3, Tq, 12, 4, 64, 16, seed=8, scale=6.0)
    got = nb.attn_decode_tree(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["parents"], rope_base=BASE, o_dtype=torch.float32)
    check(nb, s, got, False, False)


def test_strided_queries_and_pools(nb):
    s = setup([100, 37, 260], [6, 2, 5], 6, 12, 4, 64, 16, seed=12)
    args = (s["table"], s["lens"], s["parents"])
    want = nb.attn_decode_tree(s["q"], s["kp"], s["vp"], *args, tree_len=s["nodes"], rope_base=BASE)
    rows = torch.randn((3, 6, 20, 64), device="cuda").bfloat16()
    rows[:, :, :12] = s["q"]
    kp = torch.full((s["kp"].shape[0], 3, *s["kp"].shape[1:]), float("nan"), dtype=torch.float16, device="cuda")
    vp = torch.full(kp.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    kp[:, 1], vp[:, 1] = s["kp"], s["vp"]
    wide = torch.full((3, 9), 99, dtype=torch.int32, device="cuda")
    wide[:, :6] = s["parents"]
    got = nb.attn_decode_tree(rows[:, :, :12], kp[:, 1], vp[:, 1], args[0], args[1], wide[:, :6], tree_len=s["nodes"], rope_base=BASE)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    nb.check_status()


def test_bad_pages_lengths_and_trees(nb):
    s = setup([100, 90, 64], [20, 20, 20], 20, 4, 2, 64, 16, seed=13)
    call = lambda **c: nb.attn_decode_tree(s["q"], s["kp"], s["vp"], c.get("table", s["table"]), c.get("lens", s["lens"]),
                                           c.get("parents", s["parents"]), tree_len=c.get("nodes", s["nodes"]), rope_base=BASE)
    want = call()
    nb.check_status()

    def others(got, but):
        return all(torch.equal(got[0][b], want[0][b]) and torch.equal(got[1][b], want[1][b]) for b in range(3) if b != but)

    for bad in (-1, s["kp"].shape[0], 2 ** 31 - 1, -2 ** 31):
        t = s["table"].clone()
        t[1, 2] = bad
        got = call(table=t)
        assert nb.status_of_last_kernels() == -8 and torch.isfinite(got[0].float()).all() and others(got, 1)
        kp, vp = s["kp"].clone(), s["vp"].clone()
        pg = int(s["table"][1, 2])
        kp[pg], vp[pg] = 0, 0
        zero = nb.attn_decode_tree(s["q"], kp, vp, s["table"], s["lens"], s["parents"], tree_len=s["nodes"], rope_base=BASE)
        assert torch.equal(got[0], zero[0]) and torch.equal(got[1], zero[1])
    idle = lambda got, b: bool((got[0][b] == 0).all() and torch.isneginf(got[1][b]).all())
    for lens, status in ((-5, 0), (0, 0), (19, 0), (s["table"].shape[1] * 16 + 1, -8), (2 ** 31 - 1, -8), (-2 ** 31, 0)):
        n = s["lens"].clone()
        n[2] = lens
        got = call(lens=n)
        assert nb.status_of_last_kernels() == status and idle(got, 2) and others(got, 2)
    for nodes, status in ((-1, -9), (21, -9), (2 ** 31 - 1, -9), (-2 ** 31, -9), (0, 0)):
        n = s["nodes"].clone()
        n[0] = nodes
        got = call(nodes=n)
        assert nb.status_of_last_kernels() == status and idle(got, 0) and others(got, 0)
    # a parent that is none: its token hangs on the context
    for bad in (3, 7, -2, 2 ** 31 - 1, -2 ** 31):
        p = s["parents"].clone()
        p[1, 3] = bad
        got = call(parents=p)
        assert nb.status_of_last_kernels() == -9 and others(got, 1)
        p[1, 3] = -1
        root = call(parents=p)
        nb.check_status()
        assert torch.equal(got[0], root[0]) and torch.equal(got[1], root[1])


def test_binding_refusals(nb):
    s = setup([40], [4], 4, 4, 2, 64, 16, seed=1)
    call = lambda **c: nb.attn_decode_tree(c.get("q", s["q"]), s["kp"], s["vp"], s["table"], s["lens"], c.get("parents", s["parents"]),
                                           **{k: v for k, v in c.items() if k not in ("q", "parents")})
    call()
    for bad in (dict(parents=s["parents"].long()), dict(parents=s["parents"][:, :3]), dict(parents=s["parents"].cpu()),
                dict(parents=i32([[-1, 0, 1, 2]] * 2)), dict(parents=i32([[-1, -1]] * 4).t()[:1]), dict(tree_len=i32([4, 4])),
                dict(q=s["q"][..., ::2]), dict(o=torch.empty((1, 4, 4, 64), device="cuda").half()),
                dict(lse=torch.empty((1, 4, 5), device="cuda")), dict(workspace=torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 28))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(nb.NeAttnError):
        call(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    n = i32([44])
    for out in (n, torch.cat((n, n))[:1]):
        ok = out.data_ptr() != n.data_ptr()
        f = lambda: nb.kv_keep_paged(s["kp"], s["vp"], s["table"], n, 4, i32([[0, 1]]), i32([1]), kv_len_out=out)
        if ok:
            assert f().tolist() == [41]
        else:
            with pytest.raises(ValueError):
                f()
    t = i32([[0], [1]])
    both = i32([3, 4, 5])
    with pytest.raises(ValueError):
        nb.paged_plan(t, i32([2]), i32([1, 1]), i32([0, 1]), both[:2], i32([1, 1]), 2, 16, kv_len_out=both[1:])
    nb.check_status()


# ------------------------------------------------------------------ keep
KEEPS = [
    # ctx, nodes, paths, Hkv, D, page
    ([0], [1], [[0]], 1, 32, 16),
    ([14, 100, None, 31], [7, 7, 7, 5], [[0, 1, 3, 6], [2, 4, 5], [1], []], 4, 64, 16),
    ([250, 5], [64, 64], [list(range(64)), list(range(1, 64))], 2, 64, 256),
    ([7, 8, 9], [40, 33, 12], [[39], [0, 32], [3, 4, 5, 6, 7, 8, 9, 10, 11]], 3, 32, 32),
]


@pytest.mark.parametrize("case", KEEPS, ids=lambda c: "b%d_%dx%d_p%d" % (len(c[0]), c[3], c[4], c[5]))
@pytest.mark.parametrize("one", [False, True])
def test_keep(nb, case, one):
    ctx, nodes, paths, Hkv, D, page = case
    if one:  # one number of tokens for all
        nodes = [max(nodes)] * len(nodes)
    s = setup(ctx, nodes, max(nodes), Hkv, Hkv, D, page, seed=4)
    wide = max(1, max(len(p) for p in paths)) + (0 if max(len(p) for p in paths) == 64 else 1)
    path = i32([p + [-7] * (wide - len(p)) for p in paths])
    layers = [torch.full((s["kp"].shape[0], 2 * Hkv, page, D), 7.0, dtype=t, device="cuda") for t in (torch.float16, torch.bfloat16)]
    layers[0][:, Hkv:], layers[1][:, Hkv:] = s["kp"], s["vp"]
    wk, wv, n = tree.keep(layers[0].cpu().view(torch.int16).numpy(), layers[1].cpu().view(torch.int16).numpy(), s["ftable"], s["flens"],
                          nodes, paths, [len(p) for p in paths], page)
    got = nb.kv_keep_paged(*layers, s["table"], s["lens"], max(nodes) if one else s["nodes"], path, i32([len(p) for p in paths]))
    nb.check_status()
    assert got.tolist() == n
    assert (layers[0].cpu().view(torch.int16).numpy() == wk).all() and (layers[1].cpu().view(torch.int16).numpy() == wv).all()


def test_keep_bad_paths(nb):
    s = setup([20, 30], [8, 8], 8, 2, 2, 64, 16, seed=5)
    kp, vp = s["kp"].clone(), s["vp"].clone()
    for path, m in (([1, 1], 2), ([3, 2], 2), ([-1, 2], 2), ([2, 8], 2), ([0, 2 ** 31 - 1], 2), ([0, 1], 3), ([0, 1], -1)):
        got = nb.kv_keep_paged(kp, vp, s["table"], s["lens"], 8, i32([path, [0, 1]]), i32([m, 2]))
        assert nb.status_of_last_kernels() == -9 and got.tolist() == [20, 32]
        assert torch.equal(kp.view(torch.int16), s["kp"].view(torch.int16)) and torch.equal(vp.view(torch.int16), s["vp"].view(torch.int16))
    t = s["table"].clone()
    t[0, 1] = 999
    got = nb.kv_keep_paged(kp, vp, t, s["lens"], 8, i32([[5], [0]]), i32([1, 1]))
    assert nb.status_of_last_kernels() == -8 and got.tolist() == [21, 31]
    assert torch.equal(vp.view(torch.int16), s["vp"].view(torch.int16))


# ------------------------------------------------------------------ together
def steps(nb, B, layers, Hq, Hkv, D, page, seed, graph):
    """Four steps of a drafting batch: plan, append, attention, keep; the accepted tokens' rows are checked
    against the paged decode over the sequences as they have become."""
    rng = np.random.default_rng(seed)
    Tq, P, width = 12, 60, 9
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    kp = torch.zeros((P, layers * Hkv, page, D), dtype=torch.float16, device="cuda")
    vp = torch.zeros((P, layers * Hkv, page, D), dtype=torch.bfloat16, device="cuda")
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    ring, held = torch.randperm(P, generator=g, device="cuda").to(torch.int32), i32([0] * B)
    span, n, total = i32([0, P]), i32([0] * B), i32([0] * B)
    prompt = [int(x) for x in rng.integers(3, 60, B)]
    p = nb.paged_plan(table, ring, held, span, n, i32(prompt), sum(prompt), page, held_out=held, span_out=span)
    k, v = r(sum(prompt), layers * Hkv, D), r(sum(prompt), layers * Hkv, D)
    nb.kv_append_slots(k, v, kp, vp, p.slots, p.positions, width * page, rope_base=BASE)
    n.copy_(p.kv_len)
    q = [r(B, Tq, Hq, D) for _ in range(layers)]
    k, v = r(B * Tq, layers * Hkv, D), r(B * Tq, layers * Hkv, D)
    parents, new = i32([[-1] * Tq] * B), i32([Tq] * B)
    path, m = i32([[0] * Tq] * B), i32([0] * B)

    def front():
        p = nb.paged_plan(table, ring, held, span, n, new, B * Tq, page, parents=parents, kv_len_out=total, held_out=held, span_out=span)
        nb.kv_append_slots(k, v, kp, vp, p.slots, p.positions, width * page, rope_base=BASE)
        return [nb.attn_decode_tree(q[i], kp[:, i * Hkv:(i + 1) * Hkv], vp[:, i * Hkv:(i + 1) * Hkv], table, total, parents,
                                    tree_len=new, rope_base=BASE, o_dtype=torch.float32) for i in range(layers)]

    back = lambda: nb.kv_keep_paged(kp, vp, table, total, new, path, m, kv_len_out=n)
    if graph:
        new.zero_()
        front(), back()  # nothing is added: tables of the shape exist before the capture
        gf, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(gf):
            out = front()
        with torch.cuda.graph(gb):
            back()
    lens = list(prompt)
    for step in range(4):
        size = [int(x) for x in rng.integers(1, Tq + 1, B)]
        trees = [grow(rng, Tq) for _ in range(B)]
        new.copy_(i32(size))
        parents.copy_(i32(trees))
        for x in q + [k, v]:
            x.copy_(r(*x.shape))
        if graph:
            gf.replay()
        else:
            out = front()
        nb.check_status()
        ends = [int(rng.integers(0, s)) for s in size]
        lines = [tree.ancestors(t, e)[::-1] for t, e in zip(trees, ends)]
        path.copy_(i32([x + [0] * (Tq - len(x)) for x in lines]))
        m.copy_(i32([len(x) for x in lines]))
        if graph:
            gb.replay()
        else:
            back()
        lens = [a + len(x) for a, x in zip(lens, lines)]
        assert n.tolist() == lens
        for i in range(layers):
            for b in range(B):
                rows = q[i][b:b + 1, lines[b]].contiguous()
                o, lse = nb.attn_decode_paged(rows, kp[:, i * Hkv:(i + 1) * Hkv], vp[:, i * Hkv:(i + 1) * Hkv], table[b:b + 1],
                                              n[b:b + 1], rope_base=BASE, o_dtype=torch.float32)
                # the same bound on both sides, |v| below 5
                assert float((out[i][0][b, lines[b]] - o[0]).abs().max()) <= 2e-3
                assert float((out[i][1][b][:, lines[b]] - lse[0]).abs().max()) <= 1e-3
        nb.check_status()
    # all pages are somewhere once: with the sequences or in the ring
    first, count = span.tolist()
    free = [ring.tolist()[(first + j) % P] for j in range(count)]
    mine = [x for b in range(B) for x in table.tolist()[b][:held.tolist()[b]]]
    assert sorted(free + mine) == list(range(P))
    # the sequences end: every page goes back
    p = nb.paged_plan(table, ring, held, span, i32([0] * B), i32([0] * B), 1, page)
    assert p.span.tolist()[1] == P and p.held.tolist() == [0] * B
    nb.check_status()


@pytest.mark.parametrize("graph", [False, True])
def test_steps(nb, graph):
    steps(nb, 5, 2, 12, 4, 64, 16, seed=3, graph=graph)


def test_steps_small_heads(nb):
    steps(nb, 3, 1, 4, 2, 32, 32, seed=4, graph=True)


def test_streams(nb):
    """Another stream; two streams side by side with the library's workspaces; two graphs on workspaces of their own."""
    sets = [setup([5000, 2000, 40, 3000], [16, 16, 16, 9], 16, 12, 4, 64, 16, seed=50 + i) for i in range(2)]
    call = lambda s, **kw: nb.attn_decode_tree(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["parents"], tree_len=s["nodes"],
                                               rope_base=BASE, **kw)
    wants = [call(s) for s in sets]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(20):
        for i in range(2):
            outs[i].append(call(sets[i], stream=streams[i]))
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            outs[i].append(call(sets[i]))
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            assert torch.equal(o[0], wants[i][0]) and torch.equal(o[1], wants[i][1])
    nb.check_status()


def test_far_pages(nb):
    """Pages past 2^31 values into the pool."""
    Hkv, page, D = 4, 16, 64
    P = 2 ** 31 // (Hkv * page * D) + 40
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 9 GB of device memory")
    kp = torch.empty((P, Hkv, page, D), dtype=torch.float16, device="cuda")
    vp = torch.empty((P, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
    s = setup([50, 33], [7, 7], 7, 12, 4, 64, page, seed=30)
    n = s["kp"].shape[0]
    kp[P - n:], vp[P - n:] = s["kp"], s["vp"]
    table = torch.where(s["table"] >= 0, s["table"] + (P - n), s["table"])
    want = nb.attn_decode_tree(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["parents"], rope_base=BASE)
    got = nb.attn_decode_tree(s["q"], kp, vp, table, s["lens"], s["parents"], rope_base=BASE)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    row = lambda pool, t, b, j: pool[int(t[b, j // page]), :, j % page].clone()
    old = row(vp, table, 0, 50 + 5)
    nb.kv_keep_paged(kp, vp, table, s["lens"], 7, i32([[5], [0]]), i32([1, 1]))
    assert torch.equal(row(vp, table, 0, 50), old)
    k = torch.randn((1, Hkv, D), device="cuda").bfloat16()
    nb.kv_append_slots(k, k, kp, vp, i32([P * page - 1]), i32([3]), 10)
    nb.check_status()
    assert torch.equal(vp[P - 1, :, page - 1], k[0])


def test_kernel_kinds(nb):
    s = setup([100, 90], [3, 3], 3, 4, 2, 64, 16, seed=3)
    nb.profile_start(64)
    p = nb.paged_plan(s["table"].clone(), i32([0]), i32([7, 6]), i32([0, 0]), i32([100, 90]), i32([0, 0]), 1, 16)
    nb.attn_decode_tree(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["parents"])
    nb.kv_keep_paged(s["kp"], s["vp"], s["table"], s["lens"], 3, i32([[0], [1]]), i32([1, 1]))
    nb.kv_append_slots(s["q"][:, 0, :2].contiguous(), s["q"][:, 0, 2:].contiguous(), s["kp"], s["vp"], i32([0, -1]), p.kv_len, 200)
    got = nb.profile_stop()
    assert {k: v[1] for k, v in got.items() if v[1]} == dict(paged_plan=1, decode_tree=1, kv_keep=1, kv_append_paged=1)
