"""Paged key/value cache on the GPU: append and decode against the fp64 definitions
(oracle/paged.py), and both together against the framework's own attention.

Bounds.  Append: values bit by bit; keys as the norms' forward (test_gpu_qk_norm).
Decode without a shared prefix carries q as two fp16 parts (2^-22) and the weights
as two bf16 parts (2^-17), sums in fp32: with M = max_j sum_i |q_i k_ji| / sqrt(D) a
logit is off by at most d = M (2^-18 for the norm and rotation + 2^-21 for the parts
and the fp32 sum of D terms), a weight by 2 d + 2^-16 (exp2, parts) relative, so
  |o error| <= (2 d + 2^-14) A + the output's rounding,  A = sum_j p_j |v_j|
(2^-14: the weights' 2^-16 and the fp32 sums over up to thousands of keys), and
  |lse error| <= d + 2^-14 + 2^-22 |lse|.
With a shared prefix its weights are one bf16 (2^-8): 2^-8 + 2^-14 in place of 2^-14
for o; the sums, and so the LSE, keep their bound.
"""
import numpy as np
import pytest

import _harness as H
from causal_gqa_attention_flashattention_gb300 import inputs
from oracle import paged

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


# ------------------------------------------------------------------ append
APPENDS = [
    # new rows per sequence, past, Hkv, D, page, norm, half
    ([1], [0], 1, 32, 16, False, False),
    ([1, 1, 1, 1, 1], [0, 15, 16, 17, 100], 4, 64, 16, True, False),
    ([3, 0, 40, 1, 0, 0, 130], [5, 7, 0, 255, 9, 1, 31], 2, 64, 32, True, True),
    ([0, 0, 5], [0, 0, 3], 3, 32, 128, True, False),
    ([200, 33], [250, 0], 4, 64, 256, False, True),
    ([(i * 7) % 4 for i in range(300)], [i % 50 for i in range(300)], 1, 32, 64, True, False),
]


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: "%d_%dx%d_p%d" % (len(c[0]), c[2], c[3], c[4]))
@pytest.mark.parametrize("pad", [0, 9])
def test_append(nb, case, pad):
    new, past, Hkv, D, page, norm, half = case
    rng = np.random.default_rng(1)
    B = len(new)
    cu = np.concatenate([[0], np.cumsum(new)])
    N = int(cu[-1]) + pad
    need = [-(-(a + b) // page) for a, b in zip(past, new)]
    width = max(need) + 1
    P = sum(need) + 5
    perm = rng.permutation(P)
    table = np.full((B, width), 2 ** 30)  # entries not reached may hold anything
    at = 0
    for b in range(B):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
    # rows strided: keys and values side by side, as a projection gives them
    kv, fkv = bf16(rng.standard_normal((N, 2 * Hkv, D)))
    k, v = kv[:, :Hkv], kv[:, Hkv:]
    kw, fkw = bf16(1 + 0.3 * rng.standard_normal(D))
    # the pools of two layers interleaved page by page; the other layer stays as it was
    kp = torch.full((P, 2, Hkv, page, D), 7.0, dtype=torch.float16, device="cuda")
    vp = torch.full((P, 2, Hkv, page, D), 7.0, dtype=torch.bfloat16, device="cuda")
    nb.kv_append_paged(k, v, kp[:, 1], vp[:, 1], i32(table), i32(past), cu_new=i32(cu), k_weight=kw if norm else None,
                       eps=EPS, rope_base=BASE, rope_half=half)
    nb.check_status()
    gk, gv = H.to_f64(kp), H.to_f64(vp)
    assert (gk[:, 0] == 7).all() and (gv[:, 0] == 7).all()
    rows = paged.places(table, past, cu, page)
    wk, wv, tol = np.full(gk[:, 1].shape, 7.0), np.full(gk[:, 1].shape, 7.0), np.zeros(gk[:, 1].shape)
    if rows:
        idx = np.array([r[0] for r in rows])
        n = paged.rms_heads(fkv[idx, :Hkv], fkw if norm else None, EPS)
        y = paged.rope_at(n, [r[3] for r in rows], BASE, half)
        pair = np.stack((n[..., :D // 2], n[..., D // 2:]), -1) if half else n.reshape(*n.shape[:-1], D // 2, 2)
        d = np.repeat(np.linalg.norm(pair, axis=-1), 2, -1) * 2.0 ** -19
        for i, (r, pg, slot, _) in enumerate(rows):
            wk[pg, :, slot], wv[pg, :, slot] = y[i], fkv[r, Hkv:]
            tol[pg, :, slot] = (np.abs(y[i]) + d[i]) * 2.0 ** -11 + d[i] + 2.0 ** -25
    assert (gv[:, 1] == wv).all()
    assert (np.abs(gk[:, 1] - wk) <= tol).all()


def test_append_even_rows(nb):
    """cu_new = None: N / B rows for every sequence."""
    k, v = torch.randn((6, 2, 64), device="cuda").bfloat16(), torch.randn((6, 2, 64), device="cuda").bfloat16()
    table, pos0 = i32([[1, 2], [0, 3]]), i32([14, 3])
    a, b = nb.paged_cache(4, 16, 2, 64, "cuda"), nb.paged_cache(4, 16, 2, 64, "cuda")
    nb.kv_append_paged(k, v, *a, table, pos0)
    nb.kv_append_paged(k, v, *b, table, pos0, cu_new=i32([0, 3, 6]))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and (a[1][2, :, 0] == v[2]).all()


@pytest.mark.parametrize("bad", [-1, 4, 2 ** 31 - 1, -2 ** 31])
def test_append_bad_places(nb, bad):
    """A page outside the pool and a position outside the table: not written, reported."""
    k, v = torch.ones((3, 1, 32), device="cuda").bfloat16(), torch.ones((3, 1, 32), device="cuda").bfloat16()
    kp, vp = nb.paged_cache(4, 16, 1, 32, "cuda")
    nb.kv_append_paged(k, v, kp, vp, i32([[0, 1], [bad, 2], [3, 3]]), i32([0, 5, 32]))
    assert nb.status_of_last_kernels() == -8
    assert (vp[0, :, 0] == 1).all() and float(vp.float().sum()) == 32.0
    nb.kv_append_paged(k[:1], v[:1], kp, vp, i32([[0, 1]]), i32([-1]))
    assert nb.status_of_last_kernels() == -8
    nb.kv_append_paged(k[:1], v[:1], kp, vp, i32([[0, 1]]), i32([1]))
    nb.check_status()


# ------------------------------------------------------------------ decode
def setup(lens, Tq, Hq, Hkv, D, page, seed, prefix=0, scale=1.0, layers=1):
    """Pools whose unreached rows and pages are NaN, and tables whose unreached entries are wild."""
    rng = np.random.default_rng(seed)
    B, shared = len(lens), prefix // page
    own = [max(0, -(-n // page) - shared) if n > 0 else 0 for n in lens]
    P = shared + sum(own) + 2
    perm = rng.permutation(P)
    width = shared + max(own + [0]) + 1
    table = np.full((B, width), -2 ** 31)
    kp, vp = np.full((P, Hkv, page, D), np.nan), np.full((P, Hkv, page, D), np.nan)
    ptable = perm[:shared]
    reach = max(0, min(prefix, max(lens)))
    for i, pg in enumerate(ptable):
        n = min(page, max(0, reach - i * page))
        kp[pg, :, :n] = rng.standard_normal((Hkv, n, D)) * scale
        vp[pg, :, :n] = rng.standard_normal((Hkv, n, D))
    at = shared
    for b in range(B):
        table[b, shared:shared + own[b]] = perm[at:at + own[b]]
        for i in range(own[b]):
            n = min(page, lens[b] - prefix - i * page)
            kp[perm[at + i], :, :n] = rng.standard_normal((Hkv, n, D)) * scale
            vp[perm[at + i], :, :n] = rng.standard_normal((Hkv, n, D))
        at += own[b]
    k16 = kp.astype(np.float16)
    dvp = torch.from_numpy(vp.astype(np.float32)).cuda().bfloat16()
    q, fq = bf16(rng.standard_normal((B, Tq, Hq, D)) * scale)
    qw, fqw = bf16(1 + 0.3 * rng.standard_normal(D))
    return dict(q=q, qw=qw, kp=torch.from_numpy(k16).cuda(), vp=dvp, table=i32(table), lens=i32(lens),
                ptable=i32(ptable) if shared else None, fq=fq, fqw=fqw, fk=k16.astype(np.float64),
                fv=dvp.float().cpu().numpy().astype(np.float64), ftable=table, flens=lens, fptable=list(ptable))


def check(nb, s, got, norm, half, prefix=0):
    o, lse = got
    nb.check_status()
    ro, rl, A, M = paged.decode_paged(s["fq"], s["fqw"] if norm else None, s["fk"], s["fv"], s["ftable"], s["flens"], BASE,
                                      EPS, half, s["fptable"], bounds=True)
    d = M * (2.0 ** -18 + 2.0 ** -21)
    w = 2.0 ** -14 + (2.0 ** -8 if prefix else 0)
    go, gl = H.to_f64(o), lse.cpu().numpy().astype(np.float64)
    tol = (2 * d[..., None] + w) * A
    if o.dtype == torch.bfloat16:
        tol = tol + (np.abs(ro) + tol) * 2.0 ** -8
    err = np.abs(go - ro)
    assert (err <= tol + 1e-37).all(), float((err / (tol + 1e-37)).max())
    empty = np.isneginf(rl)
    assert (np.isneginf(gl) == empty).all() and np.isfinite(gl[~empty]).all()
    dl = np.moveaxis(d, 1, 2)
    ltol = dl + 2.0 ** -14 + 2.0 ** -22 * np.abs(np.where(empty, 0, rl))
    assert (np.abs(np.where(empty, 0, gl) - np.where(empty, 0, rl)) <= ltol).all()


DECODES = [
    # lens, Tq, Hq, Hkv, D, page, norm, half, fp32 o
    ([1], 1, 1, 1, 32, 16, False, False, False),
    ([129], 1, 12, 4, 64, 16, False, False, True),
    ([0, 1, 127, 128, 129, 255, 256, 257, 1000], 1, 12, 4, 64, 16, True, False, False),
    ([16, 17, 0, 31, 33, 5000], 1, 4, 2, 32, 16, True, True, True),
    ([700, 3, 64, 65], 1, 8, 1, 64, 64, False, True, False),
    ([3, 1, 2, 900, 0, 130], 3, 12, 4, 64, 32, True, False, True),      # queries before position 0
    ([1111, 5, 6], 5, 4, 2, 32, 128, True, False, False),
    ([300, 17], 16, 4, 2, 64, 256, False, False, True),                 # 32 rows
    ([515, 40], 10, 16, 4, 64, 64, True, False, False),                 # 40 rows
    ([200, 128, 1], 32, 12, 4, 64, 16, False, False, True),             # 96 rows
    ([300, 128], 128, 2, 2, 32, 32, True, True, False),                 # 128 rows
    ([40000], 1, 16, 4, 64, 128, False, False, True),                   # one long context over every SM
    ([(i * 37) % 400 for i in range(200)], 1, 6, 3, 64, 16, True, False, False),
]


@pytest.mark.parametrize("case", DECODES, ids=lambda c: "b%d_t%d_%dx%dx%d_p%d" % (len(c[0]), c[1], c[2], c[3], c[4], c[5]))
def test_decode(nb, case):
    lens, Tq, Hq, Hkv, D, page, norm, half, o32 = case
    s = setup(lens, Tq, Hq, Hkv, D, page, seed=len(lens) + Tq)
    n = nb.decode_paged_workspace_size(len(lens), Tq, Hq, Hkv, D)
    ws = torch.full((n + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    call = lambda: nb.attn_decode_paged(s["q"], s["kp"], s["vp"], s["table"], s["lens"], q_weight=s["qw"] if norm else None,
                                        eps=EPS, rope_base=BASE, o_dtype=torch.float32 if o32 else torch.bfloat16,
                                        workspace=ws, rope_half=half)
    got = call()
    check(nb, s, got, norm, half)
    assert (ws[n:] == 0xFF).all()
    again = call()  # on the used workspace, bit by bit
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


PREFIXES = [
    # own lengths past the prefix (None: idle), prefix, Tq, Hq, Hkv, D, page, norm, half, fp32 o
    ([1, 1], 16, 1, 4, 2, 32, 16, False, False, True),
    ([1, None, 17, 128, 129, 300], 256, 1, 12, 4, 64, 64, True, False, False),
    ([5, 2, 70], 128, 2, 6, 3, 64, 32, True, True, True),
    ([(i * 13) % 90 + 1 for i in range(70)], 1024, 1, 12, 4, 64, 16, False, False, False),   # 210 rows a head
    ([3, 4, 500, 9], 768, 3, 8, 1, 32, 256, True, False, False),
    ([2, 40, 9, 8], 80, 1, 12, 4, 64, 16, False, True, True),            # tiles that end inside the prefix
    ([1, 7, 33], 416, 4, 6, 2, 64, 32, True, False, True),
    ([12, 31], 704, 1, 8, 1, 32, 64, True, False, False),
    ([600, 2, 77], 128, 12, 8, 2, 64, 16, False, False, True),           # 48 rows a sequence
    ([(i * 5) % 40 + 3 for i in range(140)], 640, 3, 4, 2, 64, 128, False, True, False),      # 840 rows a head
    # an odd number of row tiles, and blocks that take many key tiles for the last one alone
    ([3, None, 40, 9], 16384, 1, 8, 8, 64, 64, True, False, True),
    ([11], 65536, 3, 6, 2, 32, 256, False, True, True),
    ([(i * 11) % 50 + 1 for i in range(100)], 10240, 1, 12, 4, 64, 16, False, False, False),  # 300 rows a head
]


@pytest.mark.parametrize("case", PREFIXES, ids=lambda c: "b%d_p%d_t%d_%dx%dx%d" % (len(c[0]), c[1], c[2], c[3], c[4], c[5]))
def test_shared_prefix(nb, case):
    own, prefix, Tq, Hq, Hkv, D, page, norm, half, o32 = case
    lens = [0 if x is None else prefix + x for x in own]
    s = setup(lens, Tq, Hq, Hkv, D, page, seed=prefix + Tq, prefix=prefix)
    kw = dict(q_weight=s["qw"] if norm else None, eps=EPS, rope_base=BASE, rope_half=half,
              o_dtype=torch.float32 if o32 else torch.bfloat16)
    call = lambda: nb.attn_decode_paged(s["q"], s["kp"], s["vp"], s["table"], s["lens"], prefix_table=s["ptable"],
                                        prefix_len=prefix, **kw)
    got = call()
    check(nb, s, got, norm, half, prefix)
    again = call()
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def test_prefix_longer_than_a_sequence(nb):
    """Sequences that end inside the shared pages, at and before their last position, see their own part."""
    prefix, page = 256, 32
    lens = [300, 256, 255, 33, 1, 0, 2, 257]
    s = setup(lens, 2, 12, 4, 64, page, seed=5, prefix=prefix)
    got = nb.attn_decode_paged(s["q"], s["kp"], s["vp"], s["table"], s["lens"], prefix_table=s["ptable"], prefix_len=prefix,
                               rope_base=BASE, o_dtype=torch.float32)
    check(nb, s, got, False, False, prefix)


def test_prefix_only(nb):
    """No sequence has a position of its own past the shared pages."""
    s = setup([64, 64, 0, 64], 1, 4, 2, 64, 16, seed=6, prefix=64)
    got = nb.attn_decode_paged(s["q"], s["kp"], s["vp"], s["table"], s["lens"], prefix_table=s["ptable"], prefix_len=64,
                               rope_base=BASE, o_dtype=torch.float32)
    check(nb, s, got, False, False, 64)


def test_many_sequences(nb):
    """More sequences than the sweep has threads, one of them long enough to be cut among blocks."""
    lens = [(i * 29) % 75 for i in range(900)]
    lens[417] = 6000
    s = setup(lens, 2, 6, 3, 32, 16, seed=14)
    got = nb.attn_decode_paged(s["q"], s["kp"], s["vp"], s["table"], s["lens"], q_weight=s["qw"], rope_base=BASE)
    check(nb, s, got, True, False)


def test_most_sequences_and_rows(nb):
    """The largest batch with the most rows, against the same sequences in smaller batches (short
    ones are never cut, so the results are the same bit by bit)."""
    B, Tq = 2048, 128
    lens = [(i * 61) % 200 for i in range(B)]
    lens[2047] = 200
    pages, D = 16, 64
    P = 64
    g = torch.Generator(device="cuda").manual_seed(2)
    kp = torch.randn((P, 1, pages, D), generator=g, device="cuda").half()
    vp = torch.randn((P, 1, pages, D), generator=g, device="cuda").bfloat16()
    table = torch.randint(0, P, (B, 13), generator=g, device="cuda", dtype=torch.int32)
    q = torch.randn((B, Tq, 1, D), generator=g, device="cuda").bfloat16()
    n = i32(lens)
    o, lse = nb.attn_decode_paged(q, kp, vp, table, n, rope_base=BASE)
    nb.check_status()
    for lo, hi in ((0, 700), (700, 2048)):
        a, b = nb.attn_decode_paged(q[lo:hi], kp, vp, table[lo:hi], n[lo:hi], rope_base=BASE)
        assert torch.equal(a, o[lo:hi]) and torch.equal(b, lse[lo:hi])


def test_keys_after_a_query_do_not_matter(nb):
    """Infinite and NaN keys at the positions of later new tokens."""
    s = setup([300, 33], 3, 4, 2, 64, 16, seed=15)
    args = (s["vp"], s["table"], s["lens"])
    want = nb.attn_decode_paged(s["q"], s["kp"], *args, rope_base=BASE)
    kp = s["kp"].clone()
    for b, n in enumerate((300, 33)):
        kp[int(s["table"][b, (n - 1) // 16]), :, (n - 1) % 16] = float("nan") if b else float("inf")
    got = nb.attn_decode_paged(s["q"], kp, *args, rope_base=BASE)
    assert torch.equal(got[0][:, :2], want[0][:, :2]) and torch.equal(got[1][:, :, :2], want[1][:, :, :2])


def test_large_logits(nb):
    """Logits of a few hundred: one key takes the whole weight, the maximum moves a lot."""
    s = setup([700, 129, 2], 2, 12, 4, 64, 16, seed=8, scale=6.0)
    got = nb.attn_decode_paged(s["q"], s["kp"], s["vp"], s["table"], s["lens"], rope_base=BASE, o_dtype=torch.float32)
    check(nb, s, got, False, False)


def test_strided_queries_and_pools(nb):
    """q inside a fused projection's rows, two layers' pools interleaved."""
    s = setup([100, 37, 260], 1, 12, 4, 64, 16, seed=12)
    want = nb.attn_decode_paged(s["q"], s["kp"], s["vp"], s["table"], s["lens"], rope_base=BASE)
    rows = torch.randn((3, 1, 20, 64), device="cuda").bfloat16()
    rows[:, :, :12] = s["q"]
    kp = torch.full((s["kp"].shape[0], 3, *s["kp"].shape[1:]), float("nan"), dtype=torch.float16, device="cuda")
    vp = torch.full(kp.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    kp[:, 1], vp[:, 1] = s["kp"], s["vp"]
    got = nb.attn_decode_paged(rows[:, :, :12], kp[:, 1], vp[:, 1], s["table"], s["lens"], rope_base=BASE)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_bad_pages_and_lengths(nb):
    """A bad page counts as zeros, a length past the table is cut to it; both are reported, and
    the other sequences keep their results."""
    s = setup([100, 90, 64], 1, 4, 2, 64, 16, seed=13)
    args = (s["q"], s["kp"], s["vp"])
    want = nb.attn_decode_paged(*args, s["table"], s["lens"], rope_base=BASE)
    nb.check_status()
    for bad in (-1, s["kp"].shape[0], 2 ** 31 - 1, -2 ** 31):
        t = s["table"].clone()
        t[1, 2] = bad
        got = nb.attn_decode_paged(*args, t, s["lens"], rope_base=BASE)
        assert nb.status_of_last_kernels() == -8
        assert torch.isfinite(got[0].float()).all()
        for b in (0, 2):
            assert torch.equal(got[0][b], want[0][b]) and torch.equal(got[1][b], want[1][b])
    width = s["table"].shape[1]
    lens = s["lens"].clone()
    lens[2] = width * 16 + 1000
    t = s["table"].clone()
    t[2] = t[2, 0]
    got = nb.attn_decode_paged(*args, t, lens, rope_base=BASE)
    assert nb.status_of_last_kernels() == -8
    lens[2] = width * 16
    cut = nb.attn_decode_paged(*args, t, lens, rope_base=BASE)
    nb.check_status()
    assert torch.equal(got[0], cut[0]) and torch.equal(got[1], cut[1])
    lens[0] = -5
    got = nb.attn_decode_paged(*args, t, lens, rope_base=BASE)
    nb.check_status()
    assert (got[0][0] == 0).all() and torch.isneginf(got[1][0]).all()
    p = nb.attn_decode_paged(*args, s["table"], s["lens"], rope_base=BASE, prefix_table=i32([0, 10 ** 6]), prefix_len=32)
    assert nb.status_of_last_kernels() == -8 and torch.isfinite(p[0].float()).all()


def test_streams_and_graphs(nb):
    """Another stream; a graph replayed with longer sequences; two graphs on one workspace in turn."""
    Tq, Hq, Hkv, D, page = 1, 12, 4, 64, 16
    s = setup([700, 300, 129, 40], Tq, Hq, Hkv, D, page, seed=21)
    full = [700, 300, 129, 40]
    call = lambda lens, **kw: nb.attn_decode_paged(s["q"], s["kp"], s["vp"], s["table"], lens, rope_base=BASE, **kw)
    wants = {k: call(i32([max(0, n - k) for n in full])) for k in (0, 1, 39, 200)}
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = call(s["lens"], stream=st)
    st.synchronize()
    assert torch.equal(got[0], wants[0][0])
    ws = torch.empty(nb.decode_paged_workspace_size(4, Tq, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    lens = [i32([1, 1, 1, 1]), i32([1, 1, 1, 1])]
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(lens[i], workspace=ws))
        graphs.append(g)
    for k in (200, 39, 1, 0):
        for i in range(2):
            lens[i].copy_(i32([max(0, n - k) for n in full]))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o[0], wants[k][0]) and torch.equal(o[1], wants[k][1])


def test_many_streams(nb):
    """More streams than the library keeps workspaces for, each used once, then the first again."""
    import ctypes
    s = setup([700, 3000, 40], 1, 8, 2, 64, 32, seed=12)
    call = lambda: nb.attn_decode_paged(s["q"], s["kp"], s["vp"], s["table"], s["lens"], o_dtype=torch.float32)
    want = call()
    rt, handles = torch.cuda.cudart(), []
    torch.cuda.synchronize()
    for _ in range(70):
        h = ctypes.c_void_p()
        assert int(rt.cudaStreamCreate(ctypes.addressof(h))) == 0
        handles.append(h.value)
    try:
        for h in handles + handles[:3]:
            stream = torch.cuda.ExternalStream(h)
            with torch.cuda.stream(stream):
                got = call()
            stream.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    finally:
        torch.cuda.synchronize()
        for h in handles:
            rt.cudaStreamDestroy(h)
    got = call()
    assert torch.equal(got[0], want[0])
    nb.check_status()


def test_two_streams_at_once(nb):
    """Calls that run side by side on streams of their own, with the library's workspaces."""
    lens = [5000, 2000, 40, 3000]
    sets = [setup(lens, 1, 12, 4, 64, 16, seed=50 + i) for i in range(2)]
    call = lambda s, **kw: nb.attn_decode_paged(s["q"], s["kp"], s["vp"], s["table"], s["lens"], rope_base=BASE, **kw)
    wants = [call(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(20):
        for i in range(2):
            outs[i].append(call(sets[i], stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            assert torch.equal(o[0], wants[i][0]) and torch.equal(o[1], wants[i][1])


def test_step_in_a_graph(nb):
    """Append and decode over a shared prefix captured together and replayed as the sequences grow."""
    B, Hq, Hkv, D, page, prefix = 5, 12, 4, 64, 32, 128
    g = torch.Generator(device="cuda").manual_seed(9)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    kp, vp = r(40, Hkv, page, D).half(), r(40, Hkv, page, D).bfloat16()
    table = torch.randperm(40, generator=g, device="cuda")[:35].to(torch.int32).view(B, 7).contiguous()
    shared = table[0, :4].clone()
    table[:, :4] = shared
    q, k, v = r(B, 1, Hq, D).bfloat16(), r(B, Hkv, D).bfloat16(), r(B, Hkv, D).bfloat16()
    kw, qw = torch.ones(D, device="cuda").bfloat16(), (1 + 0.1 * r(D)).bfloat16()
    pos = i32([130, 128, 140, 131, 200])
    n = pos + 1

    def step(kp, vp, n, pos):
        nb.kv_append_paged(k, v, kp, vp, table, pos, k_weight=kw, rope_base=BASE)
        return nb.attn_decode_paged(q, kp, vp, table, n, q_weight=qw, rope_base=BASE, prefix_table=shared, prefix_len=prefix)

    eager_k, eager_v = kp.clone(), vp.clone()
    step(eager_k.clone(), eager_v.clone(), n, pos)  # tables of the shape exist before the capture
    gpos, gn = torch.zeros_like(pos), torch.zeros_like(n)
    gpos.copy_(pos)
    gn.copy_(n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(kp, vp, gn, gpos)
    for i in range(4):
        for t, x in ((k, r(B, Hkv, D)), (v, r(B, Hkv, D)), (q, r(B, 1, Hq, D))):
            t.copy_(x)
        gpos.copy_(pos + i)
        gn.copy_(n + i)
        graph.replay()
        want = step(eager_k, eager_v, n + i, pos + i)
        torch.cuda.synchronize()
        assert torch.equal(kp, eager_k) and torch.equal(vp, eager_v)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_kernel_kinds(nb):
    """Every launch of the new calls is counted under its kind."""
    s = setup([100, 90], 1, 4, 2, 64, 16, seed=3, prefix=64)
    nb.profile_start(64)
    nb.attn_decode_paged(s["q"], s["kp"], s["vp"], s["table"], s["lens"], prefix_table=s["ptable"], prefix_len=64)
    nb.attn_decode_paged(s["q"], s["kp"], s["vp"], s["table"].clamp(0), s["lens"])
    nb.kv_append_paged(s["q"][:, 0, :2].contiguous(), s["q"][:, 0, 2:].contiguous(), s["kp"], s["vp"], s["table"], i32([99, 89]))
    q = torch.randn((1, 4, 2, 32), device="cuda").bfloat16()
    w = torch.ones(32, device="cuda").bfloat16()
    nb.qk_norm(q, q, w, w)
    nb.qk_norm_bwd(q, q, w, w, q, q)
    got = nb.profile_stop()
    assert {k: v[1] for k, v in got.items() if v[1]} == dict(decode_prefix=1, decode_paged=1, kv_append_paged=1, qk_norm=1,
                                                             qk_norm_bwd=1)
    assert all(got[k][0] > 0 for k in ("decode_prefix", "decode_paged", "kv_append_paged", "qk_norm", "qk_norm_bwd"))


def test_far_pages(nb):
    """Pages past 2^31 values into the pool."""
    Hkv, page, D = 4, 16, 64
    one = Hkv * page * D
    P = 2 ** 31 // one + 40
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 9 GB of device memory")
    kp = torch.empty((P, Hkv, page, D), dtype=torch.float16, device="cuda")
    vp = torch.empty((P, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
    s = setup([50, 33], 1, 12, 4, 64, page, seed=30)
    n = s["kp"].shape[0]
    kp[P - n:], vp[P - n:] = s["kp"], s["vp"]
    table = torch.where(s["table"] >= 0, s["table"] + (P - n), s["table"])
    want = nb.attn_decode_paged(s["q"], s["kp"], s["vp"], s["table"], s["lens"], rope_base=BASE)
    got = nb.attn_decode_paged(s["q"], kp, vp, table, s["lens"], rope_base=BASE)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    k, v = torch.randn((2, Hkv, D), device="cuda").bfloat16(), torch.randn((2, Hkv, D), device="cuda").bfloat16()
    nb.kv_append_paged(k, v, kp, vp, table, i32([49, 32]))
    nb.check_status()
    assert torch.equal(vp[int(table[0, 3]), :, 1], v[0]) and torch.equal(vp[int(table[1, 2]), :, 0], v[1])


@pytest.mark.parametrize("half", [False, True])
def test_serving_chain(nb, half):
    """Prompts appended in two parts, then tokens one by one, with norms: every decode equals the
    rows of the training path (norm, rotation, attention) over the whole sequence, to its bounds."""
    B, T, Hq, Hkv, D, page = 2, 150, 12, 4, 64, 32
    rng = np.random.default_rng(40)
    q, _ = bf16(rng.standard_normal((B, T, Hq, D)))
    k, _ = bf16(rng.standard_normal((B, T, Hkv, D)))
    v, _ = bf16(rng.standard_normal((B, T, Hkv, D)))
    qw, _ = bf16(1 + 0.2 * rng.standard_normal(D))
    kw, _ = bf16(1 + 0.2 * rng.standard_normal(D))
    ws = nb.qk_norm(q, k, qw, kw, eps=EPS, rope_base=BASE, rope_half=half)
    o, lse = nb.attn_fwd(None, None, v, BASE, workspace=ws, qk_rotated=True, Hq=Hq, rope_half=half)
    kp, vp = nb.paged_cache(12, page, Hkv, D, "cuda")
    table = i32([[3, 11, 0, 7, 9], [2, 5, 10, 1, 4]])
    put = lambda lo, hi: nb.kv_append_paged(k[:, lo:hi].reshape(-1, Hkv, D), v[:, lo:hi].reshape(-1, Hkv, D), kp, vp, table,
                                            i32([lo] * B), k_weight=kw, eps=EPS, rope_base=BASE, rope_half=half)
    put(0, 61)
    put(61, 140)
    for t in range(140, T):
        put(t, t + 1)
        got = nb.attn_decode_paged(q[:, t:t + 1], kp, vp, table, i32([t + 1] * B), q_weight=qw, eps=EPS, rope_base=BASE,
                                   rope_half=half)
        rel, mx = H.errors(H.to_f64(got[0]), H.to_f64(o[:, t:t + 1]))
        assert rel <= H.REL_L2_TOL and mx <= H.MAX_ABS_TOL
        assert float((got[1][:, :, 0] - lse[:, :, t]).abs().max()) <= H.LSE_ABS_TOL
    nb.check_status()
