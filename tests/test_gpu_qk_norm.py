"""Query/key norms with the rotation (ne_attn_qk_norm) and their backward on the GPU
against the fp64 definitions (oracle/paged.py), and the training chain norm ->
attention -> backward -> norm's backward against the oracle.

Bounds, from the number formats (n the normalised pair, |n| its length):
  forward: the fp16 rounding 2^-11 |y| (2^-25 below the normal range) on top of the
    fp32 arithmetic: the sum of squares (11 roundings, halved by the root), rsqrt
    (2^-22.4), the products with x and w, the table's cos and sin and the two-term
    rotation: together below 30 * 2^-24 < 2^-19 of |n|.
  backward, fp32: dx = r (w g - xh m): the sum m has 13 roundings relative to
    sum |w g xh| / D, the rest fewer than 27: below 40 * 2^-24 < 2^-18 of
    r (|w g| + |xh| mean |w g xh|); bf16 adds 2^-8 |dx|.
  dw: sums of (rows a thread takes) + 2 + 8 + (blocks / 32) + 32 terms in fp32, each
    term itself within 8 * 2^-24: below 2^-24 * (that count + 8) of sum |g xh|.
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
# (B, T, Hq, Hkv, D): one row, odd lengths, heads that do not fill a thread's group, the 12/4 and 16/4 models
SHAPES = [(1, 1, 1, 1, 32), (2, 77, 4, 2, 32), (3, 333, 6, 3, 64), (1, 1030, 5, 1, 64), (2, 512, 12, 4, 64),
          (1, 700, 16, 4, 64), (5, 129, 7, 7, 32)]


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


def make(B, T, Hq, Hkv, D, seed, fused):
    """(device q, k, qw, kw), (fp64 q, k, qw, kw); rows of very different size, one of zeros."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((B, T, Hq + 2 * Hkv, D)) * np.exp(rng.standard_normal((B, T, Hq + 2 * Hkv, 1)) * 2)
    x[0, 0, 0] = 0
    dx, fx = bf16(x)
    qw, fqw = bf16(1 + 0.3 * rng.standard_normal(D))
    kw, fkw = bf16(1 + 0.3 * rng.standard_normal(D))
    q, k = dx[:, :, :Hq], dx[:, :, Hq:Hq + Hkv]
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    return (q, k, qw, kw), (fx[:, :, :Hq], fx[:, :, Hq:Hq + Hkv], fqw, fkw)


def rotated(x, w, half):
    B, T = x.shape[:2]
    n = paged.rms_heads(x, w, EPS)
    y = paged.rope_at(n.reshape(B * T, *x.shape[2:]), np.tile(np.arange(T), B), BASE, half).reshape(x.shape)
    D = x.shape[-1]
    pair = np.stack((n[..., :D // 2], n[..., D // 2:]), -1) if half else n.reshape(*n.shape[:-1], D // 2, 2)
    size = np.repeat(np.linalg.norm(pair, axis=-1), 2, -1)
    return y, size


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("half,fused", [(False, False), (True, True), (False, True)])
def test_forward(nb, shape, half, fused):
    B, T, Hq, Hkv, D = shape
    dev, ref = make(*shape, seed=100 + T, fused=fused)
    n = nb.fwd_workspace_size(*shape)
    ws = torch.full((n + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    out = nb.qk_norm(*dev, eps=EPS, rope_base=BASE, rope_half=half, workspace=ws)
    nb.check_status()
    assert out is ws and (ws[n:] == 0x5A).all()
    for got, x, w in zip(nb.rotated_qk(ws, *shape), ref[:2], ref[2:]):
        y, size = rotated(x, w, half)
        err = np.abs(H.to_f64(got) - y)
        d = size * 2.0 ** -19
        assert (err <= (np.abs(y) + d) * 2.0 ** -11 + d + 2.0 ** -25).all(), float(err.max())


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("fp32,fused,inplace", [(False, False, True), (True, True, False), (True, False, True),
                                                (False, True, False)])
def test_backward(nb, shape, fp32, fused, inplace):
    B, T, Hq, Hkv, D = shape
    dev, ref = make(*shape, seed=200 + T, fused=fused)
    rng = np.random.default_rng(7)
    g = [rng.standard_normal((B, T, h, D)).astype(np.float32) for h in (Hq, Hkv)]
    if fp32:
        gd, gf = [torch.from_numpy(x).cuda() for x in g], [x.astype(np.float64) for x in g]
    else:
        gd, gf = zip(*[bf16(x) for x in g])
    kw = {}
    guard = None
    if inplace:
        gd = [x.clone() for x in gd]
        kw = dict(dq=gd[0], dk=gd[1])
    elif fused:  # into the fused projection's gradient: the value heads' part stays as it was
        guard = torch.full((B, T, Hq + 2 * Hkv, D), 3.0, dtype=gd[0].dtype, device="cuda")
        kw = dict(dq=guard[:, :, :Hq], dk=guard[:, :, Hq:Hq + Hkv])
    dq, dk, dqw, dkw = nb.qk_norm_bwd(*dev, *gd, eps=EPS, **kw)
    nb.check_status()
    if guard is not None:
        assert (guard[:, :, Hq + Hkv:] == 3.0).all()
    for got, gw, x, w, gg in zip((dq, dk), (dqw, dkw), ref[:2], ref[2:], gf):
        rx, rw = paged.rms_heads_bwd(x, w, gg, EPS)
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
        xh = x * r
        size = r * (np.abs(w * gg) + np.abs(xh) * np.abs(w * gg * xh).mean(-1, keepdims=True))
        tol = size * 2.0 ** -18
        if not fp32:
            tol = tol + (np.abs(rx) + tol) * 2.0 ** -8
        err = np.abs(H.to_f64(got) - rx)
        assert got.dtype == gd[0].dtype and (err <= tol + 1e-37).all(), float((err / (tol + 1e-37)).max())
        rows = B * T * (Hq + Hkv)
        terms = rows // 32 + 2 + 8 + 20 + 32  # one block takes at least 32 rows at a time
        assert (np.abs(gw.cpu().numpy() - rw) <= 2.0 ** -24 * (terms + 8) * np.abs(gg * xh).reshape(-1, D).sum(0)).all()


def test_backward_is_reproducible(nb):
    dev, _ = make(2, 500, 12, 4, 64, 5, False)
    g = [torch.randn_like(dev[0]), torch.randn_like(dev[1])]
    one = nb.qk_norm_bwd(*dev, *g)
    two = nb.qk_norm_bwd(*dev, *g)
    assert all(torch.equal(a, b) for a, b in zip(one, two))


def test_gradient_against_differences(nb):
    """The GPU's gradients against central differences of the fp64 definition."""
    shape = (1, 3, 2, 1, 32)
    dev, ref = make(*shape, seed=9, fused=False)
    q, w = ref[0].copy(), ref[2]
    rng = np.random.default_rng(3)
    g = rng.standard_normal(q.shape).astype(np.float32)
    gk = torch.zeros(dev[1].shape, dtype=torch.float32, device="cuda")
    dq, dk, dqw, dkw = nb.qk_norm_bwd(*dev, torch.from_numpy(g).cuda(), gk, eps=EPS)
    assert (dk == 0).all() and (dkw == 0).all()
    f = lambda a, b: float((g * paged.rms_heads(a, b, EPS)).sum())
    got = H.to_f64(dq)
    for idx in [(0, 1, 0, 3), (0, 2, 1, 31), (0, 0, 1, 0), (0, 1, 1, 17)]:
        h = 1e-5 * max(np.abs(q[idx[:3]]).max(), 1e-3)
        a, b = q.copy(), q.copy()
        a[idx] += h
        b[idx] -= h
        fd = (f(a, w) - f(b, w)) / (2 * h)
        scale = np.abs(got[idx[:3]]).max()
        assert abs(got[idx] - fd) <= 1e-4 * scale, (got[idx], fd)
    for i in (0, 13, 31):
        a, b = w.copy(), w.copy()
        a[i] += 1e-4
        b[i] -= 1e-4
        fd = (f(q, a) - f(q, b)) / 2e-4
        assert abs(float(dqw[i]) - fd) <= 1e-4 * (1 + abs(fd))


@pytest.mark.parametrize("shape", [(2, 200, 4, 2, 64), (1, 130, 6, 3, 32)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("half", [False, True])
def test_training_chain(nb, oracle_mod, shape, half):
    """norm -> attention -> attention backward -> norm's backward, the workspace handed on.

    dq, dk pass two fp32 stages beyond the attention's bound: the attention's dq, dk
    (relative L2 5e-3) go through the norm's linear map, whose rows have norm at most
    2 max|w| r; relative to the result the bound doubles at most on these inputs'
    weights (0.3 .. 2): 1e-2 relative L2."""
    B, T, Hq, Hkv, D = shape
    dev, ref = make(*shape, seed=31, fused=True)
    rng = np.random.default_rng(11)
    v, fv = bf16(rng.standard_normal((B, T, Hkv, D)))
    do, fdo = bf16(rng.standard_normal((B, T, Hq, D)))
    ws = nb.alloc_workspace(B, T, Hq, Hkv, D)
    nb.qk_norm(*dev, eps=EPS, rope_base=BASE, rope_half=half, workspace=ws)
    o, lse = nb.attn_fwd(None, None, v, BASE, workspace=ws, qk_rotated=True, Hq=Hq, rope_half=half)
    gq, gk, dv = nb.attn_bwd(None, None, v, o, lse, do, BASE, grad_dtype=torch.float32, workspace=ws, qk_rotated=True,
                             rope_half=half)
    dq, dk, dqw, dkw = nb.qk_norm_bwd(*dev, gq, gk, eps=EPS, dq=gq, dk=gk)
    nb.check_status()
    nq, nk = paged.rms_heads(ref[0], ref[2], EPS), paged.rms_heads(ref[1], ref[3], EPS)
    r = oracle_mod.attn_bwd(nq, nk, fv, fdo, BASE, half=half)
    rel, mx = H.errors(H.to_f64(o), r["o"])
    assert rel <= H.REL_L2_TOL and mx <= H.MAX_ABS_TOL
    for name, gx, gw, x, w, gn in (("q", dq, dqw, ref[0], ref[2], r["dq"]), ("k", dk, dkw, ref[1], ref[3], r["dk"])):
        rx, rw = paged.rms_heads_bwd(x, w, gn, EPS)
        assert H.errors(H.to_f64(gx), rx)[0] <= 2 * H.REL_L2_TOL, name
        assert H.errors(gw.cpu().numpy().astype(np.float64), rw)[0] <= 2 * H.REL_L2_TOL, name


def test_other_stream_and_graph(nb):
    """On a stream of its own, and captured into a graph replayed on new inputs."""
    dev, _ = make(2, 300, 12, 4, 64, 17, False)
    want = nb.rotated_qk(nb.qk_norm(*dev), 2, 300, 12, 4, 64)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = nb.rotated_qk(nb.qk_norm(*dev, stream=s), 2, 300, 12, 4, 64)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    q, k = torch.zeros_like(dev[0]), torch.zeros_like(dev[1])
    g = [torch.randn_like(q), torch.randn_like(k)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ws = nb.qk_norm(q, k, dev[2], dev[3])
        back = nb.qk_norm_bwd(q, k, dev[2], dev[3], g[0], g[1])
    q.copy_(dev[0])
    k.copy_(dev[1])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(nb.rotated_qk(ws, 2, 300, 12, 4, 64), want))
    eager = nb.qk_norm_bwd(dev[0], dev[1], dev[2], dev[3], g[0], g[1])
    assert all(torch.equal(a, b) for a, b in zip(back, eager))
