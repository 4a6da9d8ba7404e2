"""Query/key norms and their backward on more rows than the blocks of one wave take at once: threads go
around their loops several times, the blocks are shared between q and k by their heads, and dw is summed
over every group of blocks. Bounds as in test_gpu_qk_norm; for dw, the terms of its longest chain: at most
24 rows a thread in these shapes, 2 additions among lanes, 8 among warps, 32 blocks of a group and 16 groups."""
import numpy as np
import pytest

import _harness as H
from oracle import paged
from test_gpu_qk_norm import BASE, EPS, bf16, make, nb, rotated  # noqa: F401  (nb is a fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# (B, T, Hq, Hkv, D): the 12/4 and 16/4 models, one key head for many query heads, D = 32, equal heads
SHAPES = [(16, 512, 12, 4, 64), (5, 1021, 16, 4, 64), (3, 1500, 32, 1, 64), (16, 1031, 4, 2, 32), (7, 999, 9, 9, 64)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("half,fused", [(False, True), (True, False)])
def test_forward(nb, shape, half, fused):
    dev, ref = make(*shape, seed=shape[1], fused=fused)
    n = nb.fwd_workspace_size(*shape)
    ws = torch.full((n + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    nb.qk_norm(*dev, eps=EPS, rope_base=BASE, rope_half=half, workspace=ws)
    nb.check_status()
    assert (ws[n:] == 0x5A).all()
    for got, x, w in zip(nb.rotated_qk(ws, *shape), ref[:2], ref[2:]):
        y, size = rotated(x, w, half)
        d = size * 2.0 ** -19
        assert (np.abs(H.to_f64(got) - y) <= (np.abs(y) + d) * 2.0 ** -11 + d + 2.0 ** -25).all()


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("fp32,fused", [(False, False), (True, True)])
def test_backward(nb, shape, fp32, fused):
    B, T, Hq, Hkv, D = shape
    dev, ref = make(*shape, seed=shape[1] + 1, fused=fused)
    rng = np.random.default_rng(8)
    g = [rng.standard_normal((B, T, h, D)).astype(np.float32) for h in (Hq, Hkv)]
    if fp32:
        gd, gf = [torch.from_numpy(x).cuda() for x in g], [x.astype(np.float64) for x in g]
    else:
        gd, gf = zip(*[bf16(x) for x in g])
    kw = {}
    if fused:
        out = torch.full((B, T, Hq + 2 * Hkv, D), 3.0, dtype=gd[0].dtype, device="cuda")
        kw = dict(dq=out[:, :, :Hq], dk=out[:, :, Hq:Hq + Hkv])
    got = nb.qk_norm_bwd(*dev, *gd, eps=EPS, **kw)
    nb.check_status()
    if fused:
        assert (out[:, :, Hq + Hkv:] == 3.0).all()
    for gx, gw, x, w, gg in zip(got[:2], got[2:], ref[:2], ref[2:], gf):
        rx, rw = paged.rms_heads_bwd(x, w, gg, EPS)
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
        xh = x * r
        tol = 2.0 ** -18 * r * (np.abs(w * gg) + np.abs(xh) * np.abs(w * gg * xh).mean(-1, keepdims=True))
        if not fp32:
            tol = tol + (np.abs(rx) + tol) * 2.0 ** -8
        assert (np.abs(H.to_f64(gx) - rx) <= tol + 1e-37).all()
        terms = 24 + 2 + 8 + 32 + 16
        assert (np.abs(gw.cpu().numpy() - rw) <= 2.0 ** -24 * (terms + 8) * np.abs(gg * xh).reshape(-1, D).sum(0)).all()
    ws = torch.empty(int(nb.lib().ne_attn_qk_norm_bwd_workspace_size(*shape)), dtype=torch.uint8, device="cuda")
    again = nb.qk_norm_bwd(*dev, *gd, eps=EPS, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
