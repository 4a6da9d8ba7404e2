"""CPU checks of the query/key norms' and the paged cache's entry points: argument
errors are found on the host before the device is touched."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def libne():
    from causal_gqa_attention_flashattention_gb300 import build, binding
    build.build()
    return binding.lib()


@pytest.fixture(scope="module")
def mem():
    buf = ctypes.create_string_buffer(1 << 16)
    base = (ctypes.addressof(buf) + 255) // 256 * 256
    return buf, base


def call(fn, names, good, **change):
    args = dict(good, **change)
    return fn(*[args[n] for n in names.split()])


NORM = "q k qw kw B T Hq Hkv D qs ks eps base flags ws bytes stream"
NORM_BWD = "q k qw kw gq gk dq dk dqw dkw B T Hq Hkv D qs ks dqs dks eps flags ws bytes stream"
APPEND = "k v kw kp vp table pos0 cu N B Hkv D page P width pstride ks vs eps base flags stream"
DECODE = "q qw kp vp table len ptable o lse B Tq Hq Hkv D page P width pstride qs prefix eps base flags ws bytes stream"


def test_qk_norm(libne, mem):
    p = mem[1]
    good = dict(q=p, k=p, qw=p, kw=p, B=1, T=4, Hq=4, Hkv=2, D=32, qs=128, ks=64, eps=1e-6, base=1e4, flags=0, ws=p,
                bytes=1 << 15, stream=None)
    f = lambda **c: call(libne.ne_attn_qk_norm, NORM, good, **c)
    for n in ("q", "k", "qw", "kw"):
        assert f(**{n: None}) == -1
        assert f(**{n: p + 2}) == -2
    assert f(eps=0.0) == -1 and f(eps=float("nan")) == -1 and f(eps=float("inf")) == -1
    assert f(base=1.0) == -1
    assert f(flags=8) == -1 and f(flags=4) == -1
    assert f(Hq=3) == -1 and f(T=0) == -1 and f(D=48) == -3
    assert f(qs=127) == -1 and f(qs=124) == -1 and f(ks=63) == -1 and f(ks=0) == -1
    assert f(ws=None) == -5 and f(ws=p + 16) == -5 and f(bytes=100) == -5
    # the workspace is the forward's
    n = libne.ne_attn_fwd_workspace_size(1, 4, 4, 2, 32, 0)
    assert f(bytes=n - 1) == -5


def test_qk_norm_bwd(libne, mem):
    p = mem[1]
    n = libne.ne_attn_qk_norm_bwd_workspace_size(1, 4, 4, 2, 32)
    assert n > 0 and n % 256 == 0
    assert libne.ne_attn_qk_norm_bwd_workspace_size(1, 4, 4, 3, 32) == 0
    assert libne.ne_attn_qk_norm_bwd_workspace_size(1, 4, 4, 2, 40) == 0
    good = dict(q=p, k=p, qw=p, kw=p, gq=p, gk=p, dq=p, dk=p, dqw=p, dkw=p, B=1, T=4, Hq=4, Hkv=2, D=32, qs=128, ks=64,
                dqs=128, dks=64, eps=1e-6, flags=0, ws=p, bytes=n, stream=None)
    f = lambda **c: call(libne.ne_attn_qk_norm_bwd, NORM_BWD, good, **c)
    for name in "q k qw kw gq gk dq dk dqw dkw".split():
        assert f(**{name: None}) == -1
        assert f(**{name: p + 8}) == -2
    assert f(eps=-1.0) == -1 and f(flags=16) == -1 and f(flags=1) == -1
    assert f(dqs=120) == -1 and f(dks=60) == -1 and f(qs=132) == -1
    assert f(bytes=n - 1) == -5 and f(ws=p + 128) == -5


def test_kv_append_paged(libne, mem):
    p = mem[1]
    good = dict(k=p, v=p, kw=p, kp=p, vp=p, table=p, pos0=p, cu=p, N=5, B=2, Hkv=2, D=32, page=16, P=4, width=3,
                pstride=1024, ks=64, vs=64, eps=1e-6, base=1e4, flags=0, stream=None)
    f = lambda **c: call(libne.ne_attn_kv_append_paged, APPEND, good, **c)
    for name in "k v kp vp table pos0".split():
        assert f(**{name: None}) == -1
    for name in "k v kw kp vp".split():
        assert f(**{name: p + 8}) == -2
    for name in "table pos0 cu".split():
        assert f(**{name: p + 2}) == -2
    assert f(cu=None) == -1                      # 5 rows do not divide into 2 sequences
    assert f(N=0) == -1 and f(B=0) == -1 and f(P=0) == -1 and f(width=0) == -1
    assert f(page=8) == -3 and f(page=48) == -3 and f(page=512) == -3 and f(D=48) == -3
    assert f(B=2049) == -3 and f(width=(1 << 16) + 1) == -3
    assert f(pstride=1023) == -1 and f(pstride=1028) == -1 and f(pstride=1 << 40) == -3
    assert f(ks=60) == -1 and f(vs=72 + 4) == -1
    assert f(eps=0.0) == -1 and f(base=0.5) == -1 and f(flags=1) == -1
    assert f(kw=None, eps=0.0, flags=1) == -1    # eps is not looked at without a weight, the flag is


def test_decode_paged(libne, mem):
    p = mem[1]
    size = libne.ne_attn_decode_paged_workspace_size
    n = size(2, 1, 4, 2, 32, 0)
    assert 0 < n and n % 256 == 0
    assert size(2, 1, 4, 2, 32, 64) >= n
    assert size(2, 0, 4, 2, 32, 0) == 0 and size(0, 1, 4, 2, 32, 0) == 0 and size(2, 1, 3, 2, 32, 0) == 0
    assert size(2, 1, 4, 2, 48, 0) == 0 and size(2, 65, 4, 2, 32, 0) == 0 and size(2, 1, 4, 2, 32, -16) == 0
    good = dict(q=p, qw=p, kp=p, vp=p, table=p, len=p, ptable=None, o=p, lse=p, B=2, Tq=1, Hq=4, Hkv=2, D=32, page=16,
                P=4, width=3, pstride=1024, qs=128, prefix=0, eps=1e-6, base=1e4, flags=0, ws=p, bytes=1 << 40,
                stream=None)
    f = lambda **c: call(libne.ne_attn_decode_paged, DECODE, good, **c)
    for name in "q kp vp table len o".split():
        assert f(**{name: None}) == -1
    for name in "q qw kp vp o".split():
        assert f(**{name: p + 8}) == -2
    for name in "lse table len ptable".split():
        assert f(**{name: p + 2}) == -2
    assert f(Tq=0) == -1 and f(Tq=65) == -3 and f(Hq=3) == -1 and f(B=0) == -1 and f(B=5000) == -3
    assert f(page=24) == -3 and f(D=128) == -3 and f(qs=120) == -1 and f(pstride=1000) == -1
    assert f(prefix=16) == -1                    # needs its table
    # more key tiles than the sweep counts
    assert f(B=2048, Hq=64, Hkv=64, page=256, width=4096, pstride=64 * 256 * 32, qs=64 * 32) == -3
    assert f(prefix=-16, ptable=p) == -1 and f(prefix=24, ptable=p) == -1 and f(prefix=64, ptable=p) == -1
    assert f(eps=0.0) == -1 and f(base=float("inf")) == -1 and f(flags=2) == -1 and f(flags=4) == -1
    assert f(bytes=n - 1) == -5 and f(ws=p + 64) == -5


def test_status_text(libne):
    assert b"page" in libne.ne_attn_status_string(-8)


def test_binding_refusals():
    """Shapes, types and layouts the binding refuses before it calls the library."""
    torch = pytest.importorskip("torch")
    from causal_gqa_attention_flashattention_gb300 import binding as nb
    q = torch.zeros((1, 4, 4, 32), dtype=torch.bfloat16)
    k = torch.zeros((1, 4, 2, 32), dtype=torch.bfloat16)
    w = torch.ones(32, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        nb.qk_norm(q, k, w, w)                    # not on a CUDA device
    with pytest.raises(ValueError):
        nb.qk_norm(q, k[:, :3], w, w)
    with pytest.raises(ValueError):
        nb.qk_norm_bwd(q, k, w, w, q.half(), k.half())
    kp, vp = nb.paged_cache(3, 16, 2, 32, "cpu")
    table, one = torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        nb.kv_append_paged(k[0], k[0], kp, vp, table, one)
    with pytest.raises(ValueError):
        nb.attn_decode_paged(q[:, :1], kp, vp, table, one)
