"""CPU checks of the drafted trees' entry points: argument errors are found on the host before the
device is touched."""
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


PLAN = "table ring held span len new parents held_o span_o len_o cu slots pos N B Tq page P width pstride stream"
APPEND = "k v kw kp vp slots pos N Hkv D page P cap stride ks vs eps base flags stream"
TREE = "q qw kp vp table len parents nodes o lse B Tq Hq Hkv D page P width stride qs pstride eps base flags ws bytes stream"
KEEP = "kp vp table len nodes path count out B tokens width Hkv D page P tw stride stream"


def test_plan(libne, mem):
    p = mem[1]
    good = dict(table=p, ring=p, held=p, span=p, len=p, new=p, parents=p, held_o=p, span_o=p, len_o=p + 64, cu=p, slots=p,
                pos=p, N=5, B=2, Tq=4, page=16, P=4, width=3, pstride=4, stream=None)
    f = lambda **c: call(libne.ne_attn_paged_plan, PLAN, good, **c)
    for name in "table ring held span len new held_o span_o len_o cu slots pos".split():
        assert f(**{name: None}) == -1
    for name in "table ring held span len new parents held_o span_o len_o cu slots pos".split():
        assert f(**{name: p + 2}) == -2
    assert f(len_o=p) == -1                       # the old lengths are read until the end
    assert f(N=-1) == -1 and f(B=0) == -1 and f(P=0) == -1 and f(width=0) == -1
    assert f(N=0, slots=None, pos=None, page=8) == -3
    assert f(page=8) == -3 and f(page=48) == -3 and f(page=512) == -3
    assert f(B=2049) == -3 and f(width=(1 << 16) + 1) == -3 and f(P=1 << 27) == -3 and f(N=(1 << 30) + 1) == -3
    assert f(Tq=0) == -1 and f(Tq=65, pstride=65) == -3 and f(pstride=3) == -1 and f(pstride=-4) == -1


def test_append_slots(libne, mem):
    p = mem[1]
    good = dict(k=p, v=p, kw=p, kp=p, vp=p, slots=p, pos=p, N=5, Hkv=2, D=32, page=16, P=4, cap=100, stride=1024, ks=64,
                vs=64, eps=1e-6, base=1e4, flags=0, stream=None)
    f = lambda **c: call(libne.ne_attn_kv_append_slots, APPEND, good, **c)
    for name in "k v kp vp slots pos".split():
        assert f(**{name: None}) == -1
    for name in "k v kw kp vp".split():
        assert f(**{name: p + 8}) == -2
    for name in "slots pos".split():
        assert f(**{name: p + 2}) == -2
    assert f(N=0) == -1 and f(P=0) == -1 and f(cap=0) == -1 and f(cap=(1 << 20) + 1) == -3
    assert f(page=8) == -3 and f(page=48) == -3 and f(D=48) == -3 and f(P=1 << 27) == -3
    assert f(stride=1023) == -1 and f(ks=60) == -1 and f(vs=76) == -1
    assert f(eps=0.0) == -1 and f(base=0.5) == -1 and f(flags=1) == -1


def test_decode_tree(libne, mem):
    p = mem[1]
    size = libne.ne_attn_decode_tree_workspace_size
    n = size(2, 5, 4, 2, 32)
    assert 0 < n and n % 256 == 0
    assert size(2, 0, 4, 2, 32) == 0 and size(0, 1, 4, 2, 32) == 0 and size(2, 1, 3, 2, 32) == 0
    assert size(2, 1, 4, 2, 48) == 0 and size(2, 65, 4, 2, 32) == 0 and size(2048, 64, 4096, 1, 64) == 0
    good = dict(q=p, qw=p, kp=p, vp=p, table=p, len=p, parents=p, nodes=p, o=p, lse=p, B=2, Tq=5, Hq=4, Hkv=2, D=32, page=16,
                P=4, width=3, stride=1024, qs=128, pstride=5, eps=1e-6, base=1e4, flags=0, ws=p, bytes=1 << 40, stream=None)
    f = lambda **c: call(libne.ne_attn_decode_tree, TREE, good, **c)
    for name in "q kp vp table len parents o".split():
        assert f(**{name: None}) == -1
    for name in "q qw kp vp o".split():
        assert f(**{name: p + 8}) == -2
    for name in "lse table len parents nodes".split():
        assert f(**{name: p + 2}) == -2
    assert f(Tq=0) == -1 and f(Tq=65, pstride=65) == -3 and f(Hq=3) == -1 and f(B=0) == -1 and f(B=5000) == -3
    assert f(page=24) == -3 and f(D=128) == -3 and f(qs=120) == -1 and f(stride=1000) == -1
    assert f(pstride=4) == -1 and f(pstride=-1) == -1
    assert f(B=2048, Hq=64, Hkv=64, page=256, width=4096, stride=64 * 256 * 32, qs=64 * 32) == -3
    assert f(eps=0.0) == -1 and f(base=float("inf")) == -1 and f(flags=2) == -1 and f(flags=8) == -1
    assert f(bytes=n - 1) == -5 and f(ws=p + 64) == -5


@pytest.mark.parametrize("fp32", [0, 1])
def test_tree_outputs_on_the_queries(libne, mem, fp32):
    """q has 10 rows of 128 values 160 apart, 3136 bytes; o 10 of 128, 2560 bytes or 5120: any common byte is refused."""
    p = mem[1]
    good = dict(q=p + 8192, qw=p, kp=p, vp=p, table=p, len=p, parents=p, nodes=p, o=p, lse=p, B=2, Tq=5, Hq=4, Hkv=2, D=32, page=16,
                P=4, width=3, stride=1024, qs=160, pstride=5, eps=1e-6, base=1e4, flags=fp32, ws=p, bytes=1 << 40, stream=None)
    f = lambda **c: call(libne.ne_attn_decode_tree, TREE, good, **c)
    q, n = p + 8192, 5120 if fp32 else 2560
    for o in (q, q + 16, q + 3136 - 16, q - 16, q - n + 16):
        assert f(o=o) == -1


def test_keep(libne, mem):
    p = mem[1]
    good = dict(kp=p, vp=p, table=p, len=p, nodes=p, path=p, count=p, out=p + 64, B=2, tokens=0, width=4, Hkv=2, D=32,
                page=16, P=4, tw=3, stride=1024, stream=None)
    f = lambda **c: call(libne.ne_attn_kv_keep_paged, KEEP, good, **c)
    for name in "kp vp table len path count out".split():
        assert f(**{name: None}) == -1
    for name in "kp vp".split():
        assert f(**{name: p + 8}) == -2
    for name in "table len nodes path count out".split():
        assert f(**{name: p + 2}) == -2
    assert f(out=p) == -1 and f(width=0) == -1 and f(width=65) == -3 and f(tokens=-1) == -1
    assert f(B=0) == -1 and f(D=128) == -3 and f(page=20) == -3 and f(stride=1000) == -1 and f(P=0) == -1


def test_status_text(libne):
    assert b"tree" in libne.ne_attn_status_string(-9)


def test_binding_refusals():
    """Shapes, types and devices the binding refuses before it calls the library."""
    torch = pytest.importorskip("torch")
    from causal_gqa_attention_flashattention_gb300 import binding as nb
    q = torch.zeros((1, 4, 4, 32), dtype=torch.bfloat16)
    kp, vp = nb.paged_cache(3, 16, 2, 32, "cpu")
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(ValueError):
        nb.paged_plan(i(1, 2), i(3), i(1), i(2), i(1), i(1), 4, 16)
    with pytest.raises(ValueError):
        nb.kv_append_slots(q[0, :, :2], q[0, :, :2], kp, vp, i(4), i(4), 32)
    with pytest.raises(ValueError):
        nb.attn_decode_tree(q, kp, vp, i(1, 2), i(1), i(1, 4))
    with pytest.raises(ValueError):
        nb.kv_keep_paged(kp, vp, i(1, 2), i(1), 4, i(1, 4), i(1))
