"""Rotary tables that a call needs for the first time: the host does not wait for what is queued on
the call's stream, calls on other streams see a finished table, and a captured call may need one too."""
import numpy as np
import pytest

from oracle import paged

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

B, Hq, Hkv, D, CAP = 2, 4, 2, 64, 4096


@pytest.fixture(scope="module")
def nb():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_gqa_attention_flashattention_gb300 import binding
    binding.lib()
    return binding


@pytest.fixture(scope="module")
def bases():
    """A base that no call has had before, one after another."""
    return iter(20000.0 + 7 * i for i in range(10 ** 6))


def rows(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn((B, 40, h, D), generator=g, device="cuda").bfloat16() for h in (Hq, Hkv, Hkv)]


def step(nb, x, base, **kw):
    """Keys appended at far positions of a contiguous cache."""
    q, k, v = x
    kc, vc = nb.kv_cache(B, CAP, Hkv, D, "cuda")
    nb.kv_append(k, v, kc, vc, CAP - 40, rope_base=base, **kw)
    return kc


def norm(nb, x, base, **kw):
    w = torch.ones(D, device="cuda").bfloat16()
    return nb.rotated_qk(nb.qk_norm(x[0], x[1], w, w, rope_base=base, **kw), B, 40, Hq, Hkv, D)


def test_host_does_not_wait(nb, bases):
    x = rows(1)
    step(nb, x, next(bases))  # kernels loaded
    kc, vc = nb.kv_cache(B, CAP, Hkv, D, "cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    base, done = next(bases), torch.cuda.Event()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2 * 10 ** 9)  # about a second
        nb.kv_append(x[1], x[2], kc, vc, CAP - 40, rope_base=base)
        done.record()
    waited = done.query()
    torch.cuda.synchronize()
    assert not waited
    assert torch.equal(kc, step(nb, x, base))


def test_streams_find_a_finished_table(nb, bases):
    """Two streams need one new table at the same time, twenty times over; the second call's own
    stream has nothing queued before it."""
    x = rows(2)
    norm(nb, x, next(bases))
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        base = next(bases)
        torch.cuda.synchronize()
        with torch.cuda.stream(a):
            torch.cuda._sleep(10 ** 7)
            one = norm(nb, x, base)
        with torch.cuda.stream(b):
            two = norm(nb, x, base)
        torch.cuda.synchronize()
        three = norm(nb, x, base)
        for p, q, r in zip(one, two, three):
            assert torch.equal(p, r) and torch.equal(q, r)


@pytest.mark.parametrize("mode", ["global", "thread_local", "relaxed"])
def test_captured_call_with_a_new_table(nb, bases, mode):
    x = rows(3)
    norm(nb, x, next(bases))
    base = next(bases)
    ws = torch.zeros(nb.fwd_workspace_size(B, 40, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode=mode):
        got = norm(nb, x, base, workspace=ws)
        step(nb, x, base)
    eager = [t.clone() for t in norm(nb, x, base)]
    for _ in range(2):
        ws.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, eager))


def test_capture_right_after_the_build(nb, bases):
    """The table's build is queued, not finished, when a captured call needs it."""
    x = rows(4)
    norm(nb, x, next(bases))
    for _ in range(5):
        base, g = next(bases), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            first = step(nb, x, base)   # needs CAP rows
            got = norm(nb, x, base)     # finds them
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, norm(nb, x, base)))
        assert torch.equal(first, step(nb, x, base))


def test_growing_contexts_keep_few_tables(nb, bases):
    """Contexts that grow by 2048 positions at a time up to 65536: tables of 2048, 4096, 8192, ... 65536
    rows, 32 MB in all where one for each step would be 277 MB.  The keys are rotated as the oracle has
    it, to the append's bound (the fp16 rounding and 2^-19 of the pair)."""
    k = torch.randn((1, 1, 1, D), device="cuda").bfloat16()
    kc, vc = nb.kv_cache(1, 65536, 1, D, "cuda")
    put = lambda pos, base: nb.kv_append(k, k, kc, vc, pos, rope_base=base)
    put(0, next(bases))
    base = next(bases)
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    last = [2048 * i - 1 for i in range(1, 33)]
    for pos in last:
        put(pos, base)
    torch.cuda.synchronize()
    assert free - torch.cuda.mem_get_info()[0] < 64 << 20
    x = k[0].double().cpu().numpy()
    want = paged.rope_at(np.repeat(x, len(last), 0), last, base)[:, 0]
    pair = np.repeat(np.linalg.norm(x[0, 0].reshape(D // 2, 2), axis=-1), 2) * 2.0 ** -19
    got = kc[0, 0, last].double().cpu().numpy()
    assert (np.abs(got - want) <= (np.abs(want) + pair) * 2.0 ** -11 + pair + 2.0 ** -25).all()
