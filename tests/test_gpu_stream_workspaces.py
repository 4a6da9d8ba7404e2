"""The library's own workspaces per stream: a stream that is used on every step keeps its own
however many others come and go."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nb():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_gqa_attention_flashattention_gb300 import binding
    binding.lib()
    return binding


def test_a_stream_in_use_keeps_its_workspace(nb):
    """70 streams are used once each, the main one after each of them behind a tenth of a second of queued
    work, and its call returns at once: a workspace that had gone would be made anew, for which
    another has to be freed, and that waits for the device."""
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    kp, vp, q = r(60, 2, 64, 64).half(), r(60, 2, 64, 64).bfloat16(), r(1, 1, 8, 64).bfloat16()
    table = torch.arange(60, device="cuda", dtype=torch.int32).view(1, 60)
    n = torch.tensor([3800], dtype=torch.int32, device="cuda")
    call = lambda: nb.attn_decode_paged(q, kp, vp, table, n)
    want = call()
    main = torch.cuda.Stream()
    torch.cuda.synchronize()
    rt, handles = torch.cuda.cudart(), []
    try:
        with torch.cuda.stream(main):
            call()
        for _ in range(70):
            h = ctypes.c_void_p()
            assert int(rt.cudaStreamCreate(ctypes.addressof(h))) == 0
            handles.append(h.value)
            with torch.cuda.stream(torch.cuda.ExternalStream(h.value)):
                got = call()
            torch.cuda.synchronize()
            done = torch.cuda.Event()
            with torch.cuda.stream(main):
                torch.cuda._sleep(2 * 10 ** 8)
                mine = call()
                done.record()
            waited = done.query()
            torch.cuda.synchronize()
            assert not waited
            assert torch.equal(got[0], want[0]) and torch.equal(mine[0], want[0])
    finally:
        torch.cuda.synchronize()
        for h in handles:
            rt.cudaStreamDestroy(h)
    nb.check_status()
