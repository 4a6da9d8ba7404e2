"""The status word: a timeout is not hidden by a bad page met before it (the library's counters are
cleared only after a timeout), and both are gone after they have been read."""
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


def bad_page(nb):
    k = torch.ones((1, 1, 32), device="cuda").bfloat16()
    kp, vp = nb.paged_cache(2, 16, 1, 32, "cuda")
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    nb.kv_append_paged(k, k, kp, vp, torch.full((1, 1), 9, dtype=torch.int32, device="cuda"), one)


@pytest.mark.parametrize("order", ["page, timeout", "timeout, page"])
def test_timeout_beside_a_bad_page(nb, order):
    for what in order.split(", "):
        if what == "page":
            bad_page(nb)
        else:
            nb.debug_timeout_probe(1000)
    assert nb.status_of_last_kernels() == -6
    assert nb.status_of_last_kernels() == 0


def test_bad_page_alone(nb):
    bad_page(nb)
    assert nb.status_of_last_kernels() == -8
    assert nb.status_of_last_kernels() == 0


def test_calls_on_another_stream_after_a_timeout(nb):
    """The stream's counters are cleared before the status is returned: a call right after, on a
    stream that does not wait for the legacy one, gives the usual result."""
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    kp, vp = r(400, 2, 16, 64).half(), r(400, 2, 16, 64).bfloat16()
    table = torch.arange(400, device="cuda", dtype=torch.int32).view(2, 200).contiguous()
    n = torch.tensor([3100, 2500], dtype=torch.int32, device="cuda")
    q = r(2, 1, 8, 64).bfloat16()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    want = nb.attn_decode_paged(q, kp, vp, table, n, stream=st)
    st.synchronize()
    for _ in range(20):
        nb.debug_timeout_probe(200)
        assert nb.status_of_last_kernels() == -6
        got = nb.attn_decode_paged(q, kp, vp, table, n, stream=st)
        st.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    nb.check_status()
