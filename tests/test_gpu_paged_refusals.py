"""What the binding of the query/key norms and the paged calls refuses before the library is called,
with tensors on the GPU."""
import types

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


def calls(nb):
    """The four calls on one small problem, by name."""
    bf = lambda *s: torch.randn(s, device="cuda").bfloat16()
    q, k, w = bf(1, 4, 4, 32), bf(1, 4, 2, 32), bf(32)
    kp, vp = nb.paged_cache(3, 16, 2, 32, "cuda")
    table = torch.tensor([[0, 2]], dtype=torch.int32, device="cuda")
    zero, four = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((1,), 4, dtype=torch.int32, device="cuda")
    return {
        "qk_norm": lambda **a: nb.qk_norm(q, k, w, w, **a),
        "qk_norm_bwd": lambda **a: nb.qk_norm_bwd(q, k, w, w, q, k, **a),
        "append": lambda **a: nb.kv_append_paged(k[0], k[0], kp, vp, table, zero, **a),
        "decode": lambda **a: nb.attn_decode_paged(q, kp, vp, table, four, **a),
    }


@pytest.mark.parametrize("name", ["qk_norm", "qk_norm_bwd", "decode"])
def test_workspaces(nb, name):
    """A workspace whose elements are not so many bytes of memory in a row."""
    call, n = calls(nb)[name], 1 << 20
    call(workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))
    nb.check_status()
    for ws in (torch.empty(1, dtype=torch.uint8, device="cuda").expand(n),
               torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2],
               torch.empty((n, 2), dtype=torch.uint8, device="cuda").t(),
               torch.empty(n, dtype=torch.int8, device="cuda"), torch.empty(n, dtype=torch.uint8)):
        with pytest.raises(ValueError):
            call(workspace=ws)
    with pytest.raises(nb.NeAttnError):
        call(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("name", ["qk_norm", "qk_norm_bwd", "append", "decode"])
def test_stream_of_another_device(nb, name):
    """The call would run on its own device's current stream, not behind the work of the given one."""
    call = calls(nb)[name]
    with pytest.raises(ValueError):
        call(stream=types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0))
    call(stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    nb.check_status()
