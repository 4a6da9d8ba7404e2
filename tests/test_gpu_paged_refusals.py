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


def test_workspace_for_training(nb):
    """The workspace that qk_norm allocates is the forward's: the backward refuses it, and takes alloc_workspace's."""
    bf = lambda *s: torch.randn(s, device="cuda").bfloat16()
    B, T, Hq, Hkv, D = 1, 200, 4, 2, 64
    q, k, v, do, w = bf(B, T, Hq, D), bf(B, T, Hkv, D), bf(B, T, Hkv, D), bf(B, T, Hq, D), bf(D)
    short, enough = nb.qk_norm(q, k, w, w), nb.qk_norm(q, k, w, w, workspace=nb.alloc_workspace(B, T, Hq, Hkv, D))
    out = [nb.attn_fwd(None, None, v, workspace=ws, qk_rotated=True, Hq=Hq) for ws in (short, enough)]
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    with pytest.raises(nb.NeAttnError):
        nb.attn_bwd(None, None, v, *out[0], do, workspace=short, qk_rotated=True)
    assert all(torch.isfinite(g.float()).all() for g in nb.attn_bwd(None, None, v, *out[1], do, workspace=enough, qk_rotated=True))
    nb.check_status()
