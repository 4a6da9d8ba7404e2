"""Trees without any token are refused: they are not the same as no trees."""
import pytest

from test_gpu_tree import i32, nb, setup  # noqa: F401 (nb is a fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(0,), (2, 0)])
def test_empty_parents(nb, shape):
    none = torch.empty(shape, dtype=torch.int32, device="cuda")
    table = i32([[0, -1], [1, -1]])
    args = (i32([2, 3]), i32([1, 1]), i32([0, 2]), i32([3, 4]), i32([2, 1]), 3, 16)
    with pytest.raises(ValueError):
        nb.paged_plan(table, *args, parents=none)
    assert nb.paged_plan(table, *args).positions.tolist() == [3, 4, 4]  # without trees
    s = setup([40, 20], [4, 4], 4, 4, 2, 64, 16, seed=1)
    with pytest.raises(ValueError):
        nb.attn_decode_tree(s["q"], s["kp"], s["vp"], s["table"], s["lens"], none)
    with pytest.raises(ValueError):
        nb.attn_decode_tree(s["q"][:, :0], s["kp"], s["vp"], s["table"], s["lens"], none)
    nb.check_status()
