"""Which of add_norm's tensors may be one another (no GPU needed: nothing is launched)."""
import pytest
import torch

T, H = 4, 256


def layer():
    from shared_routed_expert_amd import FusedMoE
    return FusedMoE(T, H, 64, 8, 2, 16, 0, device="cpu")


def wide():
    """[T, H] rows of a buffer of 2 H columns."""
    return torch.zeros((T, 2 * H), dtype=torch.bfloat16)[:, :H]


@pytest.mark.parametrize("name", ["residual", "residual_out", "y"])
def test_only_x_may_have_strided_rows(name):
    """Also where the other tensor is the same object as x: the library takes its rows to be H values apart."""
    m, w, x = layer(), torch.ones(H), wide()
    with pytest.raises(ValueError, match=f"{name} is contiguous"):
        m.add_norm(x, w, **{name: x})
    with pytest.raises(ValueError, match="not on a GPU"):   # x alone, and dense rows of every tensor, pass the checks
        m.add_norm(x, w, **{name: torch.zeros((T, H), dtype=torch.bfloat16)})
    dense = torch.zeros((T, H), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="not on a GPU"):
        m.add_norm(dense, w, **{name: dense})


@pytest.mark.parametrize("name", ["residual", "residual_out"])
def test_the_whole_block_behind_the_attention(name):
    m, w, x = layer(), torch.ones(H), wide()
    with pytest.raises(ValueError, match=f"{name} is contiguous"):
        m.forward_normed(x, w, None, None, None, **{name: x})
