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


# Bases of 2 MiB each that no call touches: every refusal comes before a launch.
X, R, RO, W, Y, XQ, SX = (0x1000000 + 0x200000 * i for i in range(7))
INVALID = -1


def norm(**kw):
    from shared_routed_expert_amd import _lib as L
    a = dict(x=X, x_stride=H, residual=R, residual_out=RO, weight=W, eps=1e-5, T=T, H=H, scale_mode=0, y=Y, xq=XQ, sx=SX)
    a.update(kw)
    return L.moe_add_rms_norm(**a, stream=0, check=False)


def test_rejects_outputs_that_are_x_where_its_rows_are_strided():
    for kw in (dict(y=X), dict(residual_out=X), dict(y=X, residual_out=R), dict(y=X, residual=None, residual_out=None)):
        assert norm(x_stride=2 * H, **kw) == INVALID, kw


def test_rejects_outputs_that_overlap():
    row, size = 2 * H, 2 * T * H
    one = dict(xq=None, sx=None)
    for kw in (dict(y=RO), dict(y=R, residual_out=R), dict(y=X, residual_out=X),                 # the same for both
               dict(y=RO + row), dict(residual_out=Y + size - 16),                               # a part of one another
               dict(y=X + row), dict(y=X - row), dict(residual_out=X + size - 16), dict(residual_out=R + 16),
               dict(y=R - size + 16, **one), dict(y=X + row, x_stride=3 * H), dict(y=X + 5 * row, x_stride=2 * H),
               dict(y=W), dict(residual_out=W + 4 * H - 16), dict(xq=X), dict(xq=X + size - 16), dict(xq=R), dict(xq=Y),
               dict(xq=RO + 16), dict(xq=W), dict(sx=W), dict(sx=X + 16), dict(sx=R), dict(sx=Y), dict(sx=RO),
               dict(sx=XQ + T * H - 16), dict(xq=SX), dict(sx=XQ - 16, scale_mode=1)):
        assert norm(**kw) == INVALID, kw


def test_pointers_apart_are_still_looked_at():
    for name in ("x", "residual", "residual_out", "weight", "y", "xq", "sx"):
        assert norm(**{name: 0x10000 + 4}) == INVALID, name
    for kw in (dict(x=None), dict(weight=None), dict(xq=None), dict(sx=None), dict(y=None, xq=None, sx=None)):
        assert norm(**kw) == INVALID, kw
