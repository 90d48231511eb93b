"""Host-side checks of moe_add_rms_norm (no GPU needed): every refusal comes before a launch, with fake 16-byte aligned
pointers that are never dereferenced; the oracle against torch."""
import numpy as np
import pytest
import torch

import oracle

FAKE, MIS = 0x10000, 0x10004


@pytest.fixture(scope="module")
def L():
    from shared_routed_expert_amd import _lib
    return _lib


def norm(L, **kw):
    a = dict(x=FAKE, x_stride=256, residual=FAKE, residual_out=FAKE, weight=FAKE, eps=1e-5, T=4, H=256, scale_mode=0, y=FAKE,
             xq=FAKE, sx=FAKE)
    a.update(kw)
    return L.moe_add_rms_norm(**a, stream=0, check=False)


def test_rejects(L):
    for kw in (dict(T=-1), dict(T=(1 << 20) + 1), dict(H=0), dict(H=-8), dict(eps=-1e-9), dict(eps=float("nan")), dict(eps=1e30),
               dict(scale_mode=2), dict(scale_mode=-1), dict(x_stride=248), dict(x_stride=260), dict(x_stride=1 << 40),
               dict(y=None, xq=None, sx=None), dict(xq=None), dict(sx=None)):
        assert norm(L, **kw) == -1, kw
    for kw in (dict(H=252), dict(H=65544, x_stride=1 << 20), dict(H=136, scale_mode=1)):
        assert norm(L, **kw) == -2, kw
    for name in ("x", "weight"):
        assert norm(L, **{name: None}) == -1, name
    for name in ("x", "residual", "residual_out", "weight", "y", "xq", "sx"):
        assert norm(L, **{name: MIS}) == -1, name
    assert norm(L, T=0, x=None) == 0
    # a shape that only the scales refuse is no matter where none are asked for
    assert norm(L, T=0, H=136, scale_mode=1, xq=None, sx=None) == 0


def test_oracle_against_torch():
    rng = np.random.default_rng(0)
    x, r, w = rng.standard_normal((5, 256)), rng.standard_normal((5, 256)), rng.standard_normal(256)
    h, y = oracle.add_rms_norm(x, r, w, 1e-3)
    t = torch.from_numpy(x + r)
    ref = torch.nn.functional.rms_norm(t, (256,), torch.from_numpy(w), 1e-3)
    assert np.allclose(h, x + r, rtol=0, atol=0) and np.allclose(y, ref.numpy(), rtol=1e-13, atol=1e-13)
    assert np.array_equal(oracle.add_rms_norm(x, None, w, 0.0)[0], x)
    assert np.allclose(oracle.act_scales(y, None)[:, 0] * 448, np.abs(y).max(axis=1), rtol=1e-15)
    assert oracle.act_scales(y, 128).shape == (5, 2) and np.all(oracle.act_scales(0 * y, 128) == 1.0)


def test_layer_object_rejects():
    """FusedMoE.add_norm's own checks, on CPU tensors (its constructor allocates, and nothing is launched)."""
    from shared_routed_expert_amd import FusedMoE
    m = FusedMoE(4, 256, 64, 8, 2, 16, 0, device="cpu")
    x, w = torch.zeros((4, 256), dtype=torch.bfloat16), torch.ones(256)
    for bad in (dict(x=x.float()), dict(x=x[:3]), dict(x=x.T.contiguous().T), dict(weight=w.double()), dict(weight=w[:128]),
                dict(weight=torch.ones(512)[::2]), dict(residual=x.float()), dict(residual=x[:, :128]),
                dict(residual=torch.zeros((4, 512), dtype=torch.bfloat16)[:, :256]), dict(y=x.half()), dict(x=None),
                dict(weight=None)):
        with pytest.raises(ValueError):
            m.add_norm(**{**dict(x=x, weight=w), **bad})
    with pytest.raises(ValueError, match="not on a GPU"):
        m.add_norm(x, w)
