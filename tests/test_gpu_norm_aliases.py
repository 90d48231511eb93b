"""moe_add_rms_norm with outputs that are inputs: the bits of the call with buffers of its own."""
import numpy as np
import pytest
import torch

from shared_routed_expert_amd import _lib as L
from tests.gpu_util import DEV, make_layer, note, small_cfg
from tests.test_gpu_add_rms_norm import make, run, up
from workloads import generate

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [8, 120, 128, 384, 512, 1280, 5120, 10240])
@pytest.mark.parametrize("T", [1, 5, 700])
@pytest.mark.parametrize("res,y", [("x", "r"), ("r", "x"), ("x", None), (None, "r"), ("r", "own"), ("own", "x")])
def test_an_output_may_be_an_input(T, H, res, y):
    x, r, w = make(T, H, 2)
    note(f"norm in place T={T} H={H} residual_out={res} y={y}")
    mode = 1 if H % 128 == 0 and T == 5 else 0
    want = run(x, r, w, 1e-5, H, mode)
    dev = {"x": up(x.view(np.int16)), "r": up(r.view(np.int16)), "own": torch.empty((T, H), dtype=torch.int16, device=DEV)}
    xq = torch.empty((T, H), dtype=torch.uint8, device=DEV)
    sx = torch.empty((T, H // 128 if mode else 1), device=DEV)
    stride = H if T > 1 else H + 8   # (one row: no matter)
    L.moe_add_rms_norm(dev["x"], stride, dev["r"], dev.get(res), up(w), 1e-5, T, H, mode, dev.get(y), xq, sx)
    torch.cuda.synchronize()
    for a, b in zip(want, (dev.get(res), dev.get(y), xq, sx)):
        assert b is None or np.array_equal(a, b.cpu().numpy())


def test_outputs_between_the_rows_of_x():
    """x's rows are far apart, and the outputs lie between them: no overlap, nothing refused, x as it was."""
    T, H = 6, 256
    x, r, w = make(T, H, 3)
    want = run(x, r, w, 1e-5, H, 0)
    wide = torch.full((T, 8 * H * T), 0x7FC1, dtype=torch.int16, device=DEV)
    wide[:, :H] = up(x.view(np.int16))
    h, y = wide[0, H:H + T * H].view(T, H), wide[3, 2 * H:2 * H + T * H].view(T, H)
    xq, sx = torch.empty((T, H), dtype=torch.uint8, device=DEV), torch.empty((T, 1), device=DEV)
    L.moe_add_rms_norm(wide, wide.stride(0), up(r.view(np.int16)), h, up(w), 1e-5, T, H, 0, y, xq, sx)
    torch.cuda.synchronize()
    for a, b in zip(want, (h, y, xq, sx)):
        assert np.array_equal(a, b.cpu().numpy())
    assert np.array_equal(wide[:, :H].cpu().numpy(), x.view(np.int16))


def test_the_layers_own_call():
    """FusedMoE.add_norm: strided x with dense outputs, dense x in place, overlaps refused by the library."""
    T, H = 9, 256
    layer, _ = make_layer(generate(small_cfg("norm_alias", T=T, H=H, I=64, E=12, K=3, seed=5)), 16)
    x, r, w = make(T, H, 4, extra=H)
    want_h, want_y, _, _ = run(x, r, w, 1e-5, H, 0)
    dw = up(w)
    wide, res = up(x.view(np.int16)).view(torch.bfloat16), up(r.view(np.int16)).view(torch.bfloat16)
    y, h = layer.add_norm(wide[:, :H], dw, res)
    torch.cuda.synchronize()
    same = lambda t, bits: np.array_equal(t.view(torch.int16).cpu().numpy(), bits)
    assert same(y, want_y) and same(h, want_h)
    for bad in (dict(y=wide[:, :H]), dict(residual=wide[:, :H]), dict(residual_out=wide[:, :H])):
        with pytest.raises(ValueError):
            layer.add_norm(wide[:, :H], dw, **{**dict(residual=res), **bad})
    dense = torch.empty((T + 1, H), dtype=torch.bfloat16, device=DEV)
    dense[:T] = wide[:, :H]
    for bad in (dict(y=dense[1:]), dict(residual_out=dense[1:]), dict(y=res, residual_out=res)):
        with pytest.raises(L.SrmoeError):
            layer.add_norm(dense[:T], dw, **{**dict(residual=res), **bad})
    y, h = layer.add_norm(dense[:T], dw, res, residual_out=res, y=dense[:T])
    torch.cuda.synchronize()
    assert same(dense[:T], want_y) and same(res, want_h)
