"""moe_add_rms_norm against the float64 oracle, with bars that count what the kernel does. With u = 2^-24:
  a row's sum of squares: A additions that round, in a thread (8 squares for each stripe that it holds), in the log2 of the
      row's lanes of a wave, and over the waves; each h is rounded once, so a square is off by 2 u
  rstd: half of (2 + A, the mean's quotient, eps), the square root and the reciprocal: (A / 2 + 4) u
  y: h and two products more, (A / 2 + 7) u.  sx: h, a product, the product or quotients with rstd and 448, (A / 2 + 8) u = e
  residual_out: (2^-8 + u) |h|       y (bf16): (2^-8 + e) |y|       xq sx: (2^-4 + e) |y| + 2^-10 sx, half a step of e4m3
"""
import numpy as np
import pytest

import oracle
from tests.gpu_util import note
from tests.test_gpu_add_rms_norm import make, run, values

pytestmark = pytest.mark.gpu


def additions(H):
    """(stripes of a thread) * 8 + log2 of a row's lanes in a wave + waves, as launch_quant has them."""
    if H <= 128:
        return 8 + 4
    if H <= 512:
        return 8 + 6
    pieces = -(-H // 512)
    stripes = 1 if pieces <= 4 else 2 if pieces <= 16 else 4 if pieces <= 64 else 8
    return 8 * stripes + 6 + -(-pieces // stripes)


@pytest.mark.parametrize("H", [8, 16, 24, 64, 120, 128, 136, 256, 384, 512, 520, 1024, 2048, 2056, 5120, 8192, 8200, 16384, 32768,
                               32776, 65536])
@pytest.mark.parametrize("T", [1, 17, 64])
def test_values(T, H):
    e = 2.0 ** -24 * (additions(H) / 2 + 8)
    for mode in (0, 1):
        if mode and H % 128:
            continue
        for eps in (1e-5, 0.0):
            x, r, w = make(T, H, H + 3 * T)
            note(f"norm bars T={T} H={H} mode={mode} eps={eps}")
            h, y = oracle.add_rms_norm(values(x), values(r), w, eps)
            gh, gy, gq, gs = run(x, r, w, eps, H, mode)
            assert np.all(np.abs(values(gh.view(np.uint16)) - h) <= (2.0 ** -8 + 2.0 ** -24) * np.abs(h))
            err = np.abs(values(gy.view(np.uint16)) - y)
            assert np.all(err <= (2.0 ** -8 + e) * np.abs(y))
            s = oracle.act_scales(y, 128 if mode else None)
            assert np.all(np.abs(gs - s) <= e * s), float(np.max(np.abs(gs - s) / s) / e)
            wide = np.repeat(gs.astype(np.float64), H // gs.shape[1], axis=1)
            err = np.abs(oracle.e4m3_decode(gq) * wide - y)
            assert np.all(err <= (2.0 ** -4 + e) * np.abs(y) + 2.0 ** -10 * wide)
