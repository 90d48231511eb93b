"""moe_add_rms_norm where h^2, a row's sum of them, or h w leaves float32's normal range and y = h rstd w does not. Bars as in
test_gpu_add_rms_norm: powers of two on h and on the weights change no rounding of y."""
import numpy as np
import pytest

import oracle
from tests.gpu_util import note
from tests.test_gpu_add_rms_norm import check, make, run, values
from workloads import bf16_bits_from_f32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [8, 128, 384, 1280, 5120, 9216, 40000])
@pytest.mark.parametrize("of_h,of_w", [(60, 70), (50, 100), (0, 120), (-50, -90), (-45, -100), (30, -100), (0, -110)])
def test_scales_of_extreme_weights(H, of_h, of_w):
    """Rows of h about 2^of_h beside ordinary ones, weights about 2^of_w; eps = 0, so that small rows count."""
    T = 6
    x, r, w = make(T, H, abs(H + of_h), spread=0.0)
    w = (w * 2.0 ** of_w).astype(np.float32)
    for t in (1, 2, 5):
        x[t] = bf16_bits_from_f32((values(x[t]) * 2.0 ** of_h).astype(np.float32))
        r[t] = bf16_bits_from_f32((values(r[t]) * 2.0 ** of_h).astype(np.float32))
    for mode in (0, 1):
        if mode and H % 128:
            continue
        note(f"norm H={H} h 2^{of_h} w 2^{of_w} mode={mode}")
        check(x, r, w, 0.0, H, mode, run(x, r, w, 0.0, H, mode))


@pytest.mark.parametrize("H", [128, 512, 5120, 40000])
def test_rows_of_zeros_and_of_ordinary_values_among_extreme_ones(H):
    """Each row by itself: the extreme ones take the second look at y, the others do not, and a row of zeros has scale 1."""
    T = 70
    x, r, w = make(T, H, 1, spread=0.0)
    for t in range(T):
        f = (0.0, 1.0, 2.0 ** 62, 2.0 ** -50)[t % 4]
        x[t] = bf16_bits_from_f32((values(x[t]) * f).astype(np.float32))
        r[t] = bf16_bits_from_f32((values(r[t]) * f).astype(np.float32))
    for scale in (2.0 ** 66, 2.0 ** -80):
        s = (w * scale).astype(np.float32)
        note(f"norm, rows of many sizes, H={H} weights {scale}")
        got = run(x, r, s, 1e-30, H, 0)
        check(x, r, s, 1e-30, H, 0, got)
        assert np.all(got[3][0::4] == 1.0) and not oracle.e4m3_decode(got[2][0::4]).any()


@pytest.mark.parametrize("H", [8, 128, 512, 1280, 5120, 9216, 40000])
@pytest.mark.parametrize("of_h", [63, 64, 100, 124, -58, -64, -80, -110])
def test_sizes_of_h(H, of_h):
    """Rows of h about 2^of_h, to the ends of bf16's normal range, among ordinary ones, with every kind of result."""
    T = 6
    x, r, w = make(T, H, abs(H + of_h), spread=0.0)
    for t in (0, 3, 4):
        x[t] = bf16_bits_from_f32((values(x[t]) * 2.0 ** of_h).astype(np.float32))
        r[t] = bf16_bits_from_f32((values(r[t]) * 2.0 ** of_h).astype(np.float32))
    for eps in (0.0, 1e-30, 1e-5):
        for mode, q in ((0, False), (0, True), (1, True)):
            if mode and H % 128:
                continue
            note(f"norm H={H} h 2^{of_h} eps={eps} mode={mode} codes={q}")
            check(x, r, w, eps, H, mode, run(x, r, w, eps, H, mode, q=q))


@pytest.mark.parametrize("H", [128, 5120, 40000])
def test_nan_and_infinity_in_far_rows(H):
    """They stay in their row, where y is NaN (a NaN), or NaN at the infinity and 0 elsewhere."""
    T = 8
    x, r, w = make(T, H, 5, spread=0.0)
    for t in range(T):
        x[t] = bf16_bits_from_f32((values(x[t]) * 2.0 ** (100 if t % 2 else -100)).astype(np.float32))
    r[:] = 0
    clean = run(x, r, w, 0.0, H, 0)
    check(x, r, w, 0.0, H, 0, clean)
    bad = x.copy()
    bad[1, 5], bad[2, H - 1], bad[5, H - 1], bad[6, 0] = 0x7FC1, 0x7FC1, 0x7F80, 0xFF80
    got = run(bad, r, w, 0.0, H, 0)
    others = [0, 3, 4, 7]
    for a, b in zip(clean, got):
        assert np.array_equal(a[others], b[others])
    y = values(got[1].view(np.uint16))
    assert np.all(np.isnan(y[[1, 2]])) and np.isnan(y[5, H - 1]) and np.isnan(y[6, 0])
    assert not np.any(y[5, :H - 1]) and not np.any(y[6, 1:])
    assert np.all(got[3][[1, 2, 5, 6]] == 1.0)


@pytest.mark.parametrize("H", [8, 128, 384, 5120, 40000])
def test_the_smallest_values(H):
    """Subnormal bf16 values, eps = 0: multiples of 2^-133 up to 60 of them, whose sums are exact in bf16."""
    rng = np.random.default_rng(H)
    small = lambda: bf16_bits_from_f32((rng.integers(-60, 61, (5, H)) * 2.0 ** -133).astype(np.float32))
    x, r = small(), small()
    x[:, 0], r[:, 0] = bf16_bits_from_f32(np.float32([2.0 ** -133]))[0], 0   # (no row of zeros)
    w = rng.uniform(-1.5, 1.5, H).astype(np.float32)
    for mode, q in ((0, False), (0, True), (1, True)):
        if mode and H % 128:
            continue
        note(f"norm of subnormal values H={H} mode={mode} codes={q}")
        got = run(x, r, w, 0.0, H, mode, q=q)
        check(x, r, w, 0.0, H, mode, got)
        assert np.array_equal(values(got[0].view(np.uint16)), values(x) + values(r))
