"""Scores at the ends of their range: caps and scales from the smallest to the largest that the calls accept, on every
kernel variant that caps, against the float64 oracle.

Bars, with A, X, u as in test_gpu_attention (A = sum_j w_j |v_j|, X the row's largest sum_d |q_d k_d| * scale, u the
weights' rounding) and s = scale q.k:
  e   error of a score: s itself 2^-24 (D + 12) X (D products and their sum, the factor's roundings), which tanh passes on
      at most once and never as more than 2 cap; and the cap, 2^-24 (32 |z| + (4 cap for caps up to 64)), where
      |z| <= min(X, cap). With t = tanh(y) = 1 - r, r = 2 / (e + 1), e = exp(2 y): r is off by 2^-24 r (2 e / (e + 1) + 1 + 2) (exponential, sum,
      reciprocal), at most 6, which is under 20 t for |y| >= 1/4 and under 20 t + 4 for all y; the factors add 6 t. Caps
      above 64 may not have the 4 (a polynomial near 0, 14 t), so the bar does not grow with them.
  out: 2^-8 |ref| + (u + 2 e + 2^-24 (2 kv + 64)) A       lse: e + 2^-24 (kv + 64 + 4 |lse|)
"""
import numpy as np
import pytest
import torch

import oracle
from tests.gpu_util import note
from tests.kv_util import make_case, random_tree
from tests.test_gpu_attention import Dev, bits_of, up
from workloads import f32_from_bf16_bits

pytestmark = pytest.mark.gpu

CAPS = [1e-6, 0.5, 30.0, 64.0, 65.0, 1e3, 1e6]


def check_rows(c, out_bits, lse, sees, scale, cap):
    u = 2.0 ** -11 if c.fp8 else 2.0 ** -8
    for s, n in enumerate(c.ns):
        a = int(c.cu_q[s])
        ref, rl, mag, dot = oracle.attend(c.q_heads(s), c.k[s], c.v[s], sees[s], scale, cap)
        e = 2.0 ** -24 * (c.D + 12) * dot
        if cap > 0:
            e = np.minimum(e, 2 * cap) + 2.0 ** -24 * (32 * np.minimum(dot, cap) + (4 * cap if cap <= 64 else 0))
        got = f32_from_bf16_bits(out_bits[a:a + n].copy()).astype(np.float64)
        bound = 2.0 ** -8 * np.abs(ref) + (u + 2 * e[..., None] + 2.0 ** -24 * (2 * c.kvs[s] + 64)) * mag + 1e-37
        err = np.abs(got - ref)
        assert np.all(err <= bound), (s, np.argwhere(~(err <= bound))[:3], np.max(err / bound))
        seen = sees[s].any(axis=1)
        g = lse[a:a + n].astype(np.float64)
        assert np.all(g[~seen] == -np.inf) and not out_bits[a:a + n][~seen].any()
        off = np.abs(g[seen] - rl[seen])
        bar = (e + 2.0 ** -24 * (c.kvs[s] + 64 + 4 * np.abs(np.where(seen[:, None], rl, 0))))[seen]
        assert np.all(off <= bar), (s, np.max(off / bar, initial=0))


def run_scores(c, which, extra, sees, scale, cap, tag):
    for wide in (False, True):     # what the block table may hold decides how the keys are split
        if wide:
            t = np.full((c.table.shape[0], 131072 // c.page), 1 << 30, np.int32)
            t[:, :c.table.shape[1]] = c.table
            c.table = t
        d = Dev(c)
        note(f"{tag} {which} Hq={c.Hq} Hkv={c.Hkv} D={c.D} fp8={c.fp8} scale={scale:g} cap={cap:g} wide={wide}")
        d.call(which, None if extra is None else up(extra), scale, cap)
        torch.cuda.synchronize()
        check_rows(c, bits_of(d.out), d.lse.cpu().numpy(), sees, float(np.float32(scale)), float(np.float32(cap)))


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D", [(12, 1, 128), (8, 2, 64), (8, 1, 256), (40, 1, 128), (40, 1, 64)])
def test_capped_single_tokens(Hq, Hkv, D, fp8, cap):
    kvs = [1, 1, 2, 16, 17, 33, 64, 65, 129, 257, 1000]
    c = make_case([1] * len(kvs), kvs, Hq, Hkv, D, 16, fp8, seed=Hq + D)
    run_scores(c, "tree", None, [oracle.visible_tree(1, k, None) for k in kvs], D ** -0.5, cap, "caps")


@pytest.mark.parametrize("cap", [30.0, 1e5])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D", [(12, 1, 128), (8, 2, 64), (8, 1, 256)])
def test_capped_prefill(Hq, Hkv, D, fp8, cap):
    ns, kvs, pre = [130, 65, 1], [400, 65, 1], [170, 0, 0]
    c = make_case(ns, kvs, Hq, Hkv, D, 32, fp8, seed=D)
    run_scores(c, "prefill", np.array(pre, np.int32), [oracle.visible_prefill(n, k, p) for n, k, p in zip(ns, kvs, pre)],
               D ** -0.5, cap, "caps")


@pytest.mark.parametrize("cap", [30.0, 1e4])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [2, 20])
@pytest.mark.parametrize("Hq,Hkv,D", [(12, 1, 128), (8, 2, 64), (8, 1, 256)])
def test_capped_trees(Hq, Hkv, D, n, fp8, cap):
    """Masked scores and capped ones together, rows that see nothing among them; on both arrangements of the waves."""
    rng = np.random.default_rng(n)
    kvs = [n, 700, 40 + n]
    c = make_case([n] * 3, kvs, Hq, Hkv, D, 16, fp8, seed=n + D)
    words = [random_tree(n, rng) for _ in kvs]
    words[0][0] = 0
    run_scores(c, "tree", np.concatenate(words).view(np.int64), [oracle.visible_tree(n, k, w) for k, w in zip(kvs, words)],
               D ** -0.5, cap, "caps")


@pytest.mark.parametrize("cap", [0.0, 1.0])
@pytest.mark.parametrize("scale,k_factor", [(1e-45, 1.0), (1e-44, 1.0), (1e-38, 1.0), (1e-15, 2.0 ** -100), (1e-20, 1.0)])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 70])
def test_tiny_scales(n, fp8, scale, k_factor, cap):
    """Scores so small that their factor (scale times the keys' own) is zero in float32: every seen token has the same
    weight, and the masked ones still none."""
    kvs = [n, 77 + n, 200]
    c = make_case([n] * 3, kvs, 12, 1, 128, 16, fp8, seed=n)
    if fp8:
        c.scales[0] *= np.float32(k_factor)
        c.k = [k * k_factor for k in c.k]
    run_scores(c, "prefill", None, [oracle.visible_prefill(n, k, 0) for k in kvs], scale, cap, "tiny scales")
