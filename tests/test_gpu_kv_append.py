"""moe_kv_append against the float64 oracle on the same bf16 inputs.

Bars, with m the length of the rotated pair a value belongs to (|ref| for unrotated dims):
  q, k in bf16: |gpu - ref| <= 2^-8 |ref| + 2^-15 m   (one bf16 rounding of a float32 result; float32 error of the
                sum of squares, rsqrt and rotation < 2^-15 m, as in the in-place call)
  k in e4m3:    with r = ref / scale held to +-448: |code - r| <= 2^-4 |r| + 2^-10 + 2^-15 m / scale  (half a step is
                2^-4 of a normal value and 2^-10 on the subnormal grid of 2^-9)
  v:            exactly the input's bits (bf16), or exactly the e4m3 code of the float32 quotient
Every other byte of the cache, of qkv and around q_out is unchanged.
"""
import numpy as np
import pytest
import torch

import oracle
from shared_routed_expert_amd import _lib as L
from tests.gpu_util import note, DEV
from tests.test_gpu_qknorm import pair_len, table
from workloads import QKConfig, generate_qk, f32_from_bf16_bits

pytestmark = pytest.mark.gpu

SHAPES = [
    # (T, Hq, Hkv, D, rd, neox, page, fp8, norm)
    (1, 12, 1, 128, 64, True, 16, False, True),
    (1, 12, 1, 128, 64, True, 16, True, True),
    (64, 12, 1, 128, 64, True, 16, False, True),
    (77, 2, 1, 64, 16, True, 32, True, True),
    (77, 2, 1, 64, 64, False, 32, False, True),
    (33, 3, 2, 256, 128, True, 64, True, True),
    (33, 3, 2, 256, 256, True, 16, False, True),
    (1000, 12, 1, 128, 64, False, 16, True, True),
    (65, 96, 8, 128, 64, True, 128, False, True),
    (65, 96, 8, 128, 64, True, 128, True, True),
    (9, 0, 3, 128, 128, False, 16, True, True),      # keys and values only
    (50, 12, 1, 128, 64, True, 16, False, False),    # rotation, no norm
    (50, 12, 1, 128, 0, True, 16, True, True),       # norm, no rotation
    (50, 4, 2, 64, 0, True, 1024, False, False),     # a plain cache write
    (3, 500, 262, 64, 32, True, 16, False, True),    # 1024 heads per token
    (4099, 12, 1, 128, 64, True, 16, True, True),
]


def inputs(T, Hq, Hkv, D, rd, neox):
    return generate_qk(QKConfig(f"append_{T}_{Hq}_{Hkv}_{D}_{rd}", T=T, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D,
                                rotary_dim=rd or 16, neox=neox, max_pos=4096, theta=10000.0, eps=1e-6,
                                seed=T * 7 + D + rd))


def run(inp, page, fp8, norm, rd, slots, pages, extra=0, fill=None):
    """Returns qkv, q_out with its guards, and the cache, as numpy; the cache starts as `fill`."""
    cfg = inp.cfg
    T, row = inp.qkv_bf16.shape
    Hq, Hkv, D = cfg.num_q_heads, cfg.num_kv_heads, cfg.head_dim
    qkv = np.full((T, row + extra), 0x7FC1, np.uint16)
    qkv[:, :row] = inp.qkv_bf16
    dq = torch.from_numpy(qkv.view(np.int16)).to(DEV)
    kv = torch.from_numpy(fill).to(DEV)
    out = torch.full((T * Hq * D + 4096,), 0x7FC1, dtype=torch.int16, device=DEV)
    scale = torch.from_numpy(np.random.default_rng(5).uniform(0.004, 0.03, (2, Hkv)).astype(np.float32)).to(DEV)
    ks, vs = scale[0].clone(), scale[1].clone()
    cs = table(cfg.max_pos, rd, cfg.theta) if rd else None
    qw, kw = (torch.from_numpy(w).to(DEV) if norm else None for w in (inp.q_norm_w, inp.k_norm_w))
    note(f"kv_append T={T} Hq={Hq} Hkv={Hkv} D={D} rd={rd} neox={cfg.neox} page={page} fp8={fp8} norm={norm}")
    L.moe_kv_append(dq, row + extra, T, Hq, Hkv, D, rd, cfg.neox, qw, kw, cfg.eps,
                    torch.from_numpy(inp.positions).to(DEV) if rd else None, cs, cfg.max_pos if rd else 0,
                    torch.from_numpy(slots).to(DEV), out[2048:].data_ptr() if Hq else None, kv[:, 0].data_ptr(),
                    kv[:, 1].data_ptr(), L.KV_E4M3 if fp8 else L.KV_BF16, ks if fp8 else None, vs if fp8 else None, pages,
                    page, kv.stride(0))
    torch.cuda.synchronize()
    out = out.cpu().numpy().view(np.uint16)
    assert np.all(out[:2048] == 0x7FC1) and np.all(out[2048 + T * Hq * D:] == 0x7FC1)
    assert np.array_equal(dq.cpu().numpy().view(np.uint16), qkv)
    return out[2048:2048 + T * Hq * D].reshape(T, Hq, D), kv.cpu().numpy(), scale.cpu().numpy()


@pytest.mark.parametrize("T,Hq,Hkv,D,rd,neox,page,fp8,norm", SHAPES)
def test_shapes(T, Hq, Hkv, D, rd, neox, page, fp8, norm):
    inp = inputs(T, Hq, Hkv, D, rd, neox)
    cfg = inp.cfg
    rng = np.random.default_rng(T + D)
    pages = -(-T // page) + 3
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    out_of = [-1, pages * page, -(1 << 31), (1 << 31) - 1]
    for i, s in enumerate(out_of):     # tokens that are not cached
        if T > 20:
            slots[5 + 3 * i] = s
    fill = rng.integers(0, 256 if fp8 else 32768, (pages, 2, Hkv, page, D)).astype(np.uint8 if fp8 else np.int16)
    q, kv, scale = run(inp, page, fp8, norm, rd, slots, pages, extra=8 * (T % 3), fill=fill)
    x = f32_from_bf16_bits(inp.qkv_bf16).astype(np.float64).reshape(T, Hq + 2 * Hkv, D)
    qk = x[:, :Hq + Hkv].copy()
    if norm:
        qk[:, :Hq] = oracle.head_rms_norm(qk[:, :Hq], inp.q_norm_w, cfg.eps)
        qk[:, Hq:] = oracle.head_rms_norm(qk[:, Hq:], inp.k_norm_w, cfg.eps)
    if rd:
        ang = oracle.rope_angles(inp.positions, rd, cfg.theta)
        qk = (oracle.rope_half if neox else oracle.rope_interleaved)(qk, ang, rd)
        m = pair_len(qk.reshape(T, -1), cfg.replace(rotary_dim=rd)).reshape(qk.shape)
    else:
        m = np.abs(qk)
    err = np.abs(f32_from_bf16_bits(q.copy()).astype(np.float64) - qk[:, :Hq])
    assert np.all(err <= 2.0 ** -8 * np.abs(qk[:, :Hq]) + 2.0 ** -15 * m[:, :Hq])
    keep = (slots >= 0) & (slots < pages * page)
    pg, at = slots[keep] // page, slots[keep] % page
    k, v = kv[pg, 0, :, at], kv[pg, 1, :, at]          # [kept, Hkv, D]
    kr, mk = qk[keep, Hq:], m[keep, Hq:]
    vbits = inp.qkv_bf16.reshape(T, -1, D)[keep, Hq + Hkv:]
    if fp8:
        s = scale[0].astype(np.float64)[None, :, None]
        r = np.clip(kr / s, -448, 448)
        assert np.all(np.abs(oracle.e4m3_decode(k) - r) <= 2.0 ** -4 * np.abs(r) + 2.0 ** -10 + 2.0 ** -15 * mk / s)
        quot = f32_from_bf16_bits(vbits.copy()).astype(np.float32) / scale[1][None, :, None]
        assert np.array_equal(v, oracle.e4m3_encode(np.clip(quot, -448, 448)))
    else:
        got = f32_from_bf16_bits(k.view(np.uint16).copy()).astype(np.float64)
        assert np.all(np.abs(got - kr) <= 2.0 ** -8 * np.abs(kr) + 2.0 ** -15 * mk)
        assert np.array_equal(v.view(np.uint16), vbits)
    want = fill.copy()
    want[pg, :, :, at] = kv[pg, :, :, at]
    assert np.array_equal(kv, want)


def test_saturation_nan_and_zero():
    """e4m3: values past 448 scales saturate, NaN stays NaN (code 0x7F or 0xFF), a zero k head stays zero."""
    inp = inputs(4, 2, 1, 64, 0, True)
    bits = inp.qkv_bf16.reshape(4, 4, 64)
    bits[0, 3] = 0x7F00                  # v: 1.7e38
    bits[1, 3] = 0xFF00                  # -1.7e38
    bits[2, 3, 7] = 0x7FC0               # NaN
    bits[2, 3, 8] = 0xFF80               # -inf
    bits[3, 2] = 0                       # k
    fill = np.full((1, 2, 1, 16, 64), 9, np.uint8)
    _, kv, _ = run(inp, 16, True, True, 0, np.arange(4, dtype=np.int32), 1, fill=fill)
    v = kv[0, 1, 0]
    assert np.all(v[0] == 0x7E) and np.all(v[1] == 0xFE)
    assert v[2, 7] & 0x7F == 0x7F and v[2, 8] == 0xFE
    assert np.all(kv[0, 0, 0, 3] & 0x7F == 0)


def test_far_pages():
    """A cache of more than 2^32 bytes (and 2^31 elements): the offsets of its last pages are 64-bit."""
    T, D, page, Hkv = 5, 128, 16, 8
    stride = 2 * Hkv * page * D
    pages = (1 << 31) // stride + 40
    kv = torch.zeros((pages, 2, Hkv, page, D), dtype=torch.bfloat16, device=DEV)
    x = torch.randn((T, 3 * Hkv * D), dtype=torch.bfloat16, device=DEV)
    slots = torch.tensor([0, pages * page - 1, (pages - 3) * page, 17, (pages - 2) * page + 5], dtype=torch.int32, device=DEV)
    q = torch.empty((T, Hkv, D), dtype=torch.bfloat16, device=DEV)
    L.moe_kv_append(x, x.stride(0), T, Hkv, Hkv, D, 0, True, None, None, 0.0, None, None, 0, slots, q, kv[:, 0], kv[:, 1],
                    L.KV_BF16, None, None, pages, page, kv.stride(0))
    torch.cuda.synchronize()
    h = x.view(T, 3, Hkv, D)
    assert torch.equal(q, h[:, 0])
    for t in range(T):
        s = int(slots[t])
        assert torch.equal(kv[s // page, :, :, s % page], h[t, 1:])
    assert int((kv[:, 0, 0, :, 0] != 0).sum()) <= T
