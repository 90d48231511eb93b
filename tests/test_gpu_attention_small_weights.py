"""Softmax weights far below the row's largest one. Over an e4m3 cache they multiply v as float16, which holds a weight
within 2^-11 of it or 2^-32 of the row's largest weight, whichever is more: a score that exceeds the running maximum by
2^8 at most moves nothing, the largest weight is between 2^7 and 2^15, and float16's subnormals are 2^-24 apart."""
import numpy as np
import pytest
import torch

from oracle import e4m3_encode
from shared_routed_expert_amd import _lib as L
from tests.gpu_util import note, DEV
from workloads import bf16_bits_from_f32, f32_from_bf16_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("order", ["largest first", "largest last"])
@pytest.mark.parametrize("steps", [10, 16, 20, 22, 24, 26, 28, 30, 32, 36])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq", [12, 40])
def test_small_weights(Hq, fp8, steps, order):
    """kv - 1 keys of weight 2^-steps each whose values are large, one of weight 1 whose value is 0."""
    D, kv, page = 128, 4001, 16
    pages = -(-kv // page)
    k, v = np.zeros((pages * page, D), np.float32), np.zeros((pages * page, D), np.float32)
    top = 0 if order == "largest first" else kv - 1
    k[:kv, 0] = -steps                       # exact in both types
    v[:kv] = np.where(np.arange(D) % 2, 448.0, -3.5)
    k[top], v[top] = 0, 0
    put = e4m3_encode if fp8 else bf16_bits_from_f32
    pool = np.stack([put(x).reshape(pages, 1, page, D) for x in (k, v)], 1)
    pool = torch.from_numpy(np.ascontiguousarray(pool if fp8 else pool.view(np.int16))).to(DEV)
    q = np.zeros((Hq, D), np.float32)
    q[:, 0] = 1
    q = torch.from_numpy(bf16_bits_from_f32(q).view(np.int16)).to(DEV)
    one = torch.ones(1, device=DEV)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    table, cu, lens = torch.arange(pages, dtype=torch.int32, device=DEV), i32(0, 1), i32(kv)
    out = torch.empty((Hq, D), dtype=torch.int16, device=DEV)
    lse = torch.empty(Hq, device=DEV)
    n = L.moe_attention_workspace_bytes(1, 1, 1, Hq, 1, D)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    scale = float(np.float32(np.log(2.0)))
    note(f"small weights Hq={Hq} fp8={fp8} 2^-{steps} {order}")
    L.moe_tree_attention(q, Hq * D, pool[:, 0], pool[:, 1], L.KV_E4M3 if fp8 else L.KV_BF16, one if fp8 else None,
                         one if fp8 else None, pages, page, pool.stride(0), table, pages, cu, lens, None, 1, 1, 1, Hq, 1, D,
                         scale, 0.0, out, lse, ws, n)
    torch.cuda.synchronize()
    w = np.exp(-scale * steps)
    total = 1 + (kv - 1) * w
    A = (kv - 1) * w * np.abs(v[1]).astype(np.float64) / total          # sum of weight times |value|
    ref = np.where(v[1] > 0, A, -A)
    lost = (kv - 1) * 2.0 ** -32 * np.abs(v[1]) / total if fp8 else 0
    # 2^-8 out; the weights' rounding; a score's error (steps times the factor's few 2^-24), the exponential's, kv sums
    bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** (-11 if fp8 else -8) + 2.0 ** -24 * (8 * steps + 2 * kv + 64)) * A + lost
    got = f32_from_bf16_bits(out.cpu().numpy().view(np.uint16)).astype(np.float64)
    assert np.all(np.abs(got - ref) <= bound), (np.max(np.abs(got - ref) / bound), got[0, :2], ref[:2])
    assert np.all(np.abs(lse.cpu().numpy() - np.log(total)) <= 2.0 ** -24 * (kv + 64))
