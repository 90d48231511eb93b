"""Attention with a window, usage and eviction over pages whose byte offsets pass 2^32 (element offsets 2^31): the last pages of a
large pool, strided."""
import numpy as np
import pytest
import torch

import oracle
from shared_routed_expert_amd import _lib as L
from tests.gpu_util import note, DEV
from tests.kv_util import make_case
from tests.test_gpu_attention import Dev, bits_of, up, check as check_attention
from tests.test_gpu_kv_usage import UseDev, some_lse, check as check_usage

pytestmark = pytest.mark.gpu

HKV, D, PAGE = 8, 128, 64
STRIDE = 4 * HKV * PAGE * D        # elements: half of every page's stretch belongs to nothing
PAGES = (1 << 32) // STRIDE + 20
HALF = HKV * PAGE * D


def far_pool(c):
    """A pool of NaN whose last pages hold the case's, every third; c.table is moved to them."""
    pool = torch.empty(PAGES * STRIDE * (1 if c.fp8 else 2), dtype=torch.uint8, device=DEV)
    pool.view(torch.int32).fill_(0x7F7F7F7F if c.fp8 else 0x7FC07FC0)
    far = np.array([PAGES - 1 - 3 * i for i in range(c.kv.shape[0])], np.int32)
    view = pool.view(torch.uint8 if c.fp8 else torch.int16).view(PAGES, STRIDE)
    for i, p in enumerate(far):
        view[int(p), :2 * HALF] = up(c.kv[i] if c.fp8 else c.kv[i].view(np.int16)).reshape(-1)
    for s, k in enumerate(c.kvs):
        n = -(-k // PAGE)
        c.table[s, :n] = far[c.table[s, :n]]
    return pool, view


def kv_type(c):
    return L.KV_E4M3 if c.fp8 else L.KV_BF16


@pytest.mark.parametrize("fp8", [False, True])
def test_window(fp8):
    c = make_case([1, 40], [500, 70], 16, HKV, D, PAGE, fp8, seed=5)
    pool, _ = far_pool(c)
    d = Dev(c)
    d.out.fill_(0x7FC1)
    d.lse.fill_(7.0)
    note(f"window, far pages fp8={fp8}")
    L.moe_window_attention(d.q, c.q.shape[1], pool.data_ptr(), pool.data_ptr() + HALF * (1 if fp8 else 2), kv_type(c),
                           d.ks if fp8 else None, d.vs if fp8 else None, PAGES, PAGE, STRIDE, up(c.table), c.table.shape[1],
                           d.cu, d.kvl, 100, 5, 2, c.T, 40, c.Hq, HKV, D, D ** -0.5, 0.0, d.out, d.lse, d.ws, d.ws_bytes)
    torch.cuda.synchronize()
    sees = [oracle.visible_window(n, k, 100, 5) for n, k in zip(c.ns, c.kvs)]
    check_attention(c, bits_of(d.out), d.lse.cpu().numpy(), sees, D ** -0.5, 0.0)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 40])
def test_usage(n, fp8):
    c = make_case([1, n], [500, 70], 16, HKV, D, PAGE, fp8, seed=6)
    sees = [oracle.visible_prefill(m, k, 0) for m, k in zip(c.ns, c.kvs)]
    lse = some_lse(c, sees)
    pool, _ = far_pool(c)
    d = UseDev(c, lse)
    note(f"usage, far pages fp8={fp8} n={n}")
    L.moe_kv_usage(d.q, c.q.shape[1], pool.data_ptr(), kv_type(c), d.ks if fp8 else None, PAGES, PAGE, STRIDE, up(c.table),
                   c.table.shape[1], d.cu, d.kvl, None, d.lse, 2, c.T, d.max_q, c.Hq, HKV, D, D ** -0.5, 0.0, None, 1.0,
                   d.usage, None, 2, d.ws, d.ws_bytes)
    torch.cuda.synchronize()
    check_usage(c, d.usage.cpu().numpy(), lse, sees, D ** -0.5, 0.0)


@pytest.mark.parametrize("fp8", [False, True])
def test_evict(fp8):
    """From the last pages to others of the last, and to one of the first."""
    c = make_case([1, 1], [500, 70], 16, HKV, D, PAGE, fp8, seed=7)
    pool, view = far_pool(c)
    used = set(c.table[0, :8].tolist())
    new = np.array([[p for p in range(PAGES - 1, 0, -1) if p not in used][:2], [3, 4]], np.int32)
    budget = 100
    new[0, 1] = 2
    rng = np.random.default_rng(1)
    usage = rng.standard_normal((2, HKV, c.table.shape[1] * PAGE)).astype(np.float32)
    out, lens = torch.zeros(usage.shape, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    kept = torch.full((2, HKV, budget), -1, dtype=torch.int32, device=DEV)
    note(f"evict, far pages fp8={fp8}")
    L.moe_kv_evict(pool.data_ptr(), pool.data_ptr() + HALF * (1 if fp8 else 2), kv_type(c), PAGES, PAGE, STRIDE, up(c.table),
                   c.table.shape[1], up(np.array(c.kvs, np.int32)), up(usage), out, None, 2, 2, HKV, D, budget, budget, 4, 20,
                   up(new), 2, lens, kept)
    torch.cuda.synchronize()
    assert lens.tolist() == [budget, 70]
    rows = view[:, :2 * HALF].view(PAGES, 2, HKV, PAGE, D)
    got = torch.cat([rows[int(p)] for p in new[0]], 2)[:, :, :budget].cpu().numpy()
    old = torch.cat([rows[int(p)] for p in c.table[0, :8]], 2).cpu().numpy()
    for h in range(HKV):
        k = oracle.kept_tokens(usage[0, h], 500, budget, 4, 20)
        assert kept[0, h].tolist() == list(k)
        assert np.array_equal(got[:, h], old[:, h, k])
