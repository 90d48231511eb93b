"""q, out and lse side by side in one allocation, and out between q's strided rows: no overlap, the result of buffers apart."""
import numpy as np
import pytest
import torch

from shared_routed_expert_amd import PagedKVCache
from tests.gpu_util import DEV, note
from tests.kv_util import make_case
from tests.test_gpu_attention import up

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("call", ["tree", "prefill", "window"])
def test_neighbours(call):
    Hq, D, n = 12, 128, 20
    c = make_case([n, 1], [300, 5000], Hq, 1, D, 16, False, seed=3)
    cache = PagedKVCache(c.kv.shape[0], 16, 1, D, device=DEV)
    cache.kv.view(torch.int16).copy_(up(c.kv.view(np.int16)))
    q = up(c.q.view(np.int16)).view(torch.bfloat16).unflatten(1, (Hq, D))
    args = (up(c.table), up(c.cu_q), up(np.array(c.kvs, np.int32)), n) + ((200, 4) if call == "window" else ())
    run = getattr(cache, call + "_attention")
    note(f"{call} attention, neighbouring buffers")
    lse = torch.empty((c.T, Hq), device=DEV)
    want = run(q, *args, lse=lse)
    size = q.numel()
    buf = torch.zeros(3 * size + 4 * c.T * Hq, dtype=torch.bfloat16, device=DEV)
    q2, out = buf[:size].view_as(q), buf[size:2 * size].view_as(q)
    lse2 = buf[2 * size:2 * size + 2 * c.T * Hq].view(torch.float32).view(c.T, Hq)
    q2.copy_(q)
    run(q2, *args, out=out, lse=lse2)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse2, lse) and torch.equal(q2, q)
    wide = torch.zeros((c.T, 2 * size + Hq * D), dtype=torch.bfloat16, device=DEV)
    q3 = wide[:, :Hq * D].unflatten(1, (Hq, D))
    q3.copy_(q)
    out = wide[7, Hq * D:Hq * D + size].view_as(q)
    run(q3, *args, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(q3, q)
    with pytest.raises(Exception, match="moe_" + call):
        run(q2, *args, out=q2)
