"""Host-side checks of moe_kv_usage and moe_kv_evict (no GPU needed): every refusal comes before a launch, with fake 16-byte
aligned pointers that are never dereferenced; PagedKVCache's own checks on CPU tensors; the oracle on small cases."""
import numpy as np
import pytest
import torch

import oracle

FAKE, FAKE2, MIS = 0x10000, 0x20000, 0x10004


@pytest.fixture(scope="module")
def L():
    from shared_routed_expert_amd import _lib
    return _lib


def usage(L, **kw):
    a = dict(q=FAKE, q_stride=12 * 128, k_cache=FAKE, kv_type=0, k_scale=None, num_pages=8, page_size=16, page_stride=4096,
             block_table=FAKE, max_pages=4, cu_q=FAKE, kv_lens=FAKE, prefix_lens=None, lse=FAKE, S=2, T=4, max_q=2,
             num_q_heads=12, num_kv_heads=1, head_dim=128, scale=0.1, softcap=0.0, prev=None, decay=1.0, usage=FAKE,
             usage_rows=None, rows=2, workspace=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return L.moe_kv_usage(**a, stream=0, check=False)


def evict(L, **kw):
    a = dict(k_cache=FAKE, v_cache=FAKE, kv_type=0, num_pages=8, page_size=16, page_stride=4096, block_table=FAKE, max_pages=4,
             kv_lens=FAKE, usage=FAKE, new_usage=FAKE, usage_rows=None, rows=2, S=2, num_kv_heads=1, head_dim=128, limit=40,
             budget=32, sinks=4, recent=8, new_table=FAKE2, new_max_pages=2, new_lens=FAKE2, kept=FAKE)
    a.update(kw)
    return L.moe_kv_evict(**a, stream=0, check=False)


def test_usage_rejects(L):
    nan = float("nan")
    for kw in (dict(S=-1), dict(T=-1), dict(T=(1 << 20) + 1), dict(max_q=0), dict(num_q_heads=0), dict(num_kv_heads=0),
               dict(num_kv_heads=5), dict(q_stride=12 * 128 - 8), dict(q_stride=12 * 128 + 4), dict(kv_type=3), dict(num_pages=0),
               dict(page_stride=2032 - 16), dict(max_pages=0), dict(scale=0.0), dict(scale=nan), dict(softcap=-1.0),
               dict(decay=-0.1), dict(decay=1.1), dict(decay=nan), dict(rows=1), dict(rows=0, usage_rows=FAKE), dict(kv_type=1)):
        assert usage(L, **kw) == -1, kw
    for kw in (dict(head_dim=80), dict(page_size=8), dict(page_size=24), dict(S=65537, rows=65537), dict(num_pages=1 << 27),
               dict(num_q_heads=129, q_stride=1 << 20), dict(max_pages=1 << 26)):
        assert usage(L, **kw) == -2, kw
    for name in ("q", "k_cache", "block_table", "cu_q", "kv_lens", "lse", "usage", "workspace"):
        assert usage(L, **{name: None}) == -1, name
        assert usage(L, **{name: MIS}) == -1, name
    for name in ("prev", "usage_rows", "prefix_lens"):
        assert usage(L, **{name: MIS}) == -1, name
    assert usage(L, kv_type=1, k_scale=MIS) == -1
    assert usage(L, ws_bytes=0) == -3
    assert usage(L, T=0, q=None) == 0 and usage(L, S=0, q=None) == 0
    assert usage(L, rows=1, usage_rows=FAKE, ws_bytes=0) == -3      # any number of rows with usage_rows
    assert L.moe_kv_usage_workspace_bytes(2, 4, 2, 12, 1, 128) > 0
    assert L.moe_kv_usage_workspace_bytes(2, 4, 2, 12, 5, 128) == 0


def test_evict_rejects(L):
    for kw in (dict(S=-1), dict(num_kv_heads=0), dict(kv_type=2), dict(num_pages=0), dict(page_stride=1024), dict(max_pages=0),
               dict(new_max_pages=0), dict(budget=0), dict(limit=31), dict(sinks=-1), dict(recent=-1), dict(sinks=33, recent=0),
               dict(sinks=4, recent=29), dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), dict(new_max_pages=1), dict(rows=1),
               dict(rows=0, usage_rows=FAKE), dict(new_lens=FAKE), dict(new_table=FAKE)):
        assert evict(L, **kw) == -1, kw
    for kw in (dict(head_dim=80), dict(page_size=8), dict(S=65536, rows=65536), dict(S=8192, rows=8192, num_kv_heads=8, page_stride=1 << 20),
               dict(max_pages=1 << 26), dict(new_max_pages=1 << 26)):
        assert evict(L, **kw) == -2, kw
    for name in ("k_cache", "v_cache", "block_table", "kv_lens", "usage", "new_usage", "new_table", "new_lens", "kept"):
        assert evict(L, **{name: None}) == -1, name
        # (new_table: a slice of a list, at any of its elements)
        assert evict(L, **{name: MIS if name != "new_table" else 0x10002}) == -1, name
    assert evict(L, usage_rows=MIS) == -1
    assert evict(L, S=0, k_cache=None) == 0


def test_cache_object_rejects(L):
    from shared_routed_expert_amd import PagedKVCache
    c = PagedKVCache(4, 16, 2, 128, device="cpu")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)
    z = torch.zeros
    good = dict(q=z((2, 12, 128), dtype=torch.bfloat16), block_table=z((1, 3), dtype=torch.int32), cu_q=i32(0, 2), kv_lens=i32(2),
                max_q=2, lse=z(2, 12), usage=z(1, 2, 48))
    for bad in (dict(lse=z(2, 11)), dict(lse=z(2, 12).double()), dict(usage=z(1, 2, 47)), dict(usage=z(1, 1, 48)),
                dict(usage=z(2, 48)), dict(usage=z(1, 2, 48).double()), dict(prev=z(2, 2, 48)), dict(rows=i32(0, 0)),
                dict(rows=i32(0).long()), dict(prefix_lens=i32(0, 0)), dict(q=good["q"].float()), dict(kv_lens=i32(2, 2)),
                dict(usage=z(0, 2, 48))):
        with pytest.raises(ValueError):
            c.usage(**{**good, **bad})
    good = dict(block_table=z((2, 3), dtype=torch.int32), kv_lens=i32(40, 2), usage=z(2, 2, 48), new_table=z((2, 2), dtype=torch.int32),
                budget=32)
    for bad in (dict(block_table=z((2, 3))), dict(kv_lens=i32(40)), dict(usage=z(1, 2, 48)), dict(usage=z(2, 2, 32)),
                dict(new_table=z((1, 2), dtype=torch.int32)), dict(new_table=z((2, 1), dtype=torch.int32)), dict(budget=0),
                dict(limit=31), dict(sinks=-1), dict(recent=-1), dict(sinks=30, recent=3), dict(new_usage=z(3, 2, 48)),
                dict(rows=i32(0)), dict(new_table=z((2, 2)))):
        with pytest.raises(ValueError):
            c.evict(**{**good, **bad})
    with pytest.raises(ValueError, match="not on a GPU"):
        c.evict(**good)


def test_oracle():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((5, 6, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    see = oracle.visible_prefill(5, 9, 0)
    _, lse, _, _ = oracle.attend(q, k, v, see, 0.3, 2.0)
    u, _ = oracle.usage(q, k, see, lse, 0.3, 2.0)
    z = torch.from_numpy(np.einsum("nhd,khd->hnk", q, np.repeat(k, 3, axis=1)) * 0.3)
    z = (2.0 * torch.tanh(z / 2.0)).masked_fill(~torch.from_numpy(see), -np.inf)
    ref = z.softmax(-1).view(2, 3, 5, 9).sum((1, 2)).numpy()
    assert np.allclose(u, ref, rtol=0, atol=1e-12) and np.allclose(u.sum(axis=1), 15)
    w = np.array([9, 1, 5, 5, np.nan, 5, 0, 2, 8, 1], float)
    assert oracle.kept_tokens(w, 10, 5, 1, 1).tolist() == [0, 2, 3, 8, 9]
    assert oracle.kept_tokens(w, 10, 9, 0, 0).tolist() == [0, 1, 2, 3, 5, 6, 7, 8, 9]
    assert oracle.kept_tokens(w, 10, 2, 2, 0).tolist() == [0, 1]
    w[6] = -np.inf
    assert oracle.kept_tokens(w, 10, 9, 0, 0).tolist() == [0, 1, 2, 3, 5, 6, 7, 8, 9]
