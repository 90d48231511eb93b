"""Host-side checks of moe_window_attention (no GPU needed): every refusal comes before a launch, with fake 16-byte
aligned pointers that are never dereferenced; PagedKVCache.window_attention's own checks on CPU tensors; the oracle's mask."""
import numpy as np
import pytest
import torch

import oracle

FAKE, MIS = 0x10000, 0x10004


@pytest.fixture(scope="module")
def L():
    from shared_routed_expert_amd import _lib
    return _lib


def window(L, **kw):
    a = dict(q=FAKE, q_stride=12 * 128, k_cache=FAKE, v_cache=FAKE, kv_type=0, k_scale=None, v_scale=None, num_pages=8,
             page_size=16, page_stride=4096, block_table=FAKE, max_pages=4, cu_q=FAKE, kv_lens=FAKE, window=64, sinks=4, S=2,
             T=4, max_q=2, num_q_heads=12, num_kv_heads=1, head_dim=128, scale=0.1, softcap=0.0, out=FAKE, lse=FAKE,
             workspace=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return L.moe_window_attention(**a, stream=0, check=False)


def test_rejects(L):
    for kw in (dict(window=0), dict(window=-1), dict(sinks=-1), dict(S=-1), dict(T=-1), dict(T=(1 << 20) + 1), dict(max_q=0),
               dict(num_q_heads=0), dict(num_kv_heads=0), dict(num_kv_heads=5), dict(q_stride=12 * 128 - 8),
               dict(q_stride=12 * 128 + 4), dict(kv_type=3), dict(num_pages=0), dict(page_stride=2032), dict(max_pages=0),
               dict(scale=0.0), dict(scale=float("nan")), dict(scale=2e6), dict(softcap=-1.0), dict(softcap=1e-7),
               dict(kv_type=1), dict(kv_type=1, k_scale=FAKE)):
        assert window(L, **kw) == -1, kw
    for kw in (dict(head_dim=80), dict(page_size=8), dict(page_size=24), dict(S=65537), dict(num_pages=1 << 27),
               dict(num_q_heads=129, q_stride=1 << 20), dict(max_pages=1 << 26)):
        assert window(L, **kw) == -2, kw
    for name in ("q", "k_cache", "v_cache", "block_table", "cu_q", "kv_lens", "out", "workspace"):
        assert window(L, **{name: None}) == -1, name
        assert window(L, **{name: MIS}) == -1, name
    assert window(L, lse=MIS) == -1
    assert window(L, ws_bytes=0) == -3
    assert window(L, T=0, q=None) == 0
    assert window(L, S=0, q=None) == 0


def test_cache_object_rejects(L):
    from shared_routed_expert_amd import PagedKVCache
    c = PagedKVCache(4, 16, 1, 128, device="cpu")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)
    good = dict(q=torch.zeros((2, 12, 128), dtype=torch.bfloat16), block_table=torch.zeros((1, 2), dtype=torch.int32),
                cu_q=i32(0, 2), kv_lens=i32(2), max_q=2, window=8, sinks=1)
    for bad in (dict(window=0), dict(window=2 ** 31), dict(window=8.0), dict(sinks=-1), dict(sinks=None),
                dict(q=good["q"].float()), dict(kv_lens=i32(2, 2)), dict(lse=torch.zeros(2, 11))):
        with pytest.raises(ValueError):
            c.window_attention(**{**good, **bad})
    with pytest.raises(ValueError, match="not on a GPU"):
        c.window_attention(**good)


def test_oracle_mask():
    assert oracle.visible_window(2, 5, 2, 1).tolist() == [[True, False, True, True, False], [True, False, False, True, True]]
    assert oracle.visible_window(3, 1, 9, 9).tolist() == [[False], [False], [True]]
    for n, kv, window, sinks in ((7, 30, 5, 3), (30, 30, 100, 0), (4, 9, 1, 9)):
        see = oracle.visible_window(n, kv, window, sinks)
        for i in range(n):
            for j in range(kv):
                p = kv - n + i
                assert see[i, j] == (j <= p and (j > p - window or j < sinks))
    assert np.array_equal(oracle.visible_window(6, 20, 20, 0), oracle.visible_prefill(6, 20, 0))
