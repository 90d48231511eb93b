"""Host-side checks of the paged-cache calls (no GPU needed): every refusal comes before a launch, with fake
16-byte aligned pointers that are never dereferenced; and PagedKVCache's own checks on CPU tensors."""
import numpy as np
import pytest
import torch

import oracle
from tests.kv_util import make_case, random_tree

FAKE, MIS = 0x10000, 0x10004


@pytest.fixture(scope="module")
def L():
    from shared_routed_expert_amd import _lib
    return _lib


def append(L, **kw):
    a = dict(qkv=FAKE, qkv_stride=14 * 128, T=4, num_q_heads=12, num_kv_heads=1, head_dim=128, rotary_dim=64, neox=True,
             q_norm_w=FAKE, k_norm_w=FAKE, eps=1e-5, positions=FAKE, cos_sin=FAKE, max_pos=4096, slots=FAKE, q_out=FAKE,
             k_cache=FAKE, v_cache=FAKE, kv_type=0, k_scale=None, v_scale=None, num_pages=8, page_size=16,
             page_stride=2048)
    a.update(kw)
    return L.moe_kv_append(**a, stream=0, check=False)


def test_append_rejects(L):
    for kw in (dict(T=-1), dict(T=(1 << 20) + 1), dict(num_q_heads=-1), dict(num_kv_heads=0), dict(eps=-1.0),
               dict(eps=float("nan")), dict(kv_type=2), dict(kv_type=-1), dict(num_pages=0), dict(max_pos=0),
               dict(qkv_stride=14 * 128 - 8), dict(qkv_stride=14 * 128 + 4), dict(page_stride=2032),
               dict(page_stride=2056), dict(q_norm_w=None), dict(k_norm_w=None), dict(kv_type=1),
               dict(kv_type=1, k_scale=FAKE), dict(kv_type=1, v_scale=FAKE)):
        assert append(L, **kw) == -1, kw
    for kw in (dict(head_dim=96), dict(rotary_dim=48), dict(rotary_dim=8), dict(rotary_dim=256), dict(page_size=8),
               dict(page_size=48), dict(page_size=2048, page_stride=1 << 20), dict(num_q_heads=1023, qkv_stride=1 << 20),
               dict(num_pages=1 << 27), dict(max_pos=1 << 26)):
        assert append(L, **kw) == -2, kw
    for name in ("qkv", "positions", "cos_sin", "slots", "q_out", "k_cache", "v_cache"):
        assert append(L, **{name: None}) == -1, name
        assert append(L, **{name: MIS}) == -1, name
    for name in ("q_norm_w", "k_norm_w", "k_scale", "v_scale"):
        assert append(L, kv_type=1, **{**dict(k_scale=FAKE, v_scale=FAKE), name: MIS}) == -1, name
    assert append(L, T=0, qkv=None) == 0


def attention(L, which, **kw):
    a = dict(q=FAKE, q_stride=12 * 128, k_cache=FAKE, v_cache=FAKE, kv_type=0, k_scale=None, v_scale=None, num_pages=8,
             page_size=16, page_stride=4096, block_table=FAKE, max_pages=4, cu_q=FAKE, kv_lens=FAKE, S=2, T=4, max_q=2,
             num_q_heads=12, num_kv_heads=1, head_dim=128, scale=0.1, softcap=0.0, out=FAKE, lse=FAKE, workspace=FAKE,
             ws_bytes=1 << 40)
    a["tree_mask" if which == "tree" else "prefix_lens"] = None
    a.update(kw)
    return getattr(L, f"moe_{which}_attention")(**a, stream=0, check=False)


@pytest.mark.parametrize("which", ["tree", "prefill"])
def test_attention_rejects(L, which):
    for kw in (dict(S=-1), dict(T=-1), dict(T=(1 << 20) + 1), dict(max_q=0), dict(num_q_heads=0), dict(num_kv_heads=0),
               dict(num_q_heads=12, num_kv_heads=5), dict(q_stride=12 * 128 - 8), dict(q_stride=12 * 128 + 4),
               dict(kv_type=3), dict(num_pages=0), dict(page_stride=2032), dict(page_stride=4104), dict(max_pages=0),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(scale=2e6), dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=1e-7), dict(softcap=1e7), dict(kv_type=1), dict(kv_type=1, k_scale=FAKE)):
        assert attention(L, which, **kw) == -1, kw
    for kw in (dict(head_dim=80), dict(page_size=8), dict(page_size=24), dict(S=65537), dict(num_pages=1 << 27),
               dict(num_q_heads=129, q_stride=1 << 20), dict(num_q_heads=2048, num_kv_heads=64, q_stride=1 << 20),
               dict(max_pages=1 << 26)):
        assert attention(L, which, **kw) == -2, kw
    for name in ("q", "k_cache", "v_cache", "block_table", "cu_q", "kv_lens", "out", "workspace"):
        assert attention(L, which, **{name: None}) == -1, name
        assert attention(L, which, **{name: MIS}) == -1, name
    for name in ("lse", "tree_mask" if which == "tree" else "prefix_lens"):
        assert attention(L, which, **{name: MIS}) == -1, name
    assert attention(L, which, ws_bytes=0) == -3
    assert attention(L, which, T=0, q=None) == 0
    assert attention(L, which, S=0, q=None) == 0


def test_tree_has_at_most_64_tokens(L):
    assert attention(L, "tree", max_q=65) == -2
    assert attention(L, "prefill", max_q=65, ws_bytes=0) == -3


def test_workspace_bytes(L):
    assert L.moe_attention_workspace_bytes(2, 4, 2, 12, 1, 128) > 0
    assert L.moe_attention_workspace_bytes(2, 4, 2, 12, 1, 96) == 0
    assert L.moe_attention_workspace_bytes(2, 4, 2, 12, 5, 128) == 0
    assert L.moe_attention_workspace_bytes(-1, 4, 2, 12, 1, 128) == 0


def test_oracle_attention_against_torch():
    """The float64 oracle against torch's softmax on one dense sequence."""
    rng = np.random.default_rng(3)
    c = make_case([5], [23], 6, 2, 64, 16, False, 4)
    see = oracle.visible_tree(5, 23, random_tree(5, rng))
    out, lse, _, _ = oracle.attend(c.q_heads(0), c.k[0], c.v[0], see, 0.125, 5.0)
    q, k, v = (torch.from_numpy(x) for x in (c.q_heads(0), c.k[0], c.v[0]))
    z = torch.einsum("nhd,khd->hnk", q, k.repeat_interleave(3, 1)) * 0.125
    z = (5.0 * torch.tanh(z / 5.0)).masked_fill(~torch.from_numpy(see), -np.inf)
    ref = torch.einsum("hnk,khd->nhd", z.softmax(-1), v.repeat_interleave(3, 1))
    assert np.allclose(out, ref.numpy(), rtol=0, atol=1e-12)
    assert np.allclose(lse, z.logsumexp(-1).T.numpy(), rtol=0, atol=1e-12)
    assert oracle.visible_prefill(2, 4, 0).tolist() == [[True, True, True, False], [True] * 4]
    assert oracle.visible_prefill(2, 4, 4).tolist() == [[True] * 4] * 2
    out, lse, _, _ = oracle.attend(c.q_heads(0), c.k[0], c.v[0], np.zeros((5, 23), bool), 0.125)
    assert not out.any() and np.all(lse == -np.inf)


def test_cache_object_rejects(L):
    from shared_routed_expert_amd import PagedKVCache, KV_E4M3
    with pytest.raises(ValueError):
        PagedKVCache(4, 24, 1, 128, device="cpu")
    with pytest.raises(ValueError):
        PagedKVCache(4, 16, 1, 96, device="cpu")
    with pytest.raises(ValueError):
        PagedKVCache(4, 16, 1, 128, KV_E4M3, device="cpu")          # no scales
    with pytest.raises(ValueError):
        PagedKVCache(4, 16, 2, 128, KV_E4M3, torch.ones(1), torch.ones(2), device="cpu")
    c = PagedKVCache(4, 16, 1, 128, device="cpu")
    q = torch.zeros((2, 12, 128), dtype=torch.bfloat16)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)
    table = torch.zeros((1, 2), dtype=torch.int32)
    good = dict(q=q, block_table=table, cu_q=i32(0, 2), kv_lens=i32(2), max_q=2)
    for bad in (dict(q=q.float()), dict(q=q[..., :64]), dict(block_table=table.long()), dict(block_table=table[0]),
                dict(cu_q=i32(0, 1, 2)), dict(kv_lens=i32(2, 2)), dict(kv_lens=i32(2).long()),
                dict(tree_mask=torch.zeros(2, dtype=torch.int32)), dict(tree_mask=torch.zeros(3, dtype=torch.int64)),
                dict(out=torch.zeros(2, 12, 128)), dict(lse=torch.zeros(2, 11))):
        with pytest.raises(ValueError):
            c.tree_attention(**{**good, **bad})
    with pytest.raises(ValueError):
        c.prefill_attention(**good, prefix_lens=i32(0, 0))
    row = torch.zeros((2, 14 * 128), dtype=torch.bfloat16)
    for bad in (dict(qkv=row.float()), dict(qkv=row[:, :-8]), dict(slots=i32(0)), dict(slots=i32(0, 1).long()),
                dict(positions=None), dict(q_norm_w=torch.ones(128)), dict(q_out=torch.zeros(2, 12, 128))):
        with pytest.raises(ValueError):
            c.append(**{**dict(qkv=row, num_q_heads=12, slots=i32(0, 1), positions=i32(0, 1),
                               cos_sin=torch.zeros(8, 64)), **bad})
