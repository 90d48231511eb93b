"""PagedKVCache names the tensor that does not start where the kernels' loads need it to (no GPU needed): slices of a
batch's arrays are the usual way to split a step, and the library itself can only say that some argument is invalid."""
import pytest
import torch

from shared_routed_expert_amd import KV_E4M3, PagedKVCache


def i32(n):
    return torch.zeros(n, dtype=torch.int32)


def bf16(n):
    return torch.zeros(n, dtype=torch.bfloat16)


def at(t, off, *shape):
    """A contiguous view of t that starts `off` elements in."""
    n = 1
    for s in shape:
        n *= s
    return t[off:off + n].view(*shape)


@pytest.fixture(scope="module")
def cache():
    return PagedKVCache(4, 16, 1, 128, device="cpu")


def test_attention_arguments(cache):
    q = at(bf16(2 * 12 * 128), 0, 2, 12, 128)
    good = dict(q=q, block_table=at(i32(2), 0, 1, 2), cu_q=i32(2), kv_lens=i32(1), max_q=2)
    bad = dict(q=at(bf16(2 * 12 * 128 + 4), 4, 2, 12, 128), block_table=at(i32(3), 1, 1, 2), cu_q=at(i32(3), 1, 2),
               kv_lens=at(i32(4), 3, 1), out=at(bf16(2 * 12 * 128 + 1), 1, 2, 12, 128),
               lse=at(torch.zeros(26), 2, 2, 12))
    for name, t in bad.items():
        for call in (cache.tree_attention, cache.prefill_attention):
            with pytest.raises(ValueError, match=f"^{name} .*16-byte"):
                call(**{**good, name: t})
    with pytest.raises(ValueError, match="^tree_mask .*16-byte"):
        cache.tree_attention(**good, tree_mask=torch.zeros(3, dtype=torch.int64)[1:])
    with pytest.raises(ValueError, match="^prefix_lens .*16-byte"):
        cache.prefill_attention(**good, prefix_lens=i32(3)[2:])
    rows = bf16(2 * 1540).view(2, 1540)   # 1540 = 12 * 128 + 4
    with pytest.raises(ValueError, match="^rows of q .*multiple of 8"):
        cache.tree_attention(**{**good, "q": rows[:, :12 * 128].unflatten(1, (12, 128))})


def test_append_arguments(cache):
    row = 14 * 128
    good = dict(qkv=bf16(2 * row).view(2, row), num_q_heads=12, slots=i32(2), positions=i32(2), cos_sin=torch.zeros(8, 64),
                q_norm_w=torch.ones(128), k_norm_w=torch.ones(128))
    bad = dict(qkv=at(bf16(2 * row + 2), 2, 2, row), slots=i32(3)[1:], positions=i32(4)[2:],
               cos_sin=at(torch.zeros(8 * 64 + 1), 1, 8, 64), q_norm_w=torch.ones(130)[2:], k_norm_w=torch.ones(129)[1:],
               q_out=at(bf16(2 * 12 * 128 + 4), 4, 2, 12, 128))
    for name, t in bad.items():
        with pytest.raises(ValueError, match=f"^{name} .*16-byte"):
            cache.append(**{**good, name: t})
    with pytest.raises(ValueError, match="^rows of qkv .*multiple of 8"):
        cache.append(**{**good, "qkv": bf16(2 * (row + 4)).view(2, row + 4)[:, :row]})


def test_scales():
    """One layer's slice of all layers' scales."""
    scales = torch.ones(40)
    with pytest.raises(ValueError, match="^k_scale .*16-byte"):
        PagedKVCache(4, 16, 1, 128, KV_E4M3, scales[1:2], scales[4:5], device="cpu")
    with pytest.raises(ValueError, match="^v_scale .*16-byte"):
        PagedKVCache(4, 16, 1, 128, KV_E4M3, scales[4:5], scales[6:7], device="cpu")
    PagedKVCache(4, 16, 1, 128, KV_E4M3, scales[4:5], scales[8:9], device="cpu")


def test_aligned_slices_pass(cache):
    """Slices that start on the boundary reach the call itself (which wants a GPU)."""
    big = bf16(6 * 14 * 128).view(6, 14 * 128)
    with pytest.raises(ValueError, match="not on a GPU"):
        cache.append(big[4:, :], 12, i32(8)[4:6], i32(8)[4:6], torch.zeros(8, 64))
    with pytest.raises(ValueError, match="not on a GPU"):
        cache.tree_attention(big[:, :12 * 128].unflatten(1, (12, 128))[4:], i32(10)[4:8].view(1, 4), i32(8)[4:6], i32(8)[4:5], 2)
