"""moe_kv_usage and moe_kv_evict where an output lies over a part of an input (no GPU needed: every refusal comes before a
launch, with addresses that are never dereferenced)."""
import pytest

ROWS, HEADS, PAGES, PAGE = 3, 2, 4, 16
BYTES = ROWS * HEADS * PAGES * PAGE * 4
U = 0x4000000
INVALID = -1


@pytest.fixture(scope="module")
def L():
    from shared_routed_expert_amd import _lib
    return _lib


def usage(L, **kw):
    a = dict(q=0x1000000, q_stride=4 * 128, k_cache=0x2000000, kv_type=0, k_scale=None, num_pages=8, page_size=PAGE,
             page_stride=HEADS * PAGE * 128, block_table=0x3000000, max_pages=PAGES, cu_q=0x3001000, kv_lens=0x3002000,
             prefix_lens=None, lse=0x3003000, S=3, T=4, max_q=2, num_q_heads=4, num_kv_heads=HEADS, head_dim=128, scale=0.1,
             softcap=0.0, prev=None, decay=1.0, usage=U, usage_rows=None, rows=ROWS, workspace=0x5000000, ws_bytes=1 << 40)
    a.update(kw)
    return L.moe_kv_usage(**a, stream=0, check=False)


def evict(L, **kw):
    a = dict(k_cache=0x1000000, v_cache=0x2000000, kv_type=0, num_pages=8, page_size=PAGE, page_stride=HEADS * PAGE * 128,
             block_table=0x3000000, max_pages=PAGES, kv_lens=0x3001000, usage=U, new_usage=0x5000000, usage_rows=None,
             rows=ROWS, S=3, num_kv_heads=HEADS, head_dim=128, limit=40, budget=32, sinks=4, recent=8, new_table=0x3002000,
             new_max_pages=2, new_lens=0x3003000, kept=0x3004000)
    a.update(kw)
    return L.moe_kv_evict(**a, stream=0, check=False)


def test_usage_over_a_part_of_prev(L):
    for off in (16, BYTES // ROWS, BYTES - 16, -16, -BYTES // ROWS, 16 - BYTES):
        assert usage(L, prev=U + off) == INVALID, off


def test_new_usage_over_a_part_of_usage(L):
    for off in (16, BYTES // ROWS, BYTES - 16, -16, -BYTES // ROWS, 16 - BYTES):
        assert evict(L, new_usage=U + off) == INVALID, off


def test_new_lens_over_a_part_of_kv_lens(L):
    for off in (0, 16, -16):
        assert evict(L, S=8, rows=8, new_lens=0x3001000 + off) == INVALID, off


def test_any_number_of_rows_is_no_overflow(L):
    """With usage_rows, rows may be as large as an int: its bytes pass 2^64 here."""
    more = dict(rows=2 ** 31 - 1, max_pages=1 << 25, usage_rows=0x3005000)
    assert usage(L, prev=U + 16, **more) == INVALID
    assert evict(L, new_usage=U + 16, **more) == INVALID
