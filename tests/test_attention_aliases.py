"""The attention calls where out or lse lies over q or over one another (no GPU needed: every refusal comes before a launch,
with addresses that are never dereferenced). Segments that are split read q in one workgroup while another writes out."""
import pytest

Q, OUT, LSE = 0x4000000, 0x5000000, 0x6000000
T, HQ, D = 40, 12, 128
ROW = HQ * D * 2
INVALID = -1


@pytest.fixture(scope="module")
def L():
    from shared_routed_expert_amd import _lib
    return _lib


def call(L, which, **kw):
    a = dict(q=Q, q_stride=HQ * D, k_cache=0x1000000, v_cache=0x2000000, kv_type=0, k_scale=None, v_scale=None, num_pages=8,
             page_size=16, page_stride=4096, block_table=0x3000000, max_pages=4, cu_q=0x3001000, kv_lens=0x3002000, S=2, T=T,
             max_q=20, num_q_heads=HQ, num_kv_heads=1, head_dim=D, scale=0.1, softcap=0.0, out=OUT, lse=LSE,
             workspace=0x7000000, ws_bytes=1 << 40)
    a |= {"window": dict(window=64, sinks=4), "prefill": dict(prefix_lens=None), "tree": dict(tree_mask=None)}[which]
    a.update(kw)
    return getattr(L, f"moe_{which}_attention")(**a, stream=0, check=False)


@pytest.mark.parametrize("which", ["window", "prefill", "tree"])
def test_rejects(L, which):
    for kw in (dict(out=Q), dict(out=Q + ROW), dict(out=Q - T * ROW + 16), dict(out=Q + T * ROW - 16), dict(lse=Q), dict(lse=Q + 16),
               dict(lse=Q - T * HQ * 4 + 16), dict(lse=OUT), dict(lse=OUT + T * ROW - 16), dict(out=LSE + T * HQ * 4 - 16),
               dict(out=Q, q_stride=2 * HQ * D), dict(out=Q + ROW, q_stride=2 * HQ * D),
               dict(lse=Q + (T - 1) * 4 * ROW, q_stride=4 * HQ * D), dict(out=Q, lse=None)):
        assert call(L, which, **kw) == INVALID, kw

