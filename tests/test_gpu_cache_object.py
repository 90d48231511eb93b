"""PagedKVCache's own results: what it returns for rows that no sequence has, and its options, against the float64 oracle
(bars as in test_gpu_attention_scores)."""
import numpy as np
import pytest
import torch

import oracle
from shared_routed_expert_amd import PagedKVCache, _lib as L
from tests.gpu_util import note, DEV
from tests.kv_util import make_case, random_tree
from tests.test_gpu_attention import bits_of, up
from tests.test_gpu_attention_scores import check_rows

pytestmark = pytest.mark.gpu


def cache_of(c):
    scales = up(c.scales) if c.fp8 else None
    cache = PagedKVCache(c.kv.shape[0], c.page, c.Hkv, c.D, L.KV_E4M3 if c.fp8 else L.KV_BF16,
                         scales[0].clone() if c.fp8 else None, scales[1].clone() if c.fp8 else None, DEV)
    cache.kv.view(torch.uint8 if c.fp8 else torch.int16).copy_(up(c.kv if c.fp8 else c.kv.view(np.int16)))
    return cache


def q_of(c):
    return up(c.q.view(np.int16)).view(torch.bfloat16)[:, :c.Hq * c.D].unflatten(1, (c.Hq, c.D))


def leave_nan_in_the_allocator(nbytes):
    """Blocks of this size that torch hands out next hold NaN patterns."""
    blocks = [torch.full((nbytes // 2,), 0x7FC1, dtype=torch.int16, device=DEV) for _ in range(4)]
    torch.cuda.synchronize()
    del blocks


@pytest.mark.parametrize("which", ["tree", "prefill"])
def test_rows_of_no_sequence_are_zero(which):
    """Padding before and behind the sequences and a sequence's tokens past max_q: zeros in a result that the call
    allocates, left as they were in the caller's own."""
    ns, kvs, max_q = [9, 3], [50, 3], 5
    c = make_case(ns, kvs, 12, 1, 128, 16, False, seed=2, lead=2, tail=7)
    cache, q = cache_of(c), q_of(c)
    call = cache.tree_attention if which == "tree" else cache.prefill_attention
    args = (q, up(c.table), up(c.cu_q), up(np.array(kvs, np.int32)), max_q)
    leave_nan_in_the_allocator(q.numel() * 2)
    note(f"rows of no sequence, {which}")
    out = bits_of(call(*args).view(torch.int16))
    mine = torch.full((c.T, 12, 128), 0x7FC1, dtype=torch.int16, device=DEV)
    kept = bits_of(call(*args, out=mine.view(torch.bfloat16)).view(torch.int16))
    computed = np.zeros(c.T, bool)
    for s, n in enumerate(ns):
        computed[c.cu_q[s]:c.cu_q[s] + min(n, max_q)] = True
    assert np.array_equal(out[computed], kept[computed]) and out[computed].any(axis=(1, 2)).all()
    assert not out[~computed].any()
    assert np.all(kept[~computed] == 0x7FC1)


def test_captured_calls_of_the_object():
    """A captured call allocates its result and workspace in the graph: every replay, on other lengths than at capture and
    with eager work between, gives the eager result, zeros behind the last sequence included."""
    c = make_case([1, 1, 1], [700, 90, 333], 12, 1, 128, 16, False, seed=6, tail=5)
    cache, q, table, cu = cache_of(c), q_of(c), up(c.table), up(c.cu_q)
    lens = torch.tensor(c.kvs, dtype=torch.int32, device=DEV)
    call = lambda: cache.tree_attention(q, table, cu, lens, 1)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        call()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            out = call()
    for kvs in ([700, 90, 333], [16, 1, 300], [5, 90, 17], [699, 80, 1]):
        lens.copy_(torch.tensor(kvs, dtype=torch.int32))
        out.fill_(9.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = bits_of(out.view(torch.int16)).copy()
        assert np.array_equal(got, bits_of(call().view(torch.int16))), kvs
        assert not got[3:].any() and got[:3].any(axis=(1, 2)).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("cap", [0.0, 25.0])
def test_options_of_the_object(fp8, cap):
    """prefix_lens, tree_mask, a scale, a cap, out and lse of the caller's own, q as a slice of wider rows."""
    ns, kvs, pre = [30, 64, 2], [200, 64, 91], [50, 0, 91]
    c = make_case(ns, kvs, 12, 1, 128, 16, fp8, seed=3, q_extra=24)
    cache, q, scale = cache_of(c), q_of(c), 0.05
    assert not q.is_contiguous()
    lens = up(np.array(kvs, np.int32))
    words = [random_tree(n, np.random.default_rng(n)) for n in ns]
    for call, extra, sees in (
            (cache.prefill_attention, dict(prefix_lens=up(np.array(pre, np.int32))),
             [oracle.visible_prefill(n, k, p) for n, k, p in zip(ns, kvs, pre)]),
            (cache.tree_attention, dict(tree_mask=up(np.concatenate(words).view(np.int64))),
             [oracle.visible_tree(n, k, w) for n, k, w in zip(ns, kvs, words)])):
        out = torch.empty((c.T, 12, 128), dtype=torch.bfloat16, device=DEV)
        lse = torch.empty((c.T, 12), device=DEV)
        got = call(q, up(c.table), up(c.cu_q), lens, 64, scale=scale, softcap=cap, out=out, lse=lse, **extra)
        torch.cuda.synchronize()
        assert got is out
        check_rows(c, bits_of(out.view(torch.int16)), lse.cpu().numpy(), sees, float(np.float32(scale)), cap)


def test_on_another_stream():
    """The calls go to torch's current stream: behind the work that made their inputs, with nothing on the default one."""
    c = make_case([1, 1], [900, 40], 12, 1, 128, 16, False, seed=5)
    cache, table, cu, lens = cache_of(c), up(c.table), up(c.cu_q), up(np.array(c.kvs, np.int32))
    src, q = q_of(c).contiguous(), torch.zeros((2, 12, 128), dtype=torch.bfloat16, device=DEV)
    want = bits_of(cache.tree_attention(src, table, cu, lens, 1).view(torch.int16)).copy()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    big = torch.randn((4096, 4096), device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for _ in range(4):
            big = big @ big * 1e-3
        q.copy_(src)
        out = cache.tree_attention(q, table, cu, lens, 1)
    stream.synchronize()
    assert np.array_equal(bits_of(out.view(torch.int16)), want)
