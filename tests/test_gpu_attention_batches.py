"""Batches that mix what a step mixes, against the float64 oracle (bars as in test_gpu_attention_scores): a long sequence
among many short segments, more drafted tokens than max_q under masks, the most heads, keys and values apart."""
import numpy as np
import pytest
import torch

import oracle
from shared_routed_expert_amd import _lib as L
from tests.gpu_util import note, DEV
from tests.kv_util import make_case, random_tree
from tests.test_gpu_attention import Dev, bits_of, run_check, up
from tests.test_gpu_attention_scores import check_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_a_long_sequence_among_many_whole_segments(fp8, first):
    """A prompt's chunk of over 1536 row tiles (each taken whole) with one decoding sequence of 20000 cached tokens, before
    or behind it in the batch."""
    ns, kvs = [1950, 1], [1950, 20000]
    if first:
        ns, kvs = ns[::-1], kvs[::-1]
    c = make_case(ns, kvs, 96, 8, 64, 64, fp8, seed=21)
    assert 8 * (c.T // (128 // 12)) >= 1536
    run_check(c, "prefill", None, [oracle.visible_prefill(n, k, 0) for n, k in zip(ns, kvs)])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("max_q", [2, 5, 64])
def test_masked_tokens_past_max_q(max_q, fp8):
    """Sequences of more drafted tokens than max_q, of more than 64 even: the first max_q rows see their context and
    the tokens that their words' 64 bits name (the later ones among them are cached too); the other rows keep their bytes."""
    ns, kvs = [9, 70, 3, 90], [50, 700, 3, 95]
    c = make_case(ns, kvs, 12, 1, 128, 16, fp8, seed=max_q, lead=1, tail=2)
    rng = np.random.default_rng(max_q)
    words = rng.integers(0, 1 << 63, c.T).astype(np.uint64) * np.uint64(2) + np.uint64(1)
    words[c.cu_q[2]] = 0
    sees = []
    for s, (n, k) in enumerate(zip(ns, kvs)):
        see = np.zeros((n, k), bool)
        see[:, :k - n] = True
        for i in range(n):
            w = int(words[c.cu_q[s] + i])
            for b in range(min(n, 64)):
                see[i, k - n + b] = bool(w >> b & 1)
        sees.append(see)
    d = Dev(c)
    d.max_q = max_q
    d.ws_bytes = L.moe_attention_workspace_bytes(4, c.T, max_q, c.Hq, c.Hkv, c.D)
    d.out.fill_(0x7FC1)
    d.lse.fill_(7.0)
    note(f"masked tokens past max_q={max_q} fp8={fp8}")
    d.call("tree", up(words.view(np.int64)))
    torch.cuda.synchronize()
    out, lse = bits_of(d.out), d.lse.cpu().numpy()
    computed = np.zeros(c.T, bool)
    for s, n in enumerate(ns):
        m = min(n, max_q)
        computed[c.cu_q[s]:c.cu_q[s] + m] = True
        sees[s] = sees[s][:m]
        c.ns[s] = m
    assert np.all(out[~computed] == 0x7FC1) and np.all(lse[~computed] == 7.0)
    check_rows(c, out, lse, sees, 128 ** -0.5, 0.0)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,n", [(1024, 1024, 64, 1), (1024, 8, 64, 3), (1024, 1024, 256, 40)])
def test_the_most_heads(Hq, Hkv, D, n, fp8):
    ns, kvs = [n, 1], [n + 33, 100]
    c = make_case(ns, kvs, Hq, Hkv, D, 16, fp8, seed=D)
    run_check(c, "tree", None, [oracle.visible_tree(a, k, None) for a, k in zip(ns, kvs)])


@pytest.mark.parametrize("which", ["tree", "prefill"])
@pytest.mark.parametrize("fp8", [False, True])
def test_keys_and_values_apart_and_shared_pages(fp8, which):
    """Two allocations with pages back to back, and two sequences whose first pages are the same ones."""
    n, kvs = 4 if which == "tree" else 50, [260, 190]
    c = make_case([n, n], kvs, 8, 2, 128, 32, fp8, seed=9)
    c.table[1, :3] = c.table[0, :3]
    for x in (c.k, c.v):
        x[1][:96] = x[0][:96]
    d = Dev(c)
    k, v = (d.kv[:, w].contiguous() for w in range(2))
    call = L.moe_tree_attention if which == "tree" else L.moe_prefill_attention
    note(f"keys and values apart, {which} fp8={fp8}")
    call(d.q, c.q.shape[1], k, v, L.KV_E4M3 if fp8 else L.KV_BF16, d.ks if fp8 else None, d.vs if fp8 else None,
         k.shape[0], 32, k.stride(0), d.table, c.table.shape[1], d.cu, d.kvl, None, 2, c.T, n, 8, 2, 128, 128 ** -0.5, 0.0,
         d.out, d.lse, d.ws, d.ws_bytes)
    torch.cuda.synchronize()
    see = oracle.visible_tree if which == "tree" else oracle.visible_prefill
    check_rows(c, bits_of(d.out), d.lse.cpu().numpy(), [see(n, x, None if which == "tree" else 0) for x in kvs],
               128 ** -0.5, 0.0)
