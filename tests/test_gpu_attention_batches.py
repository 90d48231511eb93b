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


def attention_time(ns, kvs, Hq, Hkv, D, page, width):
    """Microseconds of one prefill call on random bits, the least of seven; a table of `width` tokens."""
    pages = sum(-(-k // page) for k in kvs)
    kv = torch.randn((pages, 2, Hkv, page, D), dtype=torch.bfloat16, device=DEV)
    table, at = torch.zeros((len(ns), width // page), dtype=torch.int32, device=DEV), 0
    for s, k in enumerate(kvs):
        n = -(-k // page)
        table[s, :n] = torch.arange(at, at + n, device=DEV)
        at += n
    T = sum(ns)
    q = torch.randn((T, Hq, D), dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(q)
    cu, lens = up(np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)), up(np.array(kvs, np.int32))
    n = L.moe_attention_workspace_bytes(len(ns), T, max(ns), Hq, Hkv, D)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    best = 1e30
    for _ in range(7):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        L.moe_prefill_attention(q, Hq * D, kv[:, 0], kv[:, 1], L.KV_BF16, None, None, pages, page, kv.stride(0), table,
                                table.shape[1], cu, lens, None, len(ns), T, max(ns), Hq, Hkv, D, D ** -0.5, 0.0, out, None,
                                ws, n)
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3)
    return best


def test_a_long_sequence_does_not_hold_up_a_chunk():
    """A prompt's chunk with one decoding sequence of 131072 cached tokens takes about as long as the two alone, wherever
    in the batch it stands: its keys are shared out, not walked by one workgroup (10 times the sum)."""
    heads, width = (96, 8, 128, 64), 131072
    alone = attention_time([2048], [2048], *heads, width) + attention_time([1], [131072], *heads, width)
    for ns, kvs in (([1, 2048], [131072, 2048]), ([2048, 1], [2048, 131072])):
        both = attention_time(ns, kvs, *heads, width)
        note(f"chunk of 2048 and one of 131072: {both:.0f} us together, {alone:.0f} alone")
        assert both < 2 * alone


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ns,kvs", [
    ([1950], [1950]),                                                 # alike: whole segments
    ([1950, 1], [1950, 9000]),                                        # one long one: equal parts
    ([25] * 80, [25] * 79 + [7000]),                                  # more sequences than a wavefront has lanes, either way
    ([25] * 80, [25 + i for i in range(80)]),
    ([0] * 70 + [1950], [5] * 70 + [1950]),
])
def test_many_segments_under_a_wide_table(ns, kvs, fp8):
    """Over 1536 row tiles by the rows of q: the lengths, not the table's width, decide how they are shared out."""
    c = make_case(ns, kvs, 96, 8, 64, 64, fp8, seed=len(ns), lead=1, tail=2)
    assert 8 * (c.T // (128 // 12)) >= 1536
    see = [oracle.visible_prefill(n, k, 0) for n, k in zip(ns, kvs)]
    run_check(c, "prefill", None, see, wide=True)


@pytest.mark.parametrize("fp8", [False, True])
def test_padded_rows_are_no_segments(fp8):
    """A q of many rows behind the last sequence (a captured step's padding): few segments, shared out by their lengths."""
    c = make_case([40, 3, 1], [400, 3, 9000], 96, 8, 64, 64, fp8, seed=2, tail=2000)
    run_check(c, "prefill", None, [oracle.visible_prefill(n, k, 0) for n, k in zip(c.ns, c.kvs)], wide=True)


@pytest.mark.parametrize("fp8", [False, True])
def test_replays_that_change_how_segments_are_shared_out(fp8):
    """Captured once; lengths that make whole segments and lengths that make equal parts take turns, with eager calls between:
    each replay's bits are the eager call's, and nothing of the turn before is left in the workspace."""
    ns, page = [1950, 1], 64
    cases = []
    for kvs in ([1950, 20000], [1950, 300], [2400, 9000], [1960, 1]):
        used = sum(-(-k // page) for k in kvs)
        c = make_case(ns, kvs, 96, 8, 64, page, fp8, seed=kvs[1], extra_pages=360 - used)
        t = np.zeros((2, 400), np.int32)
        t[:, :c.table.shape[1]] = np.where(c.table == 1 << 30, 0, c.table)
        c.table = t
        cases.append(c)
    devs = [Dev(c) for c in cases]
    eager = []
    for d in devs:
        d.call("prefill")
        torch.cuda.synchronize()
        eager.append((bits_of(d.out).copy(), d.lse.cpu().numpy().copy()))
    # one of each kind against the oracle, the others against these by their bits
    for i in (0, 1):
        check_rows(cases[i], *eager[i], [oracle.visible_prefill(n, k, 0) for n, k in zip(ns, cases[i].kvs)], 64 ** -0.5, 0.0)
    g, stream, graph = Dev(cases[1]), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    note(f"replays between whole segments and equal parts fp8={fp8}")
    with torch.cuda.stream(stream):
        g.call("prefill", stream=stream)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            g.call("prefill", stream=stream)
    for i in (0, 1, 2, 3, 1, 0, 3, 2):
        for name in ("q", "kv", "table", "cu", "kvl", "ks", "vs"):
            getattr(g, name).copy_(getattr(devs[i], name))
        g.out.fill_(0x7FC1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(bits_of(g.out), eager[i][0]) and np.array_equal(g.lse.cpu().numpy(), eager[i][1]), i
        devs[i].call("prefill")
        torch.cuda.synchronize()
        assert np.array_equal(bits_of(devs[i].out), eager[i][0])
