"""moe_tree_attention and moe_prefill_attention against the float64 oracle on the same cached values.

Bars, per value, with A = sum_j w_j |v_j| (w the softmax weights) and X = the row's largest sum_d |q_d k_d| * scale:
  e   error of a score in float32: 2^-24 times (D + 8) X for the products and their sum, 4 |z| <= 4 X for scaling and the
      change to base 2, and 16 softcap for the tanh of two exponentials and a quotient
  out: 2^-8 |ref| + (u + 2 e + 2^-24 (2 kv + 64)) A: the output's own rounding to bf16, the weights' rounding u (2^-8
      for bf16 halves the spacing; 2^-11 for float16, an e4m3 cache), a score's error in numerator and denominator, and
      kv float32 additions in each of them
  lse: e + 2^-24 (kv + 64 + 4 |lse|)
Rows that see nothing: out exactly 0 and lse -inf. Rows outside every sequence keep their bytes. Cache bytes that are no
cached token hold NaN patterns.
"""
import numpy as np
import pytest
import torch

import oracle
from shared_routed_expert_amd import PagedKVCache, _lib as L
from tests.gpu_util import note, DEV
from tests.kv_util import make_case, random_tree
from workloads import f32_from_bf16_bits

pytestmark = pytest.mark.gpu


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


class Dev:
    """A case's arrays on the GPU, and one call on them."""

    def __init__(self, c):
        self.c = c
        self.q = up(c.q.view(np.int16))
        self.kv = up(c.kv if c.fp8 else c.kv.view(np.int16))
        self.scales = up(c.scales)
        self.ks, self.vs = self.scales[0].clone(), self.scales[1].clone()
        self.table, self.cu, self.kvl = up(c.table), up(c.cu_q), up(np.array(c.kvs, np.int32))
        self.max_q = max(max(c.ns), 1)
        self.out = torch.empty((c.T, c.Hq, c.D), dtype=torch.int16, device=DEV)
        self.lse = torch.empty((c.T, c.Hq), dtype=torch.float32, device=DEV)
        self.ws_bytes = L.moe_attention_workspace_bytes(len(c.ns), c.T, self.max_q, c.Hq, c.Hkv, c.D)
        self.ws = torch.full((self.ws_bytes + 512,), 0xCD, dtype=torch.uint8, device=DEV)

    def call(self, which, extra=None, scale=None, cap=0.0, lse=True, stream=None):
        c = self.c
        fn = L.moe_tree_attention if which == "tree" else L.moe_prefill_attention
        fn(self.q, c.q.shape[1], self.kv[:, 0], self.kv[:, 1], L.KV_E4M3 if c.fp8 else L.KV_BF16,
           self.ks if c.fp8 else None, self.vs if c.fp8 else None, c.kv.shape[0], c.page, self.kv.stride(0), self.table,
           c.table.shape[1], self.cu, self.kvl, extra, len(c.ns), c.T, self.max_q, c.Hq, c.Hkv, c.D,
           c.D ** -0.5 if scale is None else scale, cap, self.out, self.lse if lse else None, self.ws, self.ws_bytes, stream)


def bits_of(t):
    return t.cpu().numpy().view(np.uint16)


def check(c, out_bits, lse, sees, scale, cap, guard=0x7FC1):
    u = 2.0 ** -11 if c.fp8 else 2.0 ** -8
    touched = np.zeros(c.T, bool)
    worst = 0.0
    for s, n in enumerate(c.ns):
        if n == 0:
            continue
        a = int(c.cu_q[s])
        touched[a:a + n] = True
        ref, rl, mag, dot = oracle.attend(c.q_heads(s), c.k[s], c.v[s], sees[s], scale, cap)
        got = f32_from_bf16_bits(out_bits[a:a + n].copy()).astype(np.float64)
        X = dot[..., None]
        e = 2.0 ** -24 * ((c.D + 12) * X + 16 * cap)
        bound = 2.0 ** -8 * np.abs(ref) + (u + 2 * e + 2.0 ** -24 * (2 * c.kvs[s] + 64)) * mag + 1e-37
        err = np.abs(got - ref)
        assert np.all(err <= bound), (s, np.argwhere(~(err <= bound))[:3], np.max(err / np.maximum(bound, 1e-30)))
        worst = max(worst, float(np.max(err / np.maximum(bound, 1e-30), initial=0)))
        empty = ~sees[s].any(axis=1)
        assert not out_bits[a:a + n][empty].any()
        if lse is not None:
            g = lse[a:a + n].astype(np.float64)
            assert np.all(g[empty] == -np.inf)
            ok = ~empty
            be = e[..., 0] + 2.0 ** -24 * (c.kvs[s] + 64 + 4 * np.abs(np.where(np.isfinite(rl), rl, 0)))
            assert np.all(np.abs(g[ok] - rl[ok]) <= be[ok]), s
    assert np.all(out_bits[~touched] == guard)
    if lse is not None:
        assert np.all(lse[~touched] == 7.0)
    return worst


def run_check(c, which, extra_np, sees, scale=None, cap=0.0, lse=True, tag="", wide=False):
    """wide: a block table of far more columns than the sequences use (what they may hold, not what they do, decides
    how the kernels split the keys)."""
    if wide:
        t = np.full((c.table.shape[0], 131072 // c.page), 1 << 30, np.int32)
        t[:, :c.table.shape[1]] = c.table
        c.table = t
    d = Dev(c)
    d.out.fill_(0x7FC1)
    d.lse.fill_(7.0)
    note(f"{which} attention {tag} ns={c.ns[:6]} kvs={c.kvs[:6]} S={len(c.ns)} Hq={c.Hq} Hkv={c.Hkv} D={c.D} page={c.page} "
         f"fp8={c.fp8} cap={cap}")
    d.call(which, None if extra_np is None else up(extra_np), scale, cap, lse)
    torch.cuda.synchronize()
    assert bool((d.ws[d.ws_bytes:] == 0xCD).all())
    w = check(c, bits_of(d.out), d.lse.cpu().numpy() if lse else None, sees, c.D ** -0.5 if scale is None else scale, cap)
    note(f"  largest error / bound {w:.3f}")
    return d


HEADS = [(12, 1, 128), (96, 8, 128), (8, 2, 64), (7, 1, 64), (1, 1, 128), (4, 4, 128), (8, 1, 256), (16, 2, 256),
         (32, 1, 128), (128, 1, 64), (40, 1, 128)]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_single_tokens(Hq, Hkv, D, fp8, wide):
    """One token per sequence, lengths around the tile and page borders."""
    kvs = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000]
    c = make_case([1] * len(kvs), kvs, Hq, Hkv, D, 16, fp8, seed=Hq + D)
    run_check(c, "tree", None, [oracle.visible_tree(1, k, None) for k in kvs], wide=wide)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [16, 32, 128, 1024])
@pytest.mark.parametrize("Hq,Hkv,D", [(12, 1, 128), (8, 2, 64), (8, 1, 256)])
def test_trees(Hq, Hkv, D, page, fp8):
    rng = np.random.default_rng(page + D)
    ns = [1, 2, 3, 5, 8, 13, 33, 64, 0, 7]
    kvs = [1, 90, 3, 300, 8, 777, 97, 500, 12, 2100]
    c = make_case(ns, kvs, Hq, Hkv, D, page, fp8, seed=page, lead=2, tail=3, q_extra=8)
    words = np.zeros(c.T, np.uint64)
    sees = []
    for s, n in enumerate(ns):
        w = random_tree(n, rng)
        words[c.cu_q[s]:c.cu_q[s] + n] = w
        sees.append(oracle.visible_tree(n, kvs[s], w))
    run_check(c, "tree", words.view(np.int64), sees)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [2, 3, 5, 6, 11, 16, 22, 40])
def test_tree_sizes(n, fp8):
    """All sequences of one size, so that each row-tile size of the kernels is met with split keys."""
    rng = np.random.default_rng(n)
    kvs = [3000, n, 1500 + n]
    c = make_case([n] * 3, kvs, 12, 1, 128, 16, fp8, seed=n)
    w = [random_tree(n, rng) for _ in kvs]
    run_check(c, "tree", np.concatenate(w).view(np.int64), [oracle.visible_tree(n, k, x) for k, x in zip(kvs, w)])


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_empty_rows(fp8, wide):
    """Words that leave a row nothing, with and without a context; bits past the sequence's own tokens change nothing."""
    ns, kvs = [4, 3, 2, 1], [4, 3, 40, 1]
    c = make_case(ns, kvs, 12, 1, 128, 16, fp8, seed=1)
    words = np.array([0, 0b1111 | 1 << 63, 0b1 | 1 << 40, 0, 0, 0, 0, 0, 0b11 << 60, 0], np.uint64)
    sees, at = [], 0
    for n, k in zip(ns, kvs):
        sees.append(oracle.visible_tree(n, k, words[at:at + n]))
        at += n
    run_check(c, "tree", words.view(np.int64), sees, wide=wide)


@pytest.mark.parametrize("cap", [0.0, 4.0])
@pytest.mark.parametrize("fp8", [False, True])
def test_peaked_scores(fp8, cap):
    """Scores of some hundreds: the running maximum moves and weights underflow; lse may be left out."""
    ns, kvs = [1, 9, 2], [2000, 700, 65]
    c = make_case(ns, kvs, 12, 1, 128, 32, fp8, seed=9, big=30.0)
    sees = [oracle.visible_tree(n, k, None) for n, k in zip(ns, kvs)]
    run_check(c, "tree", None, sees, cap=cap)
    run_check(c, "tree", None, sees, cap=cap, lse=False)


PREFILL = [
    # (ns, kvs, Hq, Hkv, D, page, prefixes, cap)
    ([1], [1], 12, 1, 128, 16, None, 0.0),
    ([65], [65], 12, 1, 128, 16, None, 0.0),
    ([300], [300], 12, 1, 128, 16, None, 0.0),
    ([129, 1, 0, 77, 256], [129, 500, 5, 1077, 256], 12, 1, 128, 16, None, 0.0),
    ([130, 61], [700, 61], 96, 8, 128, 64, None, 0.0),
    ([200, 64, 128], [200, 64, 640], 8, 2, 64, 32, [50, 0, 640], 0.0),
    ([90, 200], [91, 333], 8, 1, 256, 16, None, 20.0),
    ([40, 80], [40, 333], 128, 1, 64, 16, [7, 1000], 0.0),
    ([257], [1500], 1, 1, 128, 128, [900], 5.0),
    ([70, 30], [70, 200], 40, 1, 128, 16, [-3, 30], 0.0),
    ([1030], [1031], 4, 2, 128, 16, None, 0.0),
]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ns,kvs,Hq,Hkv,D,page,prefixes,cap", PREFILL)
def test_prefill(ns, kvs, Hq, Hkv, D, page, prefixes, cap, fp8, wide):
    c = make_case(ns, kvs, Hq, Hkv, D, page, fp8, seed=sum(ns) + D, lead=1, tail=2, q_extra=16)
    pre = prefixes or [0] * len(ns)
    sees = [oracle.visible_prefill(n, k, p) for n, k, p in zip(ns, kvs, pre)]
    run_check(c, "prefill", None if prefixes is None else np.array(prefixes, np.int32), sees, cap=cap, wide=wide)


@pytest.mark.parametrize("fp8", [False, True])
def test_many_row_tiles(fp8):
    """Over 1536 row tiles: a workgroup takes a whole one, nothing is split or joined."""
    ns, kvs, pre = [1300, 0, 5, 870], [1400, 3, 5, 870], [200, 0, 0, 870]
    c = make_case(ns, kvs, 96, 8, 64, 32, fp8, seed=12, lead=3, tail=1)
    assert 8 * (c.T // (128 // 12)) >= 1536
    run_check(c, "prefill", np.array(pre, np.int32), [oracle.visible_prefill(n, k, p) for n, k, p in zip(ns, kvs, pre)])


@pytest.mark.parametrize("fp8", [False, True])
def test_what_the_workspace_held_does_not_matter(fp8):
    """Few and many sequences (one description per segment, or per part), each with the workspace full of other bytes."""
    for which, ns, kvs in (("tree", [1] * 6, [1, 700, 3, 40, 5000, 17]), ("tree", [1] * 600, [1 + i % 90 + 600 * (i == 5) for i in range(600)]),
                           ("prefill", [100, 3], [150, 900])):
        c = make_case(ns, kvs, 4, 1, 128, 16, fp8, seed=3)
        c.table = np.concatenate([c.table, np.full((len(ns), 4096), -7, np.int32)], 1)
        d = Dev(c)
        sees = [oracle.visible_tree(n, k, None) if which == "tree" else oracle.visible_prefill(n, k, 0) for n, k in zip(ns, kvs)]
        for byte in (0x01, 0x7F, 0xFF, 0x00):
            d.ws.fill_(byte)
            d.out.fill_(0x7FC1)
            d.lse.fill_(7.0)
            d.call(which)
            torch.cuda.synchronize()
            check(c, bits_of(d.out), d.lse.cpu().numpy(), sees, c.D ** -0.5, 0.0)


@pytest.mark.parametrize("fp8", [False, True])
def test_far_pages(fp8):
    """Pages whose byte offsets pass 2^32 (and element offsets 2^31): the last pages of a large pool, strided."""
    Hkv, D, page = 8, 128, 64
    stride = 4 * Hkv * page * D        # elements: half of every page's stretch belongs to nothing
    pages = (1 << 32) // stride + 20
    es = 1 if fp8 else 2
    pool = torch.empty(pages * stride * es, dtype=torch.uint8, device=DEV)
    pool.view(torch.int32).fill_(0x7FC07FC0 if not fp8 else 0x7F7F7F7F)
    kvs = [500, 70]
    c = make_case([1, 40], kvs, 16, Hkv, D, page, fp8, seed=5)
    far = np.array([pages - 1 - 3 * i for i in range(c.kv.shape[0])], np.int32)
    view = pool.view(torch.uint8 if fp8 else torch.int16).view(pages, stride)
    for i, p in enumerate(far):
        view[int(p), :2 * Hkv * page * D] = up(c.kv[i] if fp8 else c.kv[i].view(np.int16)).reshape(-1)
    for s, k in enumerate(kvs):
        n = -(-k // page)
        c.table[s, :n] = far[c.table[s, :n]]
    d = Dev(c)
    d.out.fill_(0x7FC1)
    d.lse.fill_(7.0)
    note(f"far pages fp8={fp8} pages={pages} stride={stride}")
    L.moe_tree_attention(d.q, c.q.shape[1], pool.data_ptr(), pool.data_ptr() + Hkv * page * D * es,
                         L.KV_E4M3 if fp8 else L.KV_BF16, d.ks if fp8 else None, d.vs if fp8 else None, pages, page, stride,
                         up(c.table), c.table.shape[1], d.cu, d.kvl, None, 2, c.T, 40, c.Hq, Hkv, D, D ** -0.5, 0.0, d.out,
                         d.lse, d.ws, d.ws_bytes)
    torch.cuda.synchronize()
    check(c, bits_of(d.out), d.lse.cpu().numpy(), [oracle.visible_tree(n, k, None) for n, k in zip(c.ns, kvs)], D ** -0.5, 0.0)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("which", ["tree", "prefill"])
def test_fewer_cached_tokens_than_queries(which, wide):
    """kv_lens below the query count: the first rows lie before the cache and see nothing."""
    ns, kvs = [6, 5, 70 if which == "prefill" else 50], [4, 0, 33]
    c = make_case(ns, kvs, 12, 1, 128, 16, False, seed=2)
    sees = []
    for n, k in zip(ns, kvs):
        sees.append(oracle.visible_tree(n, k, None) if which == "tree" else oracle.visible_prefill(n, k, 0))
    run_check(c, which, None, sees, wide=wide)


@pytest.mark.parametrize("which", ["tree", "prefill"])
def test_more_tokens_than_max_q(which):
    """Only the first max_q tokens of a sequence are computed, at their own places in the cache."""
    ns, kvs = [9, 40, 3], [50, 700, 3]
    c = make_case(ns, kvs, 12, 1, 128, 16, False, seed=2)
    sees = [oracle.visible_tree(n, k, None) for n, k in zip(ns, kvs)]
    d = Dev(c)
    d.max_q = 5
    d.ws_bytes = L.moe_attention_workspace_bytes(3, c.T, 5, c.Hq, c.Hkv, c.D)
    d.out.fill_(0x7FC1)
    d.lse.fill_(7.0)
    d.call(which)
    torch.cuda.synchronize()
    out, lse = bits_of(d.out).copy(), d.lse.cpu().numpy().copy()
    for s, n in enumerate(ns):
        a = int(c.cu_q[s])
        ref, rl, mag, _ = oracle.attend(c.q_heads(s)[:5], c.k[s], c.v[s], sees[s][:5], 128 ** -0.5)
        got = f32_from_bf16_bits(out[a:a + min(n, 5)].copy())
        assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -7 * mag)   # both roundings, and room for the sums
        assert np.all(out[a + 5:a + n] == 0x7FC1) and np.all(lse[a + 5:a + n] == 7.0)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("n", [1, 30])
@pytest.mark.parametrize("fp8", [False, True])
def test_a_nan_in_q_stays_in_its_row(fp8, n, wide):
    """Whole segments and split ones: the row's out and lse are NaN, the other rows within the bars."""
    c = make_case([n, n], [700, 3000], 12, 1, 128, 16, fp8, seed=4)
    sees = [oracle.visible_tree(n, k, None) for k in c.kvs]
    clean = run_check(c, "tree", None, sees, wide=wide)
    tok, head = 2 * n - 1, 5
    row, row_lse = clean.out[tok, head].clone(), clean.lse[tok, head].clone()
    d = Dev(c)
    d.out.fill_(0x7FC1)
    d.lse.fill_(7.0)
    d.q[tok, head * 128 + 77] = 0x7FC1
    d.call("tree")
    torch.cuda.synchronize()
    assert bool(d.out[tok, head].view(torch.bfloat16).isnan().all()) and bool(d.lse[tok, head].isnan())
    d.out[tok, head], d.lse[tok, head] = row, row_lse
    check(c, bits_of(d.out), d.lse.cpu().numpy(), sees, 128 ** -0.5, 0.0)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("n", [1, 30])
@pytest.mark.parametrize("fp8", [False, True])
def test_pages_outside_the_pool_are_unseen(fp8, n, wide):
    c = make_case([n, n], [200, 90], 12, 1, 128, 16, fp8, seed=3)
    c.table[0, 2], c.table[0, 7], c.table[1, 0] = -1, c.kv.shape[0], 2 ** 31 - 1
    see = [oracle.visible_tree(n, k, None) for k in c.kvs]
    see[0][:, 32:48] = see[0][:, 112:128] = False
    see[1][:, :16] = False
    run_check(c, "tree", None, see, wide=wide)


@pytest.mark.parametrize("fp8", [False, True])
def test_long_cache(fp8):
    """One long sequence (its keys split over the whole card) beside short ones, and many heads."""
    ns, kvs = [1, 1, 1], [70001, 3, 5000]
    c = make_case(ns, kvs, 12, 1, 128, 16, fp8, seed=4)
    run_check(c, "tree", None, [oracle.visible_tree(1, k, None) for k in kvs])


@pytest.mark.parametrize("wide", [False, True])
def test_many_sequences(wide):
    rng = np.random.default_rng(0)
    kvs = [int(x) for x in rng.integers(1, 60, 700)]
    c = make_case([1] * 700, kvs, 4, 2, 64, 16, False, seed=6)
    run_check(c, "tree", None, [oracle.visible_tree(1, k, None) for k in kvs], wide=wide)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 20])
def test_thousands_of_sequences(n, fp8):
    """More sequences than threads, some without tokens: every part finds its own among them."""
    rng = np.random.default_rng(1)
    ns = [int(x) for x in rng.integers(0, n + 1, 5000)]
    kvs = [int(x) for x in rng.integers(0, 40, 5000)]
    c = make_case(ns, kvs, 2, 1, 64, 16, fp8, seed=7)
    run_check(c, "tree", None, [oracle.visible_tree(a, k, None) for a, k in zip(ns, kvs)])


def test_same_bits_every_time():
    for which, ns, kvs in (("tree", [1] * 5, [40000, 3, 999, 2000, 17]), ("tree", [40, 64], [3000, 64]),
                           ("prefill", [700, 100], [900, 2000])):
        d = Dev(make_case(ns, kvs, 12, 1, 128, 16, False, seed=8))
        got = []
        for r in range(4):
            d.ws.fill_(0xFF if r % 2 else 0)
            d.call(which)
            torch.cuda.synchronize()
            got.append((bits_of(d.out).copy(), d.lse.cpu().numpy().copy()))
        assert all(np.array_equal(g[0], got[0][0]) and np.array_equal(g[1], got[0][1]) for g in got)


@pytest.mark.parametrize("which", ["tree", "prefill"])
def test_graph_replays_match_eager(which):
    """Captured once; replayed on other lengths, tables and values than at capture, with eager calls between."""
    n = 1 if which == "tree" else 90
    cases = [make_case([n] * 3, kvs, 12, 1, 128, 16, False, seed=s, extra_pages=300 - sum(-(-k // 16) for k in kvs))
             for s, kvs in enumerate(([100, 900, 95], [1000, 95, 333], [91, 92, 2000]))]
    for c in cases:
        t = np.zeros((3, 130), np.int32)
        t[:, :c.table.shape[1]] = c.table
        c.table = t
    devs = [Dev(c) for c in cases]
    eager = []
    for d in devs:
        d.call(which)
        torch.cuda.synchronize()
        eager.append((bits_of(d.out).copy(), d.lse.cpu().numpy().copy()))
    g0 = Dev(cases[0])
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        g0.call(which, stream=s)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            g0.call(which, stream=s)
    for rep in range(6):
        i = rep % 3
        d = devs[i]
        for name in ("q", "kv", "table", "cu", "kvl"):
            getattr(g0, name).copy_(getattr(d, name))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(bits_of(g0.out), eager[i][0]) and np.array_equal(g0.lse.cpu().numpy(), eager[i][1]), rep
        d.call(which)
        torch.cuda.synchronize()
        assert np.array_equal(bits_of(d.out), eager[i][0])


def test_two_streams_with_their_own_workspaces():
    devs = [Dev(make_case([1, 1], kvs, 12, 1, 128, 16, False, seed=s)) for s, kvs in enumerate(([30000, 7], [9, 20000]))]
    want = []
    for d in devs:
        d.call("tree")
        torch.cuda.synchronize()
        want.append(bits_of(d.out).copy())
        d.out.zero_()
    streams = [torch.cuda.Stream() for _ in devs]
    torch.cuda.synchronize()
    for _ in range(5):
        for d, s in zip(devs, streams):
            d.call("tree", stream=s)
    torch.cuda.synchronize()
    for d, w in zip(devs, want):
        assert np.array_equal(bits_of(d.out), w)


@pytest.mark.parametrize("fp8", [False, True])
def test_cache_object_steps(fp8):
    """A prompt in two chunks, then a drafted tree, then single tokens, all through PagedKVCache: append, then attend; the
    attention is checked against the oracle on what the cache holds."""
    torch.manual_seed(0)
    Hq, Hkv, D, page = 12, 1, 128, 16
    S, max_pages = 2, 20
    sc = torch.full((Hkv,), 0.02, device=DEV)
    cache = PagedKVCache(S * max_pages + 3, page, Hkv, D, L.KV_E4M3 if fp8 else L.KV_BF16, sc if fp8 else None,
                         sc if fp8 else None, DEV)
    cache.kv.view(torch.uint8).fill_(0x7F)
    table = torch.randperm(S * max_pages + 3, device=DEV)[:S * max_pages].view(S, max_pages).int()
    cos_sin = torch.empty((1024, 64), device=DEV)
    L.moe_rope_cos_sin_table(cos_sin, 1024, 64, 1e4)
    w = torch.rand(D, device=DEV) + 0.5
    rng = np.random.default_rng(1)
    lens = [0, 0]
    for step, ns in enumerate([[100, 37], [80, 150], [9, 4], [1, 1], [1, 1]]):
        T = sum(ns)
        cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
        words = [random_tree(min(n, 64), rng) for n in ns]
        at = np.concatenate([lens[s] + np.arange(n) for s, n in enumerate(ns)])
        seq = np.repeat(np.arange(S), ns)
        pos = at if step != 2 else np.concatenate([[lens[s] + bin(int(x)).count("1") - 1 for x in words[s]] for s in range(S)])
        t_at, t_seq = up(at), up(seq)
        slots = (table[t_seq, t_at // page] * page + t_at % page).int()
        qkv = torch.randn((T, (Hq + 2 * Hkv) * D), device=DEV).bfloat16()
        q = cache.append(qkv, Hq, slots, up(pos.astype(np.int32)), cos_sin, True, w, w)
        lens = [a + n for a, n in zip(lens, ns)]
        kvl = up(np.array(lens, np.int32))
        lse = torch.empty((T, Hq), device=DEV)
        note(f"cache object step {step} ns={ns} lens={lens} fp8={fp8}")
        if step < 2:
            out = cache.prefill_attention(q, table, up(cu), kvl, max(ns), lse=lse)
            sees = [oracle.visible_prefill(n, k, 0) for n, k in zip(ns, lens)]
        else:
            mask = up(np.concatenate(words).view(np.int64)) if step == 2 else None
            out = cache.tree_attention(q, table, up(cu), kvl, max(ns), mask, lse=lse)
            sees = [oracle.visible_tree(n, k, words[s] if step == 2 else None) for s, (n, k) in enumerate(zip(ns, lens))]
        torch.cuda.synchronize()
        c = make_case(ns, lens, Hq, Hkv, D, page, False, 0)
        c.fp8, c.q, c.T = fp8, bits_of(q.view(torch.int16)).reshape(T, -1), T
        val = cache.kv.float() * (0.02 if fp8 else 1.0)
        for s in range(S):
            pages = table[s, :-(-lens[s] // page)].long()
            both = val[pages].permute(1, 0, 3, 2, 4).reshape(2, -1, Hkv, D)[:, :lens[s]].double().cpu().numpy()
            c.k[s], c.v[s] = both[0], both[1]
        check(c, bits_of(out.view(torch.int16)), lse.cpu().numpy(), sees, D ** -0.5, 0.0)
