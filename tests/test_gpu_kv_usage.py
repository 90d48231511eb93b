"""moe_kv_usage against the float64 oracle on the same cached keys and the same lse.

Bar of one sum of N weights p with X their row's largest sum_d |q_d k_d| * scale:
  sum p (2 e + 2^-24 (N + 40)) + 2^-23 |decay prev| + N 2^-126,  e = 2^-24 ((D + 12) X + 16 softcap) the error of a score in
  float32 (products and their sum, scaling, the tanh of two exponentials and a quotient); N additions, the exponential, the split of
  lse; weights below float32's normal range may be lost. Everything that the call does not own keeps its bytes.
"""
import numpy as np
import pytest
import torch

import oracle
from shared_routed_expert_amd import PagedKVCache, _lib as L
from tests.gpu_util import note, DEV
from tests.kv_util import make_case
from tests.test_gpu_attention import up

pytestmark = pytest.mark.gpu

GUARD = 5.5


class UseDev:
    def __init__(self, c, lse, rows=None, num_rows=None, max_q=None):
        self.c = c
        S = len(c.ns)
        self.q = up(c.q.view(np.int16))
        self.kv = up(c.kv if c.fp8 else c.kv.view(np.int16))
        self.ks = up(c.scales[0].copy())
        self.table, self.cu, self.kvl = up(c.table), up(c.cu_q), up(np.array(c.kvs, np.int32))
        self.lse = up(lse)
        self.max_q = max_q or max(max(c.ns), 1)
        self.rows = None if rows is None else up(np.array(rows, np.int32))
        self.num_rows = num_rows or S
        self.tokens = c.table.shape[1] * c.page
        self.usage = torch.full((self.num_rows, c.Hkv, self.tokens), GUARD, device=DEV)
        self.ws_bytes = L.moe_kv_usage_workspace_bytes(S, c.T, self.max_q, c.Hq, c.Hkv, c.D)
        self.ws = torch.full((self.ws_bytes + 512,), 0xCD, dtype=torch.uint8, device=DEV)

    def call(self, prev=None, decay=1.0, prefix=None, scale=None, cap=0.0, stream=None):
        c = self.c
        L.moe_kv_usage(self.q, c.q.shape[1], self.kv[:, 0], L.KV_E4M3 if c.fp8 else L.KV_BF16, self.ks if c.fp8 else None,
                       c.kv.shape[0], c.page, self.kv.stride(0), self.table, c.table.shape[1], self.cu, self.kvl, prefix,
                       self.lse, len(c.ns), c.T, self.max_q, c.Hq, c.Hkv, c.D, c.D ** -0.5 if scale is None else scale, cap,
                       prev, decay, self.usage, self.rows, self.num_rows, self.ws, self.ws_bytes, stream)


def some_lse(c, sees, scale=None, cap=0.0, seed=0):
    """About what the attention gives, with noise: any lse is an input."""
    rng = np.random.default_rng(seed)
    lse = rng.standard_normal((c.T, c.Hq)).astype(np.float32)
    for s, n in enumerate(c.ns):
        a = int(c.cu_q[s])
        if n and c.kvs[s]:
            zero = np.zeros_like(c.k[s])
            _, l, _, _ = oracle.attend(c.q_heads(s), c.k[s], zero, sees[s], c.D ** -0.5 if scale is None else scale, cap)
            lse[a:a + n] = l + 0.3 * lse[a:a + n]
    return lse


def check(c, usage, lse, sees, scale, cap, prev=None, decay=1.0, rows=None, max_q=None, guard=None):
    guard = np.full_like(usage, GUARD) if guard is None else guard
    want_guard = np.ones(usage.shape, bool)
    worst = 0.0
    for s, n in enumerate(c.ns):
        row = s if rows is None else rows[s]
        if n == 0 or not 0 <= row < usage.shape[0]:
            continue
        a, kv = int(c.cu_q[s]), c.kvs[s]
        m = n if max_q is None else min(n, max_q)
        ref, spread = oracle.usage(c.q_heads(s)[:m], c.k[s], sees[s][:m], lse[a:a + m], scale, cap)
        N = m * (c.Hq // c.Hkv)
        bar = 2 * 2.0 ** -24 * ((c.D + 12) * spread + 16 * cap * ref) + 2.0 ** -24 * (N + 40) * ref + N * 2.0 ** -126
        if prev is not None:
            ctx = max(kv - n, 0)
            old = np.zeros_like(ref)
            old[:, :ctx] = decay * prev[row][:, :ctx].astype(np.float64)
            ref = ref + old
            bar = bar + 2.0 ** -23 * np.abs(old)
        got = usage[row][:, :kv].astype(np.float64)
        err = np.abs(got - ref)
        assert np.all(err <= bar), (s, np.argwhere(~(err <= bar))[:3], float(np.max(err / np.maximum(bar, 1e-300))))
        worst = max(worst, float(np.max(err / np.maximum(bar, 1e-300), initial=0)))
        want_guard[row, :, :kv] = False
    assert np.array_equal(usage[want_guard], guard[want_guard], equal_nan=True)
    return worst


def run_check(c, sees=None, prefix=None, scale=None, cap=0.0, prev=False, decay=1.0, rows=None, num_rows=None, lse=None, wide=False):
    if sees is None:
        sees = [oracle.visible_prefill(n, k, 0 if prefix is None else prefix[s]) for s, (n, k) in enumerate(zip(c.ns, c.kvs))]
    if lse is None:
        lse = some_lse(c, sees, scale, cap)
    if wide:
        t = np.full((c.table.shape[0], 32768 // c.page), 1 << 30, np.int32)
        t[:, :c.table.shape[1]] = c.table
        c.table = t
    d = UseDev(c, lse, rows, num_rows)
    note(f"usage ns={c.ns[:6]} kvs={c.kvs[:6]} S={len(c.ns)} Hq={c.Hq} Hkv={c.Hkv} D={c.D} page={c.page} fp8={c.fp8} cap={cap} "
         f"prev={prev} decay={decay} wide={wide}")
    old = None
    if prev:
        rng = np.random.default_rng(1)
        old = np.exp(2 * rng.standard_normal(d.usage.shape)).astype(np.float32)
        for s, (n, k) in enumerate(zip(c.ns, c.kvs)):   # what is not to be read
            row = s if rows is None else rows[s]
            if 0 <= row < d.num_rows:
                old[row, :, max(k - n, 0):] = np.nan
    d.call(None if old is None else up(old), decay, None if prefix is None else up(np.array(prefix, np.int32)), scale, cap)
    torch.cuda.synchronize()
    assert bool((d.ws[d.ws_bytes:] == 0xCD).all())
    w = check(c, d.usage.cpu().numpy(), lse, sees, c.D ** -0.5 if scale is None else scale, cap, old, decay, rows)
    note(f"  largest error / bound {w:.3f}")
    return d, lse, sees


HEADS = [(12, 1, 128), (96, 8, 128), (8, 2, 64), (7, 1, 64), (1, 1, 128), (8, 1, 256), (16, 2, 256), (128, 1, 64), (40, 1, 128),
         (33, 1, 64)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_single_tokens(Hq, Hkv, D, fp8):
    kvs = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 700]
    run_check(make_case([1] * len(kvs), kvs, Hq, Hkv, D, 16, fp8, seed=Hq + D), prev=True, decay=0.75)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_chunks(Hq, Hkv, D, fp8, wide):
    """Chunks with and without cached tokens before them, one of them empty, rows of q of no sequence."""
    c = make_case([130, 0, 33, 70, 1], [130, 50, 700, 90, 300], Hq, Hkv, D, 32, fp8, seed=Hq + D + 1, lead=2, tail=3, q_extra=16)
    run_check(c, prev=wide, wide=wide)


@pytest.mark.parametrize("page", [16, 64, 1024])
@pytest.mark.parametrize("n", [1, 2, 3, 31, 40, 300])
def test_lengths_and_pages(n, page):
    kvs = [n, n + 1, n + 47, 256 + n, 900, 257, 512]
    kvs = [max(k, n) for k in kvs]
    run_check(make_case([n] * len(kvs), kvs, 12, 1, 128, page, False, seed=n))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("cap", [5.0, 64.0, 100.0])
@pytest.mark.parametrize("n", [1, 90])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_caps(D, n, cap, fp8):
    run_check(make_case([n, n], [300, 77 + n], 16, 4, D, 16, fp8, seed=5, big=3.0), scale=0.3, cap=cap)


def test_prefixes():
    ns, kvs = [60, 60, 300, 5], [60, 500, 300, 700]
    run_check(make_case(ns, kvs, 12, 1, 128, 16, False, seed=6), prefix=[25, 480, 10000, 0], prev=True)
    run_check(make_case(ns, kvs, 12, 1, 128, 16, False, seed=6), prefix=[60, -5, 299, 699])


def test_rows_and_sequences_left_alone():
    """Sequences in rows of their own choice; rows outside leave nothing; more tokens than cached ones; tokens past max_q."""
    c = make_case([3, 1, 40, 1, 0], [100, 50, 60, 700, 33], 12, 1, 128, 16, False, seed=7)
    run_check(c, rows=[4, -1, 2, 1 << 30, 1], num_rows=6, prev=True)
    c = make_case([12, 100, 3], [7, 30, 50], 12, 1, 128, 16, False, seed=8)
    sees = [oracle.visible_prefill(n, k, 0) for n, k in zip(c.ns, c.kvs)]
    lse = some_lse(c, sees)
    assert np.isneginf(lse[:5]).all()
    run_check(c, sees=sees, lse=lse, prev=True)
    c = make_case([50, 9], [200, 300], 12, 1, 128, 16, False, seed=9)
    sees = [oracle.visible_prefill(n, k, 0) for n, k in zip(c.ns, c.kvs)]
    lse = some_lse(c, sees)
    d = UseDev(c, lse, max_q=6)
    d.call()
    torch.cuda.synchronize()
    check(c, d.usage.cpu().numpy(), lse, sees, 128 ** -0.5, 0.0, max_q=6)


@pytest.mark.parametrize("n", [1, 30])
def test_pages_outside_the_pool_get_nothing(n):
    c = make_case([n, n], [400, 190], 12, 1, 128, 16, False, seed=3)
    sees = [oracle.visible_prefill(n, k, 0) for k in c.kvs]
    lse = some_lse(c, sees)
    c.table[0, 0], c.table[0, 22], c.table[1, 8] = -1, c.kv.shape[0], 2 ** 31 - 1
    sees[0][:, :16] = sees[0][:, 352:368] = False
    sees[1][:, 128:144] = False
    run_check(c, sees=sees, lse=lse)


@pytest.mark.parametrize("n", [1, 2, 64])
@pytest.mark.parametrize("fp8", [False, True])
def test_long_cache(n, fp8):
    run_check(make_case([n] * 3, [70001, n + 3, 5000], 12, 1, 128, 16, fp8, seed=4), prev=True)


@pytest.mark.parametrize("n", [1, 20])
def test_thousands_of_sequences(n):
    rng = np.random.default_rng(1)
    ns = [int(x) for x in rng.integers(0, n + 1, 5000)]
    kvs = [max(a, int(x)) for a, x in zip(ns, rng.integers(0, 90, 5000))]
    run_check(make_case(ns, kvs, 2, 1, 64, 16, False, seed=7))


@pytest.mark.parametrize("Hq,Hkv,D", [(12, 1, 128), (16, 4, 128), (8, 1, 256)])
def test_a_long_prompt(Hq, Hkv, D):
    run_check(make_case([1500, 40], [2600, 500], Hq, Hkv, D, 64, False, seed=11))


def test_a_nan_row_stays_with_what_it_sees():
    """lse NaN in one row: NaN for the tokens it sees, in its kv head; a NaN in q the same."""
    for where in ("lse", "q"):
        c = make_case([60], [100], 8, 2, 64, 16, False, seed=12)
        sees = [oracle.visible_prefill(60, 100, 0)]
        lse = some_lse(c, sees)
        d, _, _ = run_check(c, sees=sees, lse=lse.copy())
        clean = d.usage.clone()
        if where == "lse":
            d.lse[20, 5] = float("nan")
        else:
            d.q[20, 5 * 64 + 3] = 0x7FC1
        d.usage.fill_(GUARD)
        d.call()
        torch.cuda.synchronize()
        got = d.usage.cpu().numpy()
        assert np.isnan(got[0, 1, :61]).all()
        got[0, 1, :61] = clean.cpu().numpy()[0, 1, :61]
        assert np.array_equal(got, clean.cpu().numpy())


def test_weights_of_the_attention_add_up():
    """With the attention's own lse each row's weights sum to 1, and so a kv head's usage to its rows."""
    c = make_case([200, 7], [900, 300], 12, 1, 128, 16, False, seed=14)
    cache = PagedKVCache(c.kv.shape[0], 16, 1, 128, device=DEV)
    cache.kv.view(torch.int16).copy_(up(c.kv.view(np.int16)))
    q = up(c.q.view(np.int16)).view(torch.bfloat16).unflatten(1, (12, 128))
    table, cu, kvl = up(c.table), up(c.cu_q), up(np.array(c.kvs, np.int32))
    lse = torch.empty((c.T, 12), device=DEV)
    cache.prefill_attention(q, table, cu, kvl, 200, lse=lse)
    u = cache.usage(q, table, cu, kvl, 200, lse, torch.zeros((2, 1, c.table.shape[1] * 16), device=DEV))
    torch.cuda.synchronize()
    total = u.double().sum(-1)[:, 0].cpu().numpy()
    # scores of up to about 8 in both calls: lse and weight within 2^-24 ((D + 12) X + kv + 64 + ..), X <= 30
    assert np.all(np.abs(total - np.array([200 * 12, 7 * 12])) <= np.array([200 * 12, 7 * 12]) * 2.0 ** -24 * (2 * 140 * 30 + 3600))


def test_in_place_and_same_bits_every_time():
    c = make_case([200, 1, 33], [900, 300, 33], 12, 1, 128, 16, False, seed=15)
    sees = [oracle.visible_prefill(n, k, 0) for n, k in zip(c.ns, c.kvs)]
    d = UseDev(c, some_lse(c, sees))
    prev = torch.rand(d.usage.shape, device=DEV)
    got = []
    for r in range(4):
        d.ws.fill_(0xFF if r % 2 else 0)
        if r < 2:
            d.usage.copy_(prev)
            d.call(d.usage, 0.5)
        else:
            d.usage.copy_(prev)
            d.call(prev, 0.5)
        torch.cuda.synchronize()
        got.append(d.usage.cpu().numpy().copy())
    assert all(np.array_equal(g, got[0]) for g in got)


@pytest.mark.parametrize("n", [1, 90])
def test_graph_replays_match_eager(n):
    cases = [make_case([n] * 3, kvs, 12, 1, 128, 16, False, seed=s, extra_pages=300 - sum(-(-k // 16) for k in kvs))
             for s, kvs in enumerate(([100, 900, 95], [1000, 95, 333], [91, 92, 2000]))]
    devs, eager = [], []
    for c in cases:
        t = np.zeros((3, 130), np.int32)
        t[:, :c.table.shape[1]] = c.table
        c.table = t
        d = UseDev(c, some_lse(c, [oracle.visible_prefill(n, k, 0) for k in c.kvs]))
        d.call()
        torch.cuda.synchronize()
        devs.append(d)
        eager.append(d.usage.cpu().numpy().copy())
    g0, s, g = UseDev(cases[0], devs[0].lse.cpu().numpy()), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        g0.call(stream=s)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            g0.call(stream=s)
    for rep in range(6):
        i = rep % 3
        d = devs[i]
        for name in ("q", "kv", "table", "cu", "kvl", "lse"):
            getattr(g0, name).copy_(getattr(d, name))
        g0.usage.fill_(GUARD)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(g0.usage.cpu().numpy(), eager[i]), rep
        d.call()
        torch.cuda.synchronize()
        assert np.array_equal(d.usage.cpu().numpy(), eager[i])


@pytest.mark.parametrize("Hq,Hkv,D", [(12, 1, 128), (16, 4, 64), (8, 1, 256)])
def test_rows_far_apart(Hq, Hkv, D):
    """q_stride of more than 2^22 values: the rows' places within a tile no longer fit 32 bits."""
    c = make_case([11, 5], [300, 40], Hq, Hkv, D, 16, False, seed=20)
    sees = [oracle.visible_prefill(n, k, 0) for n, k in zip(c.ns, c.kvs)]
    lse = some_lse(c, sees)
    d = UseDev(c, lse)
    stride = (1 << 22) + Hq * D + 8
    far = torch.full((c.T, stride), 0x7FC1, dtype=torch.int16, device=DEV)
    far[:, :Hq * D] = d.q
    d.q = far
    note(f"usage, rows {stride} values apart")
    L.moe_kv_usage(far, stride, d.kv[:, 0], L.KV_BF16, None, c.kv.shape[0], c.page, d.kv.stride(0), d.table, c.table.shape[1],
                   d.cu, d.kvl, None, d.lse, 2, c.T, d.max_q, Hq, Hkv, D, D ** -0.5, 0.0, None, 1.0, d.usage, None, 2, d.ws,
                   d.ws_bytes)
    torch.cuda.synchronize()
    check(c, d.usage.cpu().numpy(), lse, sees, D ** -0.5, 0.0)


def test_two_streams_with_their_own_workspaces():
    devs = []
    for seed, ns, kvs in ((1, [70, 5], [900, 30]), (2, [200, 1], [200, 2000]), (3, [1, 2], [5000, 9])):
        c = make_case(ns, kvs, 12, 1, 128, 16, False, seed=seed)
        devs.append(UseDev(c, some_lse(c, [oracle.visible_prefill(n, k, 0) for n, k in zip(ns, kvs)])))
    want = []
    for d in devs:
        d.call()
        torch.cuda.synchronize()
        want.append(d.usage.clone())
        d.usage.fill_(GUARD)
    streams = [torch.cuda.Stream() for _ in devs]
    torch.cuda.synchronize()
    for _ in range(4):
        for d, s in zip(devs, streams):
            d.call(stream=s)
    torch.cuda.synchronize()
    for d, w in zip(devs, want):
        assert torch.equal(d.usage, w)
