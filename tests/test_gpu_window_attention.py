"""moe_window_attention against the float64 oracle on the same cached values, with the bars of test_gpu_attention (the same
products, softmax and sums over fewer keys).

In every case the cache holds NaN patterns in all tokens that no query token sees, and the block table holds entries outside
the pool, or of other sequences' pages, for the pages without a token that is seen.
"""
import numpy as np
import pytest
import torch

import oracle
from shared_routed_expert_amd import PagedKVCache, _lib as L
from tests.gpu_util import note, DEV
from tests.kv_util import NAN_BF16, NAN_E4M3, make_case
from tests.test_gpu_attention import Dev, bits_of, check, up

pytestmark = pytest.mark.gpu


def sees_of(c, window, sinks, max_q=None):
    return [oracle.visible_window(n, k, window, sinks) for n, k in zip(c.ns, c.kvs)]


def forget(c, sees, seed=0):
    """What nobody sees: NaN in the cache, anything in the table."""
    rng = np.random.default_rng(seed)
    for s, see in enumerate(sees):
        seen = see.any(axis=0) if len(see) else np.zeros(c.kvs[s], bool)
        for i in range(-(-c.kvs[s] // c.page)):
            part = seen[i * c.page:(i + 1) * c.page]
            page = c.table[s, i]
            c.kv[page, :, :, :len(part)][:, :, ~part] = NAN_E4M3 if c.fp8 else NAN_BF16
            if not part.any():
                c.table[s, i] = rng.choice([-1, 1 << 30, c.kv.shape[0], int(rng.integers(0, c.kv.shape[0]))])


class WinDev(Dev):
    def run(self, window, sinks, scale=None, cap=0.0, lse=True, stream=None):
        c = self.c
        L.moe_window_attention(
            self.q, c.q.shape[1], self.kv[:, 0], self.kv[:, 1], L.KV_E4M3 if c.fp8 else L.KV_BF16,
            self.ks if c.fp8 else None, self.vs if c.fp8 else None, c.kv.shape[0], c.page, self.kv.stride(0), self.table,
            c.table.shape[1], self.cu, self.kvl, window, sinks, len(c.ns), c.T, self.max_q, c.Hq, c.Hkv, c.D,
            c.D ** -0.5 if scale is None else scale, cap, self.out, self.lse if lse else None, self.ws, self.ws_bytes, stream)


def run_check(c, window, sinks, scale=None, cap=0.0, lse=True, wide=False, sees=None):
    sees = sees_of(c, window, sinks) if sees is None else sees
    forget(c, sees)
    if wide:
        t = np.full((c.table.shape[0], 131072 // c.page), 1 << 30, np.int32)
        t[:, :c.table.shape[1]] = c.table
        c.table = t
    d = WinDev(c)
    d.out.fill_(0x7FC1)
    d.lse.fill_(7.0)
    note(f"window {window} sinks {sinks} ns={c.ns[:6]} kvs={c.kvs[:6]} S={len(c.ns)} Hq={c.Hq} Hkv={c.Hkv} D={c.D} "
         f"page={c.page} fp8={c.fp8} cap={cap} wide={wide}")
    d.run(window, sinks, scale, cap, lse)
    torch.cuda.synchronize()
    assert bool((d.ws[d.ws_bytes:] == 0xCD).all())
    w = check(c, bits_of(d.out), d.lse.cpu().numpy() if lse else None, sees, c.D ** -0.5 if scale is None else scale, cap)
    note(f"  largest error / bound {w:.3f}")
    return d


HEADS = [(12, 1, 128), (96, 8, 128), (8, 2, 64), (7, 1, 64), (8, 1, 256), (128, 1, 64), (40, 1, 128)]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_single_tokens(Hq, Hkv, D, fp8, wide):
    """One token per sequence: windows that begin before the cache, at its start, inside tiles and pages, far behind."""
    kvs = [1, 2, 63, 64, 65, 127, 128, 129, 193, 200, 256, 321, 1000, 2049]
    for window, sinks in ((100, 4), (1, 0), (64, 64), (65, 1)):
        run_check(make_case([1] * len(kvs), kvs, Hq, Hkv, D, 16, fp8, seed=Hq + D), window, sinks, wide=wide)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_chunks(Hq, Hkv, D, fp8, wide):
    """Chunks shorter and longer than the window, with and without cached tokens before them, one of them empty."""
    ns, kvs = [130, 0, 33, 70, 1], [130, 50, 700, 90, 300]
    for window, sinks in ((50, 4), (200, 70), (1, 1)):
        run_check(make_case(ns, kvs, Hq, Hkv, D, 32, fp8, seed=Hq + D + 1, lead=2, tail=3), window, sinks, wide=wide)


@pytest.mark.parametrize("page", [16, 64, 1024])
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 3), (15, 16), (16, 17), (31, 0), (33, 128), (63, 200), (300, 500),
                                          (1000, 0), (1 << 30, 0), (2 ** 31 - 1, 2 ** 31 - 1), (1, 2 ** 31 - 1)])
@pytest.mark.parametrize("n", [1, 2, 40])
def test_windows_and_pages(window, sinks, page, n):
    kvs = [n, n + 1, n + 47, 400 + n, 1300]
    run_check(make_case([n] * len(kvs), kvs, 12, 1, 128, page, False, seed=window % 1000), window, sinks)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("cap", [0.0, 5.0, 100.0])
@pytest.mark.parametrize("n", [1, 90])
def test_cap_stride_and_no_lse(n, cap, fp8):
    c = make_case([n, n], [500, 77 + n], 16, 4, 128, 16, fp8, seed=5, q_extra=24, big=3.0)
    run_check(c, 130, 5, scale=0.3, cap=cap, lse=False)


def test_tokens_past_max_q_and_more_tokens_than_cached():
    """max_q cuts a sequence's tokens; where a sequence has more query tokens than cached ones, the first see nothing."""
    c = make_case([9, 5], [300, 200], 12, 1, 128, 16, False, seed=9)
    sees = sees_of(c, 40, 3)
    d = WinDev(c)
    d.max_q = 6
    d.out.fill_(0x7FC1)
    d.lse.fill_(7.0)
    note("window, tokens past max_q")
    d.run(40, 3)
    torch.cuda.synchronize()
    out, lse = bits_of(d.out), d.lse.cpu().numpy()
    assert np.all(out[6:9] == 0x7FC1) and np.all(lse[6:9] == 7.0)
    e = make_case([6, 3, 5], [297, 300, 200], 12, 1, 128, 16, False, seed=9)
    e.ns, e.T = [6, 5], 11
    e.k, e.v = c.k, c.v
    e.kvs = c.kvs
    e.q = np.concatenate([c.q[:6], c.q[9:]])
    e.cu_q = np.array([0, 6, 11], np.int32)
    check(e, np.concatenate([out[:6], out[9:]]), np.concatenate([lse[:6], lse[9:]]), [sees[0][:6], sees[1]], 128 ** -0.5, 0.0)
    for n in (12, 100):
        c = make_case([n, 3], [7, 50], 12, 1, 128, 16, False, seed=4)
        run_check(c, 5, 2)


@pytest.mark.parametrize("n", [1, 30])
def test_pages_outside_the_pool_are_unseen(n):
    c = make_case([n, n], [400, 190], 12, 1, 128, 16, False, seed=3)
    sees = sees_of(c, 100, 20)
    c.table[0, 0], c.table[0, 22], c.table[1, 8] = -1, c.kv.shape[0], 2 ** 31 - 1
    sees[0][:, :16] = sees[0][:, 352:368] = False
    sees[1][:, 128:144] = False
    d = WinDev(c)
    d.out.fill_(0x7FC1)
    d.lse.fill_(7.0)
    note("window, pages outside the pool")
    d.run(100, 20)
    torch.cuda.synchronize()
    check(c, bits_of(d.out), d.lse.cpu().numpy(), sees, 128 ** -0.5, 0.0)


@pytest.mark.parametrize("n,window", [(1, 4096), (1, 60000), (9, 5000), (2, 20000)])
@pytest.mark.parametrize("fp8", [False, True])
def test_long_caches(n, window, fp8):
    """Windows split over many parts, beside short sequences."""
    run_check(make_case([n] * 3, [70001, n + 3, 9000], 12, 1, 128, 16, fp8, seed=4), window, 4)


@pytest.mark.parametrize("n", [1, 20])
def test_thousands_of_sequences(n):
    rng = np.random.default_rng(1)
    ns = [int(x) for x in rng.integers(0, n + 1, 5000)]
    kvs = [int(x) for x in rng.integers(0, 90, 5000)]
    run_check(make_case(ns, kvs, 2, 1, 64, 16, False, seed=7), 17, 3)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_long_prompt(fp8):
    """Whole segments (many row tiles) and parts of them: some of a longer prompt's rows against the oracle."""
    for wide in (False, True):
        c = make_case([1500, 40], [2600, 500], 12, 1, 128, 64, fp8, seed=11)
        run_check(c, 700, 33, wide=wide)


def test_a_window_over_everything_is_the_causal_call():
    """With no token left out, the bits are those of moe_prefill_attention on the same parts of the keys."""
    c = make_case([70, 5], [500, 300], 12, 1, 128, 16, False, seed=13)
    d = WinDev(c)
    d.run(1 << 20, 0)
    torch.cuda.synchronize()
    a = f32(bits_of(d.out))
    d.call("prefill")
    torch.cuda.synchronize()
    b = f32(bits_of(d.out))
    # each within 2^-8 of the exact value and of the mean of |v|, at most 5 here
    assert np.abs(a - b).max() <= 2 * (2.0 ** -8 * np.abs(b).max() + 2.0 ** -8 * 5)


def f32(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32)


def test_same_bits_every_time():
    for ns, kvs in (([1] * 5, [40000, 3, 999, 2000, 17]), ([700, 100], [900, 2000])):
        d = WinDev(make_case(ns, kvs, 12, 1, 128, 16, False, seed=8))
        got = []
        for r in range(4):
            d.ws.fill_(0xFF if r % 2 else 0)
            d.run(600, 4)
            torch.cuda.synchronize()
            got.append((bits_of(d.out).copy(), d.lse.cpu().numpy().copy()))
        assert all(np.array_equal(g[0], got[0][0]) and np.array_equal(g[1], got[0][1]) for g in got)


@pytest.mark.parametrize("n", [1, 90])
def test_graph_replays_match_eager(n):
    """Captured once, replayed on other lengths, tables and values, with eager calls between."""
    cases = [make_case([n] * 3, kvs, 12, 1, 128, 16, False, seed=s, extra_pages=300 - sum(-(-k // 16) for k in kvs))
             for s, kvs in enumerate(([100, 900, 95], [1000, 95, 333], [91, 92, 2000]))]
    for c in cases:
        t = np.zeros((3, 130), np.int32)
        t[:, :c.table.shape[1]] = c.table
        c.table = t
    devs = [WinDev(c) for c in cases]
    eager = []
    for d in devs:
        d.run(150, 4)
        torch.cuda.synchronize()
        eager.append((bits_of(d.out).copy(), d.lse.cpu().numpy().copy()))
    g0, s, g = WinDev(cases[0]), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        g0.run(150, 4, stream=s)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            g0.run(150, 4, stream=s)
    for rep in range(6):
        i = rep % 3
        d = devs[i]
        for name in ("q", "kv", "table", "cu", "kvl"):
            getattr(g0, name).copy_(getattr(d, name))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(bits_of(g0.out), eager[i][0]) and np.array_equal(g0.lse.cpu().numpy(), eager[i][1]), rep
        d.run(150, 4)
        torch.cuda.synchronize()
        assert np.array_equal(bits_of(d.out), eager[i][0])


def test_cache_object():
    c = make_case([20, 1], [300, 77], 12, 1, 128, 16, False, seed=21, tail=2)
    cache = PagedKVCache(c.kv.shape[0], 16, 1, 128, device=DEV)
    cache.kv.view(torch.int16).copy_(up(c.kv.view(np.int16)))
    q = up(c.q.view(np.int16)).view(torch.bfloat16).unflatten(1, (12, 128))
    lse = torch.full((c.T, 12), 7.0, device=DEV)
    note("window, PagedKVCache")
    out = cache.window_attention(q, up(c.table), up(c.cu_q), up(np.array(c.kvs, np.int32)), 20, 64, 4, lse=lse)
    torch.cuda.synchronize()
    check(c, bits_of(out.view(torch.int16)), lse.cpu().numpy(), sees_of(c, 64, 4), 128 ** -0.5, 0.0, guard=0)


@pytest.mark.parametrize("wide", [False, True])
def test_many_row_tiles_under_a_window_of_thousands(wide):
    """Thousands of segments of more than 4096 keys (the kernel looks at the lengths before it takes them whole): some of the
    tokens against the oracle."""
    n, kv, window = 3200, 6000, 4500
    c = make_case([n, 1], [kv, 100], 64, 1, 64, 64, False, seed=31)
    if wide:
        t = np.full((2, 131072 // c.page), 1 << 30, np.int32)
        t[:, :c.table.shape[1]] = c.table
        c.table = t
    d = WinDev(c)
    note(f"window {window}, {n} tokens of 64 heads, wide={wide}")
    d.run(window, 9)
    torch.cuda.synchronize()
    out, lse = bits_of(d.out), d.lse.cpu().numpy()
    rows = np.unique(np.concatenate([np.arange(0, n, 173), [1, 2, 3, n - 2, n - 1], np.arange(1500, 1520)]))
    see = oracle.visible_window(n, kv, window, 9)[rows]
    e = make_case([len(rows)], [kv], 64, 1, 64, 64, False, seed=31)
    e.q, e.k, e.v, e.T = c.q[rows], c.k[:1], c.v[:1], len(rows)
    check(e, out[rows], lse[rows], [see], 64 ** -0.5, 0.0)


def test_pages_that_the_window_leaves_are_given_away():
    """Decoding with a pool of few pages: each step appends a token, and a page that no later token will see goes back to
    the pool, from which the other sequence takes it; the attention against all that was ever appended."""
    Hq, Hkv, D, page, window, sinks = 8, 2, 64, 16, 40, 5
    rng = np.random.default_rng(2)
    cache = PagedKVCache(12, page, Hkv, D, device=DEV)
    cache.kv.view(torch.int16).fill_(0x7FC1)
    free = [int(x) for x in rng.permutation(12)]
    table = np.full((2, 16), -1, np.int32)
    owned = [[False] * 16 for _ in range(2)]
    k, v = [[], []], [[], []]
    for step in range(150):
        lens = [step + 1, step // 2 + 1]
        active = [0, 1] if step % 2 == 0 else [0]
        slots = []
        for s in active:
            at = lens[s] - 1
            if at % page == 0:
                table[s, at // page] = free.pop()
                owned[s][at // page] = True
            slots.append(int(table[s, at // page]) * page + at % page)
        qkv = torch.from_numpy(rng.standard_normal((len(active), (Hq + 2 * Hkv) * D)).astype(np.float32)).to(DEV).bfloat16()
        q = cache.append(qkv, Hq, up(np.array(slots, np.int32)))
        new = qkv.double().cpu().numpy().reshape(len(active), Hq + 2 * Hkv, D)
        for i, s in enumerate(active):
            k[s].append(new[i, Hq:Hq + Hkv])
            v[s].append(new[i, Hq + Hkv:])
        lse = torch.empty((len(active), Hq), device=DEV)
        out = cache.window_attention(q, up(table[active]), up(np.arange(len(active) + 1, dtype=np.int32)),
                                     up(np.array([lens[s] for s in active], np.int32)), 1, window, sinks, lse=lse)
        torch.cuda.synchronize()
        c = make_case([1] * len(active), [lens[s] for s in active], Hq, Hkv, D, page, False, 0)
        c.q, c.T = bits_of(q.view(torch.int16)).reshape(len(active), -1), len(active)
        c.k, c.v = [np.array(k[s]) for s in active], [np.array(v[s]) for s in active]
        check(c, bits_of(out.view(torch.int16)), lse.cpu().numpy(), sees_of(c, window, sinks), D ** -0.5, 0.0)
        for s in active:   # the next token sees from lens + 1 - window on
            for p in range(16):
                if owned[s][p] and p * page >= sinks and (p + 1) * page <= lens[s] + 1 - window:
                    free.append(int(table[s, p]))
                    owned[s][p] = False
                    table[s, p] = rng.choice([-1, 1 << 30, int(rng.integers(0, 12))])
