"""moe_kv_evict against a sort: kept places, lengths, usage and every byte of the cache exactly."""
import numpy as np
import pytest
import torch

import oracle
from shared_routed_expert_amd import PagedKVCache, _lib as L
from tests.gpu_util import note, DEV
from tests.test_gpu_attention import up

pytestmark = pytest.mark.gpu

GUARD = -77


class Cut:
    """Random bytes in a pool, a table over it, usage, and the new pages."""

    def __init__(self, kvs, budget, Hkv=2, D=64, page=16, fp8=False, seed=0, rows=None, num_rows=None, extra=0):
        rng = np.random.default_rng(seed)
        self.rng, self.kvs, self.budget, self.Hkv, self.D, self.page, self.fp8 = rng, kvs, budget, Hkv, D, page, fp8
        S = len(kvs)
        need = [-(-k // page) for k in kvs]
        new = -(-budget // page)
        width = max(max(need), 1) + extra
        pages = sum(need) + S * new + 3
        order = rng.permutation(pages).astype(np.int32)
        self.table = np.full((S, width), 1 << 30, np.int32)
        at = 0
        for s, k in enumerate(need):
            self.table[s, :k] = order[at:at + k]
            at += k
        self.new_table = order[at:at + S * new].reshape(S, new).copy()
        self.kv = rng.integers(0, 256, (pages, 2, Hkv, page, D * (1 if fp8 else 2)), dtype=np.uint8)
        self.rows, self.num_rows = rows, num_rows or S
        self.usage = np.exp(2 * rng.standard_normal((self.num_rows, Hkv, width * page))).astype(np.float32)

    def run(self, limit, sinks, recent, in_place=True, stream=None, wait=True):
        self.limit, self.sinks, self.recent = limit, sinks, recent
        S, kv = len(self.kvs), up(self.kv)
        if not self.fp8:
            kv = kv.view(torch.bfloat16)
        self.d_kv, self.d_usage = kv, up(self.usage)
        self.d_new = self.d_usage if in_place else torch.full_like(self.d_usage, GUARD)
        self.d_lens = torch.full((S + 4,), GUARD, dtype=torch.int32, device=DEV)
        self.d_kept = torch.full((S + 1, self.Hkv, self.budget), GUARD, dtype=torch.int32, device=DEV)
        note(f"evict kvs={self.kvs[:6]} S={S} limit={limit} budget={self.budget} sinks={sinks} recent={recent} Hkv={self.Hkv} "
             f"D={self.D} page={self.page} fp8={self.fp8} in_place={in_place}")
        L.moe_kv_evict(kv[:, 0], kv[:, 1], L.KV_E4M3 if self.fp8 else L.KV_BF16, kv.shape[0], self.page, kv.stride(0),
                       up(self.table), self.table.shape[1], up(np.array(self.kvs, np.int32)), self.d_usage, self.d_new,
                       None if self.rows is None else up(np.array(self.rows, np.int32)), self.num_rows, S, self.Hkv, self.D,
                       limit, self.budget, sinks, recent, up(self.new_table), self.new_table.shape[1], self.d_lens,
                       self.d_kept, stream)
        torch.cuda.synchronize()
        return self.check(in_place)

    def check(self, in_place):
        S, page, budget = len(self.kvs), self.page, self.budget
        pool = self.kv.shape[0]
        kv = self.kv.copy()
        usage = self.usage.copy() if in_place else np.full_like(self.usage, GUARD)
        kept = np.full((S + 1, self.Hkv, budget), GUARD, np.int32)
        lens = np.full(S + 4, GUARD, np.int32)
        for s, n in enumerate(self.kvs):
            n = min(n, self.table.shape[1] * page)
            lens[s] = budget if n > self.limit else n
            if n <= self.limit:
                continue
            row = s if self.rows is None else self.rows[s]
            known = 0 <= row < self.num_rows
            for h in range(self.Hkv):
                k = oracle.kept_tokens(self.usage[row, h] if known else np.zeros(n), n, budget, self.sinks, self.recent)
                assert len(k) == budget
                kept[s, h] = k
                if known:
                    usage[row, h, :budget] = self.usage[row, h, k]
                for i, j in enumerate(k):
                    src, dst = self.table[s, j // page], self.new_table[s, i // page]
                    if 0 <= dst < pool:
                        kv[dst, :, h, i % page] = self.kv[src, :, h, j % page] if 0 <= src < pool else 0
        assert np.array_equal(self.d_lens.cpu().numpy(), lens)
        assert np.array_equal(self.d_kept.cpu().numpy(), kept)
        assert np.array_equal(self.d_new.cpu().numpy(), usage, equal_nan=True)
        assert np.array_equal(self.d_kv.view(torch.uint8).cpu().numpy(), kv)
        if not in_place:
            assert np.array_equal(self.d_usage.cpu().numpy(), self.usage, equal_nan=True)
        return self


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_sizes(D, fp8, in_place):
    kvs = [1, 16, 17, 40, 41, 63, 64, 65, 100, 255, 256, 257, 1000, 0]
    Cut(kvs, 40, 2, D, 16, fp8, seed=D).run(40, 4, 8, in_place)
    Cut(kvs, 33, 1, D, 32, fp8, seed=D).run(60, 0, 0, in_place)


@pytest.mark.parametrize("budget,limit,sinks,recent", [(1, 1, 0, 0), (1, 1, 1, 0), (1, 1, 0, 1), (2, 5, 1, 1), (64, 64, 64, 0),
                                                       (64, 100, 0, 64), (100, 100, 30, 70), (17, 17, 3, 4), (299, 299, 1, 1),
                                                       (128, 200, 16, 16)])
def test_budgets(budget, limit, sinks, recent):
    for in_place in (False, True):
        Cut([300, limit, limit + 1, 290, 301], budget, 3, 64, 16, seed=budget).run(limit, sinks, recent, in_place)


@pytest.mark.parametrize("n,budget", [(5000, 4096), (5000, 100), (20000, 6000), (70000, 1000), (70000, 30000), (4200, 4100),
                                      (8192, 8191)])
def test_long(n, budget):
    for in_place in (False, True):
        Cut([n, 7, n - 3], budget, 1, 64, 64, fp8=True, seed=n).run(budget, 4, 50, in_place)


@pytest.mark.parametrize("kind", ["zeros", "two values", "few values", "near", "signs", "special", "descending", "ascending",
                                  "subnormal"])
def test_values(kind):
    """Ties, values that differ in their last bits alone, negative ones, both zeros, infinities and NaN."""
    for n, budget in ((900, 300), (9000, 2000)):
        c = Cut([n, n - 7], budget, 2, 64, 16, seed=3, extra=2)
        u, rng = c.usage, c.rng
        if kind == "zeros":
            u[:] = 0
        elif kind == "two values":
            u[:] = rng.choice(np.float32([0.25, 1.5]), u.shape)
        elif kind == "few values":
            u[:] = rng.choice(np.float32([0, 1e-20, 1, 1.0000001, 3]), u.shape, p=[0.4, 0.3, 0.1, 0.1, 0.1])
        elif kind == "near":
            u[:] = (np.float32(1.0).view(np.int32) + rng.integers(0, 700, u.shape).astype(np.int32)).view(np.float32)
        elif kind == "signs":
            u *= rng.choice(np.float32([-1, 1]), u.shape)
        elif kind == "special":
            pick = rng.integers(0, 8, u.shape)
            for i, v in enumerate([np.inf, -np.inf, np.nan, 0.0, -0.0]):
                u[pick == i] = v
        elif kind == "descending":
            u[:] = np.arange(u.shape[2], 0, -1, dtype=np.float32)
        elif kind == "ascending":
            u[:] = np.arange(u.shape[2], dtype=np.float32)
        else:
            u[:] = rng.integers(0, 50, u.shape).astype(np.int32).view(np.float32)
        for in_place in (False, True):
            c.run(budget, 4, 9, in_place)


@pytest.mark.parametrize("n", [61, 1001, 33001])
@pytest.mark.parametrize("kind", ["leading bits", "more bits", "all NaN", "NaN and lowest", "no choice"])
def test_whole_bins_kept(n, kind):
    """The kept are all values that share their leading bits, or reach into the lowest there are, or are the protected alone."""
    rng = np.random.default_rng(n)
    few = n // 5
    c = Cut([n], few + 4, 1, 64, 16, seed=n)
    row = c.usage[0, 0]
    row[:] = rng.uniform(0.001, 0.002, row.size)
    chosen = rng.permutation(np.arange(1, n - 3))[:few]
    if kind == "leading bits":      # one exponent, above the others
        row[chosen] = rng.uniform(1.0, 1.1, few)
    elif kind == "more bits":       # values that differ in their last ten bits alone
        row[:] = 1.0
        row[chosen] = (np.float32(1.5).view(np.uint32) + rng.integers(0, 1024, few).astype(np.uint32)).view(np.float32)
    elif kind == "all NaN":
        row[:] = np.nan
    elif kind == "NaN and lowest":  # some NaN are kept, the earlier ones
        row[:] = np.nan
        row[chosen[:few // 2]] = np.where(np.arange(few // 2) % 2 == 0, -np.inf, -np.finfo(np.float32).max)
    for in_place in (False, True):
        if kind == "no choice":
            c.run(few + 4, few, 4, in_place)
        else:
            c.run(few + 4, 1, 3, in_place)
            if kind in ("leading bits", "more bits"):
                assert set(c.d_kept[0, 0].tolist()) == {0, n - 3, n - 2, n - 1} | set(chosen.tolist())


def test_negative_zero_is_zero():
    """-0 and 0 are equal: the earlier is kept."""
    c = Cut([100], 10, 1, 64, 16)
    c.usage[:] = np.where(np.arange(c.usage.shape[2]) % 2 == 0, np.float32(-0.0), np.float32(0.0))
    c.run(10, 0, 0)
    assert c.d_kept[0, 0].tolist() == list(range(10))


def test_rows_and_bad_pages():
    c = Cut([200, 300, 250, 90, 400], 64, 2, 128, 16, seed=5, rows=[6, 1, -1, 2, 7], num_rows=7)
    c.table[0, 0], c.table[1, 3], c.table[4, 24] = -1, c.kv.shape[0], 2 ** 31 - 1
    c.new_table[1, 1] = -1
    for in_place in (False, True):
        c.run(100, 5, 6, in_place)


def test_lengths_past_the_table():
    c = Cut([100, 50], 32, 1, 64, 16, seed=6)
    c.kvs = [10 ** 6, 50]
    c.table[:] = c.rng.permutation(c.kv.shape[0])[:c.table.size].reshape(c.table.shape)
    new = [p for p in range(c.kv.shape[0]) if p not in set(c.table.flatten().tolist())]
    c.new_table = np.array(new[:4], np.int32).reshape(2, 2)
    c.run(32, 2, 3)


@pytest.mark.parametrize("Hkv,D,fp8", [(1, 128, False), (8, 128, True), (2, 256, False)])
def test_many_sequences(Hkv, D, fp8):
    rng = np.random.default_rng(8)
    kvs = [int(x) for x in rng.integers(0, 400, 300)]
    Cut(kvs, 96, Hkv, D, 32, fp8, seed=9).run(128, 4, 30)


def test_shared_pages_stay_whole():
    """Two sequences that share their first pages are both cut; what they shared is as it was."""
    c = Cut([256, 256, 256], 64, 2, 64, 16, seed=10)
    c.table[1, :8] = c.table[0, :8]
    c.run(64, 4, 8)


def test_graph_replays_match_eager():
    cuts = [Cut([900, 100, n], 256, 2, 64, 16, seed=n, extra=60 - (n - 900) // 16) for n in (900, 1300, 1700)]
    pages = max(c.kv.shape[0] for c in cuts)
    for c in cuts:
        c.kv = np.concatenate([c.kv, c.rng.integers(0, 256, (pages - c.kv.shape[0],) + c.kv.shape[1:], dtype=np.uint8)])
        w = max(x.table.shape[1] for x in cuts)
        t = np.full((3, w), 1 << 30, np.int32)
        t[:, :c.table.shape[1]] = c.table
        c.table = t
        c.usage = np.exp(c.rng.standard_normal((3, 2, w * 16))).astype(np.float32)
        c.run(256, 4, 16, False)
    c0 = cuts[0]
    names = ("kv", "table", "lens", "usage", "new_table")
    host = lambda c: dict(zip(names, (c.kv, c.table, np.array(c.kvs, np.int32), c.usage, c.new_table)))
    buf = {k: up(v) for k, v in host(c0).items()}
    kv = buf["kv"].view(torch.bfloat16)
    new_usage, lens = torch.empty_like(buf["usage"]), torch.empty(3, dtype=torch.int32, device=DEV)
    kept = torch.empty((3, 2, 256), dtype=torch.int32, device=DEV)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()

    def call():
        L.moe_kv_evict(kv[:, 0], kv[:, 1], L.KV_BF16, kv.shape[0], 16, kv.stride(0), buf["table"], buf["table"].shape[1],
                       buf["lens"], buf["usage"], new_usage, None, 3, 3, 2, 64, 256, 256, 4, 16, buf["new_table"],
                       buf["new_table"].shape[1], lens, kept, stream)

    with torch.cuda.stream(stream):
        call()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            call()
    for rep in range(6):
        c = cuts[rep % 3]
        for k, v in host(c).items():
            buf[k].copy_(up(v))
        new_usage.fill_(GUARD)
        kept.fill_(GUARD)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, want in ((buf["kv"], c.d_kv.view(torch.uint8)), (new_usage, c.d_new), (lens, c.d_lens[:3]), (kept, c.d_kept[:3])):
            assert torch.equal(got, want), rep


@pytest.mark.parametrize("at", [1, 2, 3])
def test_new_pages_from_a_slice(at):
    """new_table may begin at any element of a list of free pages."""
    c = Cut([300, 40], 64, 2, 128, 16, seed=12)
    free = up(np.concatenate([np.full(at, -1, np.int32), c.new_table.flatten()]))
    cache = PagedKVCache(c.kv.shape[0], 16, 2, 128, device=DEV)
    cache.kv.copy_(up(c.kv).view(torch.bfloat16))
    c.limit, c.sinks, c.recent = 64, 0, 1
    c.d_kv, c.d_usage = cache.kv, up(c.usage)
    c.d_new = torch.full_like(c.d_usage, GUARD)
    lens, kept = cache.evict(up(c.table), up(np.array(c.kvs, np.int32)), c.d_usage, free[at:].view(2, 4), 64, recent=1,
                             new_usage=c.d_new)
    kept[1] = GUARD
    c.d_kept = torch.cat([kept, torch.full((1, 2, 64), GUARD, dtype=torch.int32, device=DEV)])
    c.d_lens = torch.cat([lens, torch.full((4,), GUARD, dtype=torch.int32, device=DEV)])
    c.check(False)


def test_cache_object():
    c = Cut([300, 40], 64, 2, 128, 16, seed=12)
    cache = PagedKVCache(c.kv.shape[0], 16, 2, 128, device=DEV)
    cache.kv.copy_(up(c.kv).view(torch.bfloat16))
    usage = up(c.usage)
    lens, kept = cache.evict(up(c.table), up(np.array(c.kvs, np.int32)), usage, up(c.new_table), 64, sinks=4, recent=16)
    torch.cuda.synchronize()
    c.limit, c.sinks, c.recent = 64, 4, 16
    c.d_kv, c.d_usage, c.d_new = cache.kv, usage, usage
    assert kept[1].eq(-1).all()
    kept[1] = GUARD
    pad = torch.full((1, 2, 64), GUARD, dtype=torch.int32, device=DEV)
    c.d_kept = torch.cat([kept, pad])
    c.d_lens = torch.cat([lens, torch.full((4,), GUARD, dtype=torch.int32, device=DEV)])
    c.check(True)


@pytest.mark.parametrize("n", [3000, 40000])
def test_two_sequences_of_one_row(n):
    """What they keep is undefined where the row is compacted in place; nothing else is touched."""
    class Twice(Cut):
        def check(self, in_place):
            assert self.d_lens.tolist() == [self.budget] * 2 + [n // 4] + [GUARD] * 4
            kept = self.d_kept.cpu().numpy()
            assert (kept[2:] == GUARD).all()
            usage = self.d_usage.cpu().numpy()
            assert np.array_equal(usage[0, :, n:], self.usage[0, :, n:]) and np.array_equal(usage[1], self.usage[1])
            kv = self.d_kv.view(torch.uint8).cpu().numpy()
            new = set(self.new_table[:2].ravel().tolist())
            same = [p for p in range(len(kv)) if p not in new]
            assert np.array_equal(kv[same], self.kv[same])
            assert ((kept[:2] >= -1) & (kept[:2] < n) | (kept[:2] == GUARD)).all()
    Twice([n, n, n // 4], n // 4, 2, 64, 64, fp8=True, seed=n, rows=[0, 0, 1], num_rows=2).run(n // 4, 4, 50)
