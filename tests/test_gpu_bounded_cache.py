"""A long generation in a bounded cache, as the operators are used together: a prompt's keys are appended and attended, their usage
noted, the sequences cut to a budget on new pages; then token by token append, attention, usage, a cut when a sequence has
outgrown its limit, and the norm and the expert layer behind the attention. Every step is checked against the oracle on
what the device held before it (bars of the operators' own tests); what a cut keeps is followed byte for byte."""
import numpy as np
import pytest
import torch

import oracle
from shared_routed_expert_amd import PagedKVCache, _lib as L
from tests.gpu_util import DEV, make_layer, note, small_cfg, to_dev
from tests.kv_util import make_case
from tests.test_gpu_add_rms_norm import check as check_norm
from tests.test_gpu_attention import bits_of, check as check_attention, up
from tests.test_gpu_kv_usage import check as check_usage
from workloads import generate

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
def test_generation(fp8):
    Hq, Hkv, D, page, S = 12, 2, 64, 16, 3
    budget, limit, sinks, recent, decay = 48, 60, 4, 10, 0.9
    pool, width = 40, 8
    rng = np.random.default_rng(3)
    sc = torch.full((Hkv,), 0.02, device=DEV)
    cache = PagedKVCache(pool, page, Hkv, D, L.KV_E4M3 if fp8 else L.KV_BF16, sc if fp8 else None, sc if fp8 else None, DEV)
    cache.kv.view(torch.uint8).fill_(0x7F)   # NaN wherever nothing has been appended
    free = [int(x) for x in rng.permutation(pool)]
    table = np.full((S, width), 1 << 30, np.int32)
    cos_sin = torch.empty((256, 32), device=DEV)
    L.moe_rope_cos_sin_table(cos_sin, 256, 32, 1e4)
    w = torch.rand(D, device=DEV) + 0.5
    # rows of usage that are not the sequences' numbers
    rows = up(np.array([4, 0, 3], np.int32))
    usage = torch.full((5, Hkv, width * page), float("nan"), device=DEV)
    cfg = small_cfg("behind", T=S, H=256, I=64, E=12, K=3, seed=3)
    inp = generate(cfg)
    layer, W = make_layer(inp, 16)
    wr = to_dev(inp.router_w)
    out_w = (torch.randn((Hq * D, 256), device=DEV) * 0.05).bfloat16()
    norm_w = torch.rand(256, device=DEV) + 0.5
    stream = torch.randn((S, 256), device=DEV).bfloat16()   # the residual stream of the last tokens
    lens, pos = [0] * S, [0] * S
    cuts = 0

    def held(s):
        """Keys and values of sequence s as the device has them, float64 [2, tokens, Hkv, D]."""
        pages = up(table[s, :-(-lens[s] // page)]).long()
        val = cache.kv[pages].double() if not fp8 else cache.kv.view(torch.uint8)[pages].view(torch.float8_e4m3fn).double() * 0.02
        return val.permute(1, 0, 3, 2, 4).reshape(2, -1, Hkv, D)[:, :lens[s]].cpu().numpy()

    for step in range(40):
        ns = [100, 20, 61] if step == 0 else [1] * S
        T = sum(ns)
        cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
        slots, positions = [], []
        for s, n in enumerate(ns):
            for i in range(n):
                at = lens[s] + i
                if table[s, at // page] == 1 << 30:
                    table[s, at // page] = free.pop()
                slots.append(int(table[s, at // page]) * page + at % page)
                positions.append(pos[s] + i)
            lens[s] += n
            pos[s] += n
        qkv = torch.randn((T, (Hq + 2 * Hkv) * D), device=DEV).bfloat16()
        q = cache.append(qkv, Hq, up(np.array(slots, np.int32)), up(np.array(positions, np.int32)), cos_sin, True, w, w)
        tab, dcu, kvl = up(table), up(cu), up(np.array(lens, np.int32))
        lse = torch.empty((T, Hq), device=DEV)
        note(f"generation step {step} lens={lens} fp8={fp8}")
        attend = cache.prefill_attention if step == 0 else cache.tree_attention
        out = attend(q, tab, dcu, kvl, max(ns), lse=lse)
        before = usage.cpu().numpy()
        cache.usage(q, tab, dcu, kvl, max(ns), lse, usage, None if step == 0 else usage, decay, rows)
        torch.cuda.synchronize()
        c = make_case(ns, lens, Hq, Hkv, D, page, False, 0)
        c.fp8, c.q, c.T = fp8, bits_of(q.view(torch.int16)).reshape(T, -1), T
        both = [held(s) for s in range(S)]
        c.k, c.v = [b[0] for b in both], [b[1] for b in both]
        sees = [oracle.visible_prefill(n, k, 0) for n, k in zip(ns, lens)]
        check_attention(c, bits_of(out.view(torch.int16)), lse.cpu().numpy(), sees, D ** -0.5, 0.0)
        check_usage(c, usage.cpu().numpy(), lse.cpu().numpy(), sees, D ** -0.5, 0.0, None if step == 0 else before, decay,
                    rows.tolist(), guard=before)
        # what stands behind the attention
        if step:
            x = out.view(S, Hq * D) @ out_w
            res = stream
            y, stream = layer.add_norm(x, norm_w, res, 1e-6)
            torch.cuda.synchronize()
            check_norm(bits_of(x.view(torch.int16)), bits_of(res.view(torch.int16)), norm_w.cpu().numpy(), 1e-6, 256, 0,
                       (bits_of(stream.view(torch.int16)), bits_of(y.view(torch.int16)),
                        layer.ws_view("xq", torch.uint8, (S, 256)).cpu().numpy(),
                        layer.ws_view("sx", torch.float32, (S, 1)).cpu().numpy()))
            moe, again = layer.forward_normed(x, norm_w, wr, None, W, res, 1e-6)
            assert torch.equal(again, stream) and bool(moe.isfinite().all())
        # the cut
        new = np.full((S, budget // page), -1, np.int32)
        for s in range(S):
            if lens[s] > limit:
                new[s] = [free.pop() for _ in range(budget // page)]
        used = usage.cpu().numpy()
        got_lens, kept = cache.evict(tab, kvl, usage, up(new), budget, limit, sinks, recent, rows)
        torch.cuda.synchronize()
        now, kept = usage.cpu().numpy(), kept.cpu().numpy()
        for s in range(S):
            r = int(rows[s])
            if lens[s] <= limit:
                assert int(got_lens[s]) == lens[s] and np.all(kept[s] == -1)
                assert np.array_equal(now[r], used[r], equal_nan=True)
                continue
            cuts += 1
            for h in range(Hkv):
                k = oracle.kept_tokens(used[r, h], lens[s], budget, sinks, recent)
                assert np.array_equal(kept[s, h], k)
                assert np.array_equal(now[r, h, :budget], used[r, h, k])
            old = both[s]
            free += [int(p) for p in table[s, :-(-lens[s] // page)]]
            table[s] = 1 << 30
            table[s, :budget // page] = new[s]
            lens[s] = int(got_lens[s])
            assert lens[s] == budget
            mine = held(s)
            for h in range(Hkv):
                assert np.array_equal(mine[:, :, h], old[:, kept[s, h], h])
    assert cuts >= 6
