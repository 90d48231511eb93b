"""moe_add_rms_norm against the float64 oracle, and the layer behind it.

Bars, per value. With e = 2^-24 (H / 128 + 40): a thread adds at most H / 64 squares (64 threads to a row), each sum rounded once,
and the square root halves that; under 20 joins, and some 12 roundings of h, the square
root, the quotients and the products:
  residual_out: (2^-8 + 2^-24) |h|             y (bf16): (2^-8 + e) |y|, and 2^-134 for subnormals
  sx: e sx                                     xq sx: (2^-4 + e) |y| + 2^-10 sx: half a step of e4m3, of its subnormals
"""
import numpy as np
import pytest
import torch

import oracle
from shared_routed_expert_amd import _lib as L
from tests.gpu_util import DEV, bf16_dev, make_layer, note, small_cfg, to_dev
from workloads import CONFIGS, bf16_bits_from_f32, f32_from_bf16_bits, generate

pytestmark = pytest.mark.gpu


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def make(T, H, seed, extra=0, spread=1.0):
    rng = np.random.default_rng(seed)
    x = bf16_bits_from_f32(rng.standard_normal((T, H + extra)).astype(np.float32))
    r = bf16_bits_from_f32((rng.standard_normal((T, H)) * np.exp(spread * rng.standard_normal(H))).astype(np.float32))
    w = rng.uniform(-1.5, 1.5, H).astype(np.float32)
    return x, r, w


def values(bits):
    return f32_from_bf16_bits(np.ascontiguousarray(bits)).astype(np.float64)


def run(x, r, w, eps, H, mode, y=True, q=True, res_out=True, guard=2):
    """One call; outputs with `guard` rows behind them that stay as they were."""
    T = x.shape[0]
    groups = H // 128 if mode else 1
    dx, dw = up(x.view(np.int16)), up(w)
    dr = None if r is None else up(r.view(np.int16))
    h = torch.full((T + guard, H), 0x7FC1, dtype=torch.int16, device=DEV) if res_out else None
    yo = torch.full((T + guard, H), 0x7FC1, dtype=torch.int16, device=DEV) if y else None
    xq = torch.full((T + guard, H), 0x7F, dtype=torch.uint8, device=DEV) if q else None
    sx = torch.full((T + guard, groups), 7.0, device=DEV) if q else None
    L.moe_add_rms_norm(dx, x.shape[1], dr, h, dw, eps, T, H, mode, yo, xq, sx)
    torch.cuda.synchronize()
    for t, v in ((h, 0x7FC1), (yo, 0x7FC1), (xq, 0x7F), (sx, 7.0)):
        assert t is None or bool((t[T:] == v).all())
    return tuple(None if t is None else t[:T].cpu().numpy() for t in (h, yo, xq, sx))


def check(x, r, w, eps, H, mode, got):
    e = 2.0 ** -24 * (H / 128 + 40)
    h, y = oracle.add_rms_norm(values(x[:, :H]), None if r is None else values(r), w, eps)
    gh, gy, gq, gs = got
    if gh is not None:
        assert np.all(np.abs(values(gh.view(np.uint16)) - h) <= (2.0 ** -8 + 2.0 ** -24) * np.abs(h))
    if gy is not None:
        err, bar = np.abs(values(gy.view(np.uint16)) - y), (2.0 ** -8 + e) * np.abs(y) + 2.0 ** -134
        assert np.all(err <= bar), float(np.max(err / bar))
    if gq is not None:
        s = oracle.act_scales(y, 128 if mode else None)
        assert np.all(np.abs(gs - s) <= e * s), float(np.max(np.abs(gs - s) / s))
        wide = np.repeat(gs.astype(np.float64), H // gs.shape[1], axis=1)
        err = np.abs(oracle.e4m3_decode(gq) * wide - y)
        bar = (2.0 ** -4 + e) * np.abs(y) + 2.0 ** -10 * wide
        assert np.all(err <= bar), float(np.max(err / bar))


@pytest.mark.parametrize("H", [8, 16, 120, 128, 136, 512, 1000, 1024, 2048, 2056, 4096, 4104, 5120, 7168, 8192, 8200, 16384,
                               65536])
@pytest.mark.parametrize("T", [1, 3, 65])
def test_sizes(T, H):
    x, r, w = make(T, H, H + T)
    for mode in (0, 1):
        if mode and H % 128:
            continue
        note(f"add_rms_norm T={T} H={H} mode={mode}")
        check(x, r, w, 1e-5, H, mode, run(x, r, w, 1e-5, H, mode))


@pytest.mark.parametrize("T", [200, 2000, 5000])
@pytest.mark.parametrize("H", [128, 1280, 5120, 8448])
def test_many_tokens(T, H):
    x, r, w = make(T, H, H + T)
    for mode in (0, 1):
        note(f"add_rms_norm T={T} H={H} mode={mode}")
        check(x, r, w, 1e-6, H, mode, run(x, r, w, 1e-6, H, mode))


@pytest.mark.parametrize("H", [384, 5120, 10240])
@pytest.mark.parametrize("T", [9, 3000])
def test_optional_parts(T, H):
    """Without a residual, without either result, strided rows of x."""
    x, r, w = make(T, H, 1, extra=24)
    for kw in (dict(y=False), dict(q=False), dict(res_out=False), dict(q=False, res_out=False)):
        for res in (r, None):
            note(f"add_rms_norm T={T} H={H} {kw} residual={res is not None}")
            check(x, res, w, 1e-5, H, 0, run(x, res, w, 1e-5, H, 0, **kw))


@pytest.mark.parametrize("H", [256, 5120, 10240])
@pytest.mark.parametrize("T", [5, 2500])
def test_in_place(T, H):
    """residual_out is residual, y is x: the bits of the call with buffers of its own."""
    x, r, w = make(T, H, 2)
    want = run(x, r, w, 1e-5, H, 0)
    dx, dr = up(x.view(np.int16)), up(r.view(np.int16))
    xq, sx = torch.empty((T, H), dtype=torch.uint8, device=DEV), torch.empty((T, 1), device=DEV)
    L.moe_add_rms_norm(dx, H, dr, dr, up(w), 1e-5, T, H, 0, dx, xq, sx)
    torch.cuda.synchronize()
    for a, b in zip(want, (dr, dx, xq, sx)):
        assert np.array_equal(a, b.cpu().numpy())


@pytest.mark.parametrize("H", [1024, 5120, 9216])
def test_extremes(H):
    """Rows of zeros, of the largest and smallest values whose squares float32 holds, one large value among small ones; NaN
    and infinities stay in their row."""
    T = 8
    x, r, w = make(T, H, 3)
    x[0] = 0
    r[0] = 0
    x[1] = bf16_bits_from_f32(values(x[1]).astype(np.float32) * np.float32(2.0 ** 50))
    r[1] = x[1]
    x[2] = bf16_bits_from_f32(values(x[2]).astype(np.float32) * np.float32(2.0 ** -40))
    r[2] = 0
    x[3, H // 2] = bf16_bits_from_f32(np.float32([3e4]))[0]
    for mode in (0, 1):
        clean = run(x, r, w, 1e-5, H, mode)
        check(x, r, w, 1e-5, H, mode, clean)
        # (zeros of either sign: h is 0, the weights have signs)
        assert not values(clean[1][0].view(np.uint16)).any() and not oracle.e4m3_decode(clean[2][0]).any()
        assert np.all(clean[3][0] == 1.0)
        bad = x.copy()
        bad[4, 3], bad[6, H - 1] = 0x7FC1, 0x7F80
        got = run(bad, r, w, 1e-5, H, mode)
        others = [0, 1, 2, 3, 5, 7]
        for a, b in zip(clean, got):
            assert np.array_equal(a[others], b[others])
        y = values(got[1].view(np.uint16))
        assert np.all(np.isnan(y[4])) and np.isnan(y[6, H - 1]) and not np.any(y[6, :H - 1])


def test_same_bits_in_any_batch_and_on_any_stream():
    """A row's result depends on the row alone where the sizes take the same kernel; repeated calls agree; a captured call
    replays on new values."""
    H = 5120
    x, r, w = make(3000, H, 4)
    a = run(x, r, w, 1e-5, H, 1)
    b = run(x, r, w, 1e-5, H, 1)
    assert all(np.array_equal(p, q) for p, q in zip(a, b))
    T = 64
    dx, dr, dw = torch.empty((T, H), dtype=torch.int16, device=DEV), torch.empty((T, H), dtype=torch.int16, device=DEV), up(w)
    h, y = torch.empty_like(dx), torch.empty_like(dx)
    xq, sx = torch.empty((T, H), dtype=torch.uint8, device=DEV), torch.empty((T, H // 128), device=DEV)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    dx.copy_(up(x[:T].view(np.int16)))
    dr.copy_(up(r[:T].view(np.int16)))
    call = lambda: L.moe_add_rms_norm(dx, H, dr, h, dw, 1e-5, T, H, 1, y, xq, sx, stream)
    with torch.cuda.stream(stream):
        call()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            call()
    for k in range(4):
        rows = slice(k * T, (k + 1) * T)
        dx.copy_(up(x[rows].view(np.int16)))
        dr.copy_(up(r[rows].view(np.int16)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = run(x[rows], r[rows], w, 1e-5, H, 1)
        for p, t in zip(want, (h, y, xq, sx)):
            assert np.array_equal(p, t.cpu().numpy()), k


@pytest.mark.parametrize("cfg,bm", [
    (CONFIGS["tiny"], 16),
    (CONFIGS["decode"], 16),
    (small_cfg("ragged", T=77, H=384, I=96, E=12, K=3, seed=11), 32),
    (small_cfg("three_blocks", T=300, H=640, I=192, E=20, K=8, seed=33), 128),
    (small_cfg("block", T=50, H=384, I=256, E=6, K=2, mode="block128", seed=15), 16),
    (small_cfg("block_i128", T=140, H=256, I=128, E=5, K=2, mode="block128", seed=34), 128),
    (small_cfg("one_token", T=1, H=256, I=64, E=20, K=8, seed=35), 16),
])
def test_the_layer_behind_the_norm(cfg, bm):
    """Rows of h = +-1 and a weight of bf16 values: mean h^2 = 1 and y = h w exactly, so that the codes are those that
    moe_ffn_quant_x makes of y, and forward_normed's bits those of forward_from_x on y."""
    inp = generate(cfg)
    T, H = cfg.T, cfg.H
    rng = np.random.default_rng(5)
    sign = rng.choice([-1.0, 1.0], (T, H))
    res = rng.integers(-64, 65, (T, H)) / 64.0          # +-1 - res: a multiple of 2^-6 up to 2, exact in bf16
    w = values(bf16_bits_from_f32(rng.uniform(0.1, 2.0, H).astype(np.float32)))
    note(f"norm and layer {cfg.name} bm={bm}")
    bits = lambda a: bf16_dev(bf16_bits_from_f32(a.astype(np.float32)))
    x, r = bits(sign - res), bits(res)
    wr = to_dev(inp.router_w)
    layer, W = make_layer(inp, bm)
    out, h = layer.forward_normed(x, up(w.astype(np.float32)), wr, None, W, residual=r, eps=0.0)
    torch.cuda.synchronize()
    got, codes = out.clone(), layer.ws_view("xq", torch.uint8, (T, H)).clone()
    assert np.array_equal(h.float().cpu().numpy(), sign)
    other, _ = make_layer(inp, bm)
    want = other.forward_from_x(bits(sign * w), wr, None, W)
    torch.cuda.synchronize()
    assert torch.equal(codes, other.ws_view("xq", torch.uint8, (T, H)))
    assert torch.equal(layer.topk_ids, other.topk_ids) and torch.equal(layer.topk_w, other.topk_w)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("raw", [False, True])
def test_a_call_on_a_stream_allocates_there(raw):
    """forward_normed on a stream that is behind: what it frees on returning is not given to the current stream's tensors."""
    inp = generate(small_cfg("streams", T=64, H=384, I=96, E=12, K=3, seed=12))
    layer, W = make_layer(inp, 16)
    T, H = 64, 384
    rng = np.random.default_rng(0)
    x = bf16_dev(bf16_bits_from_f32(rng.standard_normal((T, H)).astype(np.float32)))
    w, wr = up(np.ones(H, np.float32)), to_dev(inp.router_w)
    want, h = layer.forward_normed(x, w, wr, None, W, residual=x)
    want = want.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    note(f"norm on a stream behind, raw={raw}")
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    got, other = layer.forward_normed(x, w, wr, None, W, residual=x, stream=side.cuda_stream if raw else side)
    mine = [torch.zeros((T, H), dtype=torch.bfloat16, device=DEV) for _ in range(8)]
    torch.cuda.synchronize()
    assert not any(t.any() for t in mine)
    assert torch.equal(got, want) and torch.equal(other, h)


def test_forward_normed_captured():
    """Captured and replayed on new values, with eager calls of the same layer between the replays."""
    inp = generate(small_cfg("captured", T=64, H=384, I=96, E=12, K=3, seed=12))
    layer, W = make_layer(inp, 16)
    T, H = 64, 384
    rng = np.random.default_rng(1)
    new = lambda: bf16_dev(bf16_bits_from_f32(rng.standard_normal((T, H)).astype(np.float32)))
    x, r = new(), new()
    w, wr = up(rng.uniform(0.5, 1.5, H).astype(np.float32)), to_dev(inp.router_w)
    note("norm and layer captured")
    layer.forward_normed(x, w, wr, None, W, residual=r)
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        out, h = layer.forward_normed(x, w, wr, None, W, residual=r)
    for rep in range(4):
        x.copy_(new())
        r.copy_(new())
        want, want_h = layer.forward_normed(x, w, wr, None, W, residual=r)
        want, want_h = want.clone(), want_h.clone()
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(h, want_h), rep
