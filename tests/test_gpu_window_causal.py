"""moe_window_attention with a window over everything against moe_prefill_attention: no token is left out, so both have the
causal call's value, each within test_gpu_attention's bars, and the same bits where each takes its segments whole (the parts
of split ones are cut elsewhere: a window's last tile counts a whole tile's keys)."""
import numpy as np
import pytest
import torch

import oracle
from tests.gpu_util import note
from tests.kv_util import make_case
from tests.test_gpu_attention import bits_of, check
from tests.test_gpu_window_attention import WinDev

pytestmark = pytest.mark.gpu


def both(c, window, sinks, scale, cap):
    """Out and lse of the two calls, into buffers filled anew, each against the oracle."""
    d, got = WinDev(c), []
    sees = [oracle.visible_prefill(n, k, 0) for n, k in zip(c.ns, c.kvs)]
    for run in (lambda: d.run(window, sinks, scale, cap), lambda: d.call("prefill", None, scale, cap)):
        d.out.fill_(0x7FC1)
        d.lse.fill_(7.0)
        d.ws.fill_(0xCD)
        run()
        torch.cuda.synchronize()
        out, lse = bits_of(d.out).copy(), d.lse.cpu().numpy().copy()
        check(c, out, lse, sees, c.D ** -0.5 if scale is None else scale, cap)
        got.append((out, lse))
    return got


HEADS = [(12, 1, 128), (96, 8, 128), (8, 2, 64), (8, 1, 256)]
SHAPES = {"chunks": ([70, 5, 0, 200], [400, 300, 9, 200]), "tokens": ([1] * 6, [1, 31, 64, 65, 300, 480])}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_whole_segments_give_the_same_bits(shape, Hq, Hkv, D, fp8):
    """A table of 512 tokens at most."""
    for (window, sinks), scale, cap in (((1 << 20, 0), None, 0.0), ((480, 0), 0.3, 5.0), ((1, 480), None, 0.0)):
        c = make_case(*SHAPES[shape], Hq, Hkv, D, 16, fp8, seed=13, lead=1, tail=2)
        assert c.table.shape[1] * 16 <= 512
        note(f"window {window} sinks {sinks} and causal, {shape} {Hq} {Hkv} {D} fp8={fp8} cap={cap}")
        a, b = both(c, window, sinks, scale, cap)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_split_segments_have_the_same_value(Hq, Hkv, D, fp8):
    for ns, kvs in (([70, 5, 300], [5000, 700, 2500]), ([1, 1, 1], [20000, 3, 900])):
        c = make_case(ns, kvs, Hq, Hkv, D, 16, fp8, seed=14)
        note(f"window over everything and causal, split, {ns} {kvs} {Hq} {Hkv} {D} fp8={fp8}")
        both(c, 1 << 20, 0, None, 0.0)
