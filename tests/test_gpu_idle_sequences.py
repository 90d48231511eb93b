"""A few sequences with query tokens among thousands without: runs of idle ones at the start, between and at the end, longer and
shorter than a wavefront's 64 and on its borders; usage and the attention calls against their oracles."""
import pytest

import oracle
from tests.kv_util import make_case
from tests.test_gpu_attention import run_check as check_attention
from tests.test_gpu_kv_usage import run_check as check_usage
from tests.test_gpu_window_attention import run_check as check_window

pytestmark = pytest.mark.gpu

# places of the active ones: gaps of 0, 1, 62 to 66, 127 to 129 and thousands
GAPS = [0, 1, 3, 66, 130, 195, 261, 328, 456, 585, 715, 3900, 3901]


def case(S, places, n, kv, fp8=False):
    ns, kvs = [0] * S, [(7 * s) % 40 for s in range(S)]   # (idle ones hold tokens, some none)
    for i, s in enumerate(places):
        ns[s], kvs[s] = n, kv + 37 * i
    return make_case(ns, kvs, 4, 1, 64, 16, fp8, seed=S + n, lead=1, tail=1)


@pytest.mark.parametrize("n", [1, 7, 20, 150])
@pytest.mark.parametrize("S,places", [(65, [0, 64]), (200, [3, 199]), (4000, GAPS), (4000, [0, 3999]), (4000, [1999]),
                                      (5000, [4990, 4995, 4999]), (5000, [0, 1, 2])])
def test_usage(S, places, n):
    for fp8 in (False, True):
        check_usage(case(S, places, n, n + 300, fp8), prev=True, decay=0.5)


@pytest.mark.parametrize("n", [1, 40])
def test_usage_of_active_sequences_without_cached_tokens(n):
    """They have no key blocks, so they are passed by like idle ones."""
    c = case(1000, [0, 70, 400, 900], n, n + 100)
    kvs = list(c.kvs)
    for s in (70, 400):
        kvs[s] = 0
    check_usage(make_case(c.ns, kvs, 4, 1, 64, 16, False, seed=n), prev=True)


@pytest.mark.parametrize("n", [1, 7, 20, 150])
@pytest.mark.parametrize("S,places", [(65, [0, 64]), (200, [3, 199]), (4500, GAPS + [4499]), (5000, [0, 4999]), (5000, [4990, 4999])])
def test_attention(S, places, n):
    for fp8 in (False, True):
        for wide in ((False, True) if S < 4000 or not fp8 and S == 4500 else (False,)):
            c = case(S, places, n, n + 300, fp8)
            check_attention(c, "prefill", None, [oracle.visible_prefill(a, k, 0) for a, k in zip(c.ns, c.kvs)], wide=wide)
            check_window(case(S, places, n, n + 300, fp8), 190, 5, wide=wide)
        if n <= 64:
            c = case(S, places, n, n + 300, fp8)
            check_attention(c, "tree", None, [oracle.visible_tree(a, k, None) for a, k in zip(c.ns, c.kvs)])
