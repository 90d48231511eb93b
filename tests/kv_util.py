"""Seeded inputs of the paged-cache tests, on the host: a pool of pages that holds NaN patterns everywhere except
in the cached tokens, block tables over it in random order, and the float64 values that the tokens stand for."""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np

from oracle import e4m3_decode, e4m3_encode
from workloads import bf16_bits_from_f32, f32_from_bf16_bits

NAN_BF16, NAN_E4M3 = 0x7FC1, 0x7F


@dataclass
class Case:
    ns: list            # query tokens per sequence
    kvs: list           # cached tokens per sequence
    Hq: int
    Hkv: int
    D: int
    page: int
    fp8: bool
    q: np.ndarray       # uint16 [T, q_stride]: bf16 bits, the heads first
    kv: np.ndarray      # [pages, 2, Hkv, page, D] uint16 bits or uint8 codes
    scales: np.ndarray  # float32 [2, Hkv] (ones for bf16)
    table: np.ndarray   # int32 [S, max_pages]
    cu_q: np.ndarray    # int32 [S + 1]
    k: list             # per sequence [kv, Hkv, D] float64
    v: list
    T: int

    def q_heads(self, s):
        a, b = self.cu_q[s], self.cu_q[s] + self.ns[s]
        x = f32_from_bf16_bits(self.q[a:b, :self.Hq * self.D].copy())
        return x.reshape(-1, self.Hq, self.D).astype(np.float64)


def make_case(ns, kvs, Hq, Hkv, D, page, fp8, seed, lead=0, tail=0, q_extra=0, extra_pages=3, big=1.0):
    """lead / tail: rows of q before the first and behind the last sequence; q_extra: values between two tokens'
    heads; big: a factor on q (peaked softmax)."""
    rng = np.random.default_rng(seed)
    S = len(ns)
    need = [-(-k // page) for k in kvs]
    pages = sum(need) + extra_pages
    kv = np.full((pages, 2, Hkv, page, D), NAN_E4M3 if fp8 else NAN_BF16, np.uint8 if fp8 else np.uint16)
    order = rng.permutation(pages)
    table = np.full((S, max(max(need), 1) + 1), 1 << 30, np.int32)   # entries past a sequence's pages are not read
    scales = rng.uniform(0.01, 0.03, (2, Hkv)).astype(np.float32) if fp8 else np.ones((2, Hkv), np.float32)
    ks, vs, used = [], [], 0
    for s in range(S):
        got = order[used:used + need[s]]
        used += need[s]
        table[s, :need[s]] = got
        vals = []
        for w in range(2):
            x = rng.standard_normal((kvs[s], Hkv, D)).astype(np.float32) * (1.0 if w == 0 else np.exp(0.7 * rng.standard_normal(D)).astype(np.float32))
            if fp8:
                codes = e4m3_encode(np.clip(x / scales[w][None, :, None], -448, 448))
                vals.append(e4m3_decode(codes).astype(np.float64) * scales[w].astype(np.float64)[None, :, None])
            else:
                codes = bf16_bits_from_f32(x)
                vals.append(f32_from_bf16_bits(codes).astype(np.float64))
            for i, p in enumerate(got):
                part = codes[i * page:(i + 1) * page]
                kv[p, w, :, :len(part)] = part.transpose(1, 0, 2)
        ks.append(vals[0])
        vs.append(vals[1])
    cu = (lead + np.concatenate([[0], np.cumsum(ns)])).astype(np.int32)
    T = int(cu[-1]) + tail
    q = bf16_bits_from_f32((big * rng.standard_normal((T, Hq * D + q_extra))).astype(np.float32))
    return Case(list(ns), list(kvs), Hq, Hkv, D, page, fp8, q, kv, scales, table, cu, ks, vs, T)


def random_tree(n, rng, own=True):
    """Mask words of n drafted tokens: each sees its ancestors (and itself when `own`)."""
    words = []
    for i in range(n):
        p = int(rng.integers(-1, i)) if i else -1
        words.append((words[p] | (1 << p) if p >= 0 else 0) | (1 << i if own else 0))
    return np.array(words, dtype=np.uint64)
