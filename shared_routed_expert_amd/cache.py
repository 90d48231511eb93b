"""A paged key/value cache on the GPU and the calls that write and read it.

Torch provides device memory and the stream (always torch's current stream of the cache's device); the
writes (moe_kv_append) and the attention (moe_tree_attention, moe_prefill_attention) run in
libsrmoe.so's HIP kernels. Every tensor starts on a 16-byte boundary, as torch allocates them; a slice that does not is
refused by name.
"""
from __future__ import annotations

import torch

from . import _lib as L


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _need_aligned(t, name):
    # every pointer that the library takes; said here, where the tensor has a name
    _need(t.data_ptr() % 16 == 0, f"{name} starts on a 16-byte boundary (clone a slice that does not)")


class PagedKVCache:
    """num_pages pages of page_size tokens: kv [num_pages, 2 (keys, values), num_kv_heads, page_size, head_dim],
    bf16, or float8_e4m3fn with one positive float32 scale per kv head for keys and one for values."""

    def __init__(self, num_pages, page_size, num_kv_heads, head_dim, kv_type=L.KV_BF16, k_scale=None, v_scale=None,
                 device="cuda"):
        dev = torch.device(device)
        _need(num_pages >= 1 and num_kv_heads >= 1, "num_pages and num_kv_heads are at least 1")
        _need(page_size in (16, 32, 64, 128, 256, 512, 1024), "page_size is a power of two in 16..1024")
        _need(head_dim in (64, 128, 256), "head_dim is 64, 128 or 256")
        _need(kv_type in (L.KV_BF16, L.KV_E4M3), "kv_type is KV_BF16 or KV_E4M3")
        self.kv_type = kv_type
        self.k_scale = self.v_scale = None
        if kv_type == L.KV_E4M3:
            for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                _need(isinstance(t, torch.Tensor) and t.dtype == torch.float32 and tuple(t.shape) == (num_kv_heads,),
                      "an e4m3 cache needs k_scale and v_scale, float32 [num_kv_heads]")
                t = t.to(dev).contiguous()
                _need_aligned(t, name)
                setattr(self, name, t)
        dtype = torch.bfloat16 if kv_type == L.KV_BF16 else torch.float8_e4m3fn
        self.kv = torch.empty((num_pages, 2, num_kv_heads, page_size, head_dim), dtype=dtype, device=dev)
        self.num_pages, self.page_size = num_pages, page_size
        self.num_kv_heads, self.head_dim = num_kv_heads, head_dim

    @property
    def k(self):
        return self.kv[:, 0]

    @property
    def v(self):
        return self.kv[:, 1]

    def _tensor(self, t, name, dtype, shape, strided=False):
        _need(isinstance(t, torch.Tensor) and t.dtype == dtype and tuple(t.shape) == tuple(shape),
              f"{name} is {dtype} {list(shape)}")
        _need(strided or t.is_contiguous(), f"{name} is contiguous")
        _need(t.device == self.kv.device, f"{name} is on the cache's device")
        _need_aligned(t, name)
        return t

    def _run(self, call, *args):
        if self.kv.device.type != "cuda":
            raise ValueError("the cache is not on a GPU")
        with torch.cuda.device(self.kv.device):
            call(*args)

    def append(self, qkv, num_q_heads, slots, positions=None, cos_sin=None, neox=True, q_norm_w=None, k_norm_w=None,
               eps=1e-5, q_out=None):
        """Norm (when the weights are given) and rotation (when cos_sin [max_pos, rotary_dim] is given) of the q and
        k heads of qkv [T, (num_q_heads + 2 num_kv_heads) * head_dim] bf16 (rows may be strided); k and v go to their
        slots [T] int32 (-1: not cached). Returns the q heads [T, num_q_heads, head_dim]."""
        Hq, Hkv, D = num_q_heads, self.num_kv_heads, self.head_dim
        _need(isinstance(qkv, torch.Tensor) and qkv.dim() == 2, "qkv is bf16 [T, (q + 2 kv heads) * head_dim]")
        T = qkv.shape[0]
        self._tensor(qkv, "qkv", torch.bfloat16, (T, (Hq + 2 * Hkv) * D), strided=True)
        _need(qkv.stride(1) == 1, "a row of qkv is contiguous")
        _need(T < 2 or qkv.stride(0) % 8 == 0, "rows of qkv are a multiple of 8 values apart")
        self._tensor(slots, "slots", torch.int32, (T,))
        rd = max_pos = 0
        if cos_sin is not None:
            _need(isinstance(cos_sin, torch.Tensor) and cos_sin.dim() == 2, "cos_sin is [max_pos, rotary_dim]")
            max_pos, rd = cos_sin.shape
            self._tensor(cos_sin, "cos_sin", torch.float32, (max_pos, rd))
            self._tensor(positions, "positions", torch.int32, (T,))
        _need((q_norm_w is None) == (k_norm_w is None), "q_norm_w and k_norm_w are given together")
        for w, name in ((q_norm_w, "q_norm_w"), (k_norm_w, "k_norm_w")):
            if w is not None:
                self._tensor(w, name, torch.float32, (D,))
        if q_out is None:
            q_out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=self.kv.device)
        self._tensor(q_out, "q_out", torch.bfloat16, (T, Hq, D))
        row = (Hq + 2 * Hkv) * D
        self._run(L.moe_kv_append, qkv, qkv.stride(0) if T > 1 else row, T, Hq, Hkv, D, rd, neox, q_norm_w, k_norm_w,
                  eps, positions, cos_sin, max_pos, slots, q_out, self.k, self.v, self.kv_type, self.k_scale,
                  self.v_scale, self.num_pages, self.page_size, self.kv.stride(0))
        return q_out

    def _attention(self, call, q, block_table, cu_q, kv_lens, extra, max_q, scale, softcap, out, lse):
        D = self.head_dim
        _need(isinstance(q, torch.Tensor) and q.dim() == 3, "q is bf16 [T, q heads, head_dim]")
        T, Hq = q.shape[:2]
        self._tensor(q, "q", torch.bfloat16, (T, Hq, D), strided=True)
        _need(q.stride(2) == 1 and (q.stride(1) == D or Hq == 1), "a token's heads are contiguous in q")
        _need(T < 2 or q.stride(0) % 8 == 0, "rows of q are a multiple of 8 values apart")
        _need(isinstance(block_table, torch.Tensor) and block_table.dim() == 2, "block_table is int32 [S, max_pages]")
        S, max_pages = block_table.shape
        self._tensor(block_table, "block_table", torch.int32, (S, max_pages))
        self._tensor(cu_q, "cu_q", torch.int32, (S + 1,))
        self._tensor(kv_lens, "kv_lens", torch.int32, (S,))
        if out is None:
            out = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device=q.device)   # rows of no sequence are not written
        self._tensor(out, "out", torch.bfloat16, (T, Hq, D))
        if lse is not None:
            self._tensor(lse, "lse", torch.float32, (T, Hq))
        n = L.moe_attention_workspace_bytes(S, T, max_q, Hq, self.num_kv_heads, D)
        # from torch's allocator for each call: stream-ordered, and a captured graph keeps its own
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device=q.device)
        self._run(call, q, q.stride(0) if T > 1 else Hq * D, self.k, self.v, self.kv_type, self.k_scale, self.v_scale,
                  self.num_pages, self.page_size, self.kv.stride(0), block_table, max_pages, cu_q, kv_lens, extra, S, T,
                  max_q, Hq, self.num_kv_heads, D, D ** -0.5 if scale is None else scale, softcap, out, lse, ws, n)
        return out

    def tree_attention(self, q, block_table, cu_q, kv_lens, max_q, tree_mask=None, scale=None, softcap=0.0, out=None,
                       lse=None):
        """Attention of each sequence's last tokens (drafted ones: tree_mask [T] int64 words, bit b = the sequence's
        drafted token b is seen; None: a chain, with one token per sequence ordinary decoding) over its cached tokens.
        scale: head_dim^-1/2 unless given. Returns out [T, q heads, head_dim]; rows outside every sequence and a
        sequence's tokens past max_q are zero, or left as they were in an out (and lse) that is given."""
        if tree_mask is not None:
            self._tensor(tree_mask, "tree_mask", torch.int64, (q.shape[0],))
        return self._attention(L.moe_tree_attention, q, block_table, cu_q, kv_lens, tree_mask, max_q, scale, softcap, out,
                               lse)

    def prefill_attention(self, q, block_table, cu_q, kv_lens, max_q, prefix_lens=None, scale=None, softcap=0.0, out=None,
                          lse=None):
        """Causal attention of a chunk's tokens over the cached tokens, its own among them (append first);
        prefix_lens [S]: every token also sees its sequence's first prefix_lens[s] tokens. scale, out, lse and the rows
        outside every sequence as in tree_attention."""
        if prefix_lens is not None:
            self._tensor(prefix_lens, "prefix_lens", torch.int32, (block_table.shape[0],))
        return self._attention(L.moe_prefill_attention, q, block_table, cu_q, kv_lens, prefix_lens, max_q, scale, softcap,
                               out, lse)
