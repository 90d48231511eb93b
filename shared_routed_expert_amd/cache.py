"""A paged key/value cache on the GPU and the calls that write and read it.

Torch provides device memory and the stream (always torch's current stream of the cache's device); the
writes (moe_kv_append) and the attention (moe_tree_attention, moe_prefill_attention, moe_window_attention), the
tokens' usage and the eviction by it (moe_kv_usage, moe_kv_evict) run in libsrmoe.so's HIP kernels. Every tensor starts on a 16-byte boundary, as torch allocates them; a slice that does not is
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

    def _tensor(self, t, name, dtype, shape, strided=False, slice_too=False):
        _need(isinstance(t, torch.Tensor) and t.dtype == dtype and tuple(t.shape) == tuple(shape),
              f"{name} is {dtype} {list(shape)}")
        _need(strided or t.is_contiguous(), f"{name} is contiguous")
        _need(t.device == self.kv.device, f"{name} is on the cache's device")
        if not slice_too:   # a contiguous slice may begin at any element
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

    def _queries(self, q, block_table, cu_q, kv_lens):
        """Checks of what every call with queries takes; (S, T, q heads, max_pages)."""
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
        return S, T, Hq, max_pages

    def _attention(self, call, q, block_table, cu_q, kv_lens, extra, max_q, scale, softcap, out, lse):
        D = self.head_dim
        S, T, Hq, max_pages = self._queries(q, block_table, cu_q, kv_lens)
        if out is None:
            out = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device=q.device)   # rows of no sequence are not written
        self._tensor(out, "out", torch.bfloat16, (T, Hq, D))
        if lse is not None:
            self._tensor(lse, "lse", torch.float32, (T, Hq))
        n = L.moe_attention_workspace_bytes(S, T, max_q, Hq, self.num_kv_heads, D)
        # from torch's allocator for each call: stream-ordered, and a captured graph keeps its own
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device=q.device)
        self._run(call, q, q.stride(0) if T > 1 else Hq * D, self.k, self.v, self.kv_type, self.k_scale, self.v_scale,
                  self.num_pages, self.page_size, self.kv.stride(0), block_table, max_pages, cu_q, kv_lens, *extra, S, T,
                  max_q, Hq, self.num_kv_heads, D, D ** -0.5 if scale is None else scale, softcap, out, lse, ws, n)
        return out

    def tree_attention(self, q, block_table, cu_q, kv_lens, max_q, tree_mask=None, scale=None, softcap=0.0, out=None,
                       lse=None):
        """Attention of each sequence's last tokens (drafted ones: tree_mask [T] int64 words, bit b = the sequence's
        drafted token b is seen; None: a chain, with one token per sequence ordinary decoding) over its cached tokens.
        scale: head_dim^-1/2 unless given. Returns out [T, q heads, head_dim]; rows outside every sequence and a
        sequence's tokens past max_q are zero, or left as they were in an out (and lse) that is given. out is not q."""
        if tree_mask is not None:
            self._tensor(tree_mask, "tree_mask", torch.int64, (q.shape[0],))
        return self._attention(L.moe_tree_attention, q, block_table, cu_q, kv_lens, (tree_mask,), max_q, scale, softcap,
                               out, lse)

    def prefill_attention(self, q, block_table, cu_q, kv_lens, max_q, prefix_lens=None, scale=None, softcap=0.0, out=None,
                          lse=None):
        """Causal attention of a chunk's tokens over the cached tokens, its own among them (append first);
        prefix_lens [S]: every token also sees its sequence's first prefix_lens[s] tokens. scale, out, lse and the rows
        outside every sequence as in tree_attention."""
        if prefix_lens is not None:
            self._tensor(prefix_lens, "prefix_lens", torch.int32, (block_table.shape[0],))
        return self._attention(L.moe_prefill_attention, q, block_table, cu_q, kv_lens, (prefix_lens,), max_q, scale,
                               softcap, out, lse)

    def window_attention(self, q, block_table, cu_q, kv_lens, max_q, window, sinks=0, scale=None, softcap=0.0, out=None,
                         lse=None):
        """Causal attention of a chunk's tokens (max_q 1: decoding), each over the last `window` cached tokens up to
        itself and the sequence's first `sinks`. Tokens that nobody sees are not used and their pages' entries in
        block_table may hold anything: pages that the window has left may be given to others. scale, out, lse and the rows
        outside every sequence as in tree_attention."""
        _need(isinstance(window, int) and isinstance(sinks, int) and 1 <= window < 2 ** 31 and 0 <= sinks < 2 ** 31,
              "window is a whole number of at least 1, sinks of at least 0")
        return self._attention(L.moe_window_attention, q, block_table, cu_q, kv_lens, (window, sinks), max_q, scale,
                               softcap, out, lse)

    def _usage_rows(self, usage, rows, S, max_pages, name="usage"):
        _need(isinstance(usage, torch.Tensor) and usage.dim() == 3, f"{name} is float32 [rows, kv heads, tokens of a table's row]")
        self._tensor(usage, name, torch.float32, (usage.shape[0], self.num_kv_heads, max_pages * self.page_size))
        if rows is not None:
            self._tensor(rows, "rows", torch.int32, (S,))
        _need(usage.shape[0] >= (1 if rows is not None else S), f"{name} has a row for every sequence, or rows is given")

    def usage(self, q, block_table, cu_q, kv_lens, max_q, lse, usage, prev=None, decay=1.0, rows=None, prefix_lens=None,
              scale=None, softcap=0.0):
        """The attention weight that each cached token gets from q (lse [T, q heads]: of the attention call on the same rows),
        summed over the tokens and the heads of a kv head, plus decay * prev for the tokens before the call's own, into
        usage [rows, kv heads, block_table.shape[1] * page_size] float32 (prev: None, usage itself or another array like
        it; rows [S] int32: each sequence's row, None: its number). Sequences without tokens in q keep their row. Returns
        usage."""
        S, T, Hq, max_pages = self._queries(q, block_table, cu_q, kv_lens)
        D = self.head_dim
        self._tensor(lse, "lse", torch.float32, (T, Hq))
        self._usage_rows(usage, rows, S, max_pages)
        if prev is not None:
            self._tensor(prev, "prev", torch.float32, usage.shape)
        if prefix_lens is not None:
            self._tensor(prefix_lens, "prefix_lens", torch.int32, (S,))
        n = L.moe_kv_usage_workspace_bytes(S, T, max_q, Hq, self.num_kv_heads, D)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device=q.device)
        self._run(L.moe_kv_usage, q, q.stride(0) if T > 1 else Hq * D, self.k, self.kv_type, self.k_scale, self.num_pages,
                  self.page_size, self.kv.stride(0), block_table, max_pages, cu_q, kv_lens, prefix_lens, lse, S, T, max_q, Hq,
                  self.num_kv_heads, D, D ** -0.5 if scale is None else scale, softcap, prev, decay, usage, rows,
                  usage.shape[0], ws, n)
        return usage

    def evict(self, block_table, kv_lens, usage, new_table, budget, limit=None, sinks=0, recent=0, rows=None,
              new_usage=None):
        """Cuts every sequence of more than `limit` tokens (budget unless given) to `budget`: each kv head keeps the first
        `sinks`, the last `recent` and, between them, those of largest usage, in order, copied to the pages of new_table
        [S, pages of the budget] int32, which no sequence may read in this call. usage is compacted into new_usage (itself
        unless given). Returns (new_lens [S], kept [S, kv heads, budget]: old places of the kept tokens; -1 for a sequence
        that is not cut). The caller takes new_table's row for the sequences that were cut and gives their old
        pages back."""
        _need(isinstance(block_table, torch.Tensor) and block_table.dim() == 2, "block_table is int32 [S, max_pages]")
        S, max_pages = block_table.shape
        self._tensor(block_table, "block_table", torch.int32, (S, max_pages))
        self._tensor(kv_lens, "kv_lens", torch.int32, (S,))
        _need(isinstance(new_table, torch.Tensor) and new_table.dim() == 2, "new_table is int32 [S, pages of the budget]")
        self._tensor(new_table, "new_table", torch.int32, (S, new_table.shape[1]), slice_too=True)
        self._usage_rows(usage, rows, S, max_pages)
        if new_usage is None:
            new_usage = usage
        self._tensor(new_usage, "new_usage", torch.float32, usage.shape)
        limit = budget if limit is None else limit
        _need(1 <= budget <= limit < 2 ** 31, "budget is at least 1 and at most limit")
        _need(sinks >= 0 and recent >= 0 and sinks + recent <= budget, "sinks and recent fit into budget")
        _need(new_table.shape[1] * self.page_size >= budget, "new_table's rows hold budget tokens")
        new_lens = torch.empty_like(kv_lens)
        kept = torch.full((S, self.num_kv_heads, budget), -1, dtype=torch.int32, device=kv_lens.device)
        self._run(L.moe_kv_evict, self.k, self.v, self.kv_type, self.num_pages, self.page_size, self.kv.stride(0),
                  block_table, max_pages, kv_lens, usage, new_usage, rows, usage.shape[0], S, self.num_kv_heads, self.head_dim,
                  limit, budget, sinks, recent, new_table, new_table.shape[1], new_lens, kept)
        return new_lens, kept
