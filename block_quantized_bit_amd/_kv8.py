"""Binding of the 8-bit paged key/value cache and its attention (include/kv8.h): argument marshalling only.

The cache is four tensors that the caller owns (kv8_cache makes them): codes int8 or float8_e4m3fn, K as
[pages][kv heads][page size][d] and V transposed, [pages][kv heads][d][page size], and a float32 scale [pages][kv heads]
for each."""
from __future__ import annotations

import torch

from ._args import native
from ._lib import _empty

KV8_EXPORTS = ("kv8_append", "kv8_read", "kv8_attention_work_bytes", "kv8_attention")
KV8_DTYPES = (torch.int8, torch.float8_e4m3fn)


def kv8_cache(pages: int, kv_heads: int, page_size: int, head_dim: int, dtype=torch.int8, device="cuda"):
    """Zeroed tensors (k_codes, v_codes, k_scale, v_scale) of an empty cache."""
    if dtype not in KV8_DTYPES:
        raise ValueError(f"unsupported cache dtype {dtype} (int8 or float8_e4m3fn)")
    codes = [torch.zeros(shape, dtype=torch.int8, device=device).view(dtype)
             for shape in ((pages, kv_heads, page_size, head_dim), (pages, kv_heads, head_dim, page_size))]
    scales = [torch.zeros((pages, kv_heads), dtype=torch.float32, device=device) for _ in range(2)]
    return (*codes, *scales)


def kv8_append(k, v, k_codes, v_codes, k_scale, v_scale, page_table, kv_len, cu, max_new: int, stream=None):
    """Stores the packed new tokens k, v [total][kv heads][d] (float32 or bfloat16) as the last cu[b+1] - cu[b] tokens
    of each sequence b, whose length kv_len[b] already counts them. max_new bounds the tokens of one sequence."""
    native().kv8_append(k, v, k_codes, v_codes, k_scale, v_scale, page_table, kv_len, cu, max_new, stream)


def kv8_read(k_codes, v_codes, k_scale, v_scale, page_table, kv_len, cu, max_new: int, total: int | None = None,
             dtype=torch.bfloat16, out=None, stream=None):
    """Values (code * scale) of the last cu[b+1] - cu[b] tokens of each sequence, packed: (k, v), each
    [total][kv heads][d]. total (= cu[-1]) may be left out where `out` is given."""
    if out is None:
        if total is None:
            raise ValueError("total (the last entry of cu) or out is needed")
        shape = (total, k_codes.shape[1], k_codes.shape[3])
        out = tuple(_empty(stream, shape, dtype, k_codes.device) for _ in range(2))
    native().kv8_read(k_codes, v_codes, k_scale, v_scale, page_table, kv_len, cu, max_new, out[0], out[1], stream)
    return out[0], out[1]


def kv8_attention(q, k_codes, v_codes, k_scale, v_scale, page_table, kv_len, cu, max_new: int, max_kv: int,
                  scale: float | None = None, window: int = 0, out=None, lse=None, work=None, stream=None):
    """Causal attention of the packed queries q [total][heads][d] (float32 or bfloat16) over the cache -> out
    [total][heads][d] in q's dtype. The queries of sequence b are its last cu[b+1] - cu[b] tokens (already appended).
    max_new and max_kv bound the queries and the length of one sequence; window > 0 limits each query to its last
    `window` keys; scale defaults to d ** -0.5. lse, if given, is float32 [total][heads]."""
    return native().kv8_attention(q, k_codes, v_codes, k_scale, v_scale, page_table, kv_len, cu, max_new, max_kv, scale,
                                  window, out, lse, work, stream)
