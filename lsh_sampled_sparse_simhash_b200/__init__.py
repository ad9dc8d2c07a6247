"""B200 (sm_100a) LSH-sampled decode attention (MagicPIG hot path).

The compute lives in ``libmagicpig_b200.so`` (hand-written CUDA kernels behind
the C ABI of ``include/magicpig.h``); this package is a thin ctypes binding
that marshals torch tensors (device memory and streams only) into those calls.
There is no fallback: if the library is missing or cannot load, every call
raises.

Beside the sampled decode: causal attention over packed prompts
(``prompt_attend``), exact decode over a paged key-value cache
(``paged_attend``), the append into its pages (``paged_append``) and the
operations on them (``pages_reserve``, ``pages_fork``, ``pages_free``,
``pages_compact``, ``pages_copy``).  A cache from prompt to prompt::

    pages_reserve(shape, lens_of_new, table, lens, refs)       # pages for the prompts
    prompt_attend(prompt_shape, q, k, v, cu, out, lse)          # every layer
    paged_append(shape, k, v, table, lens, k_pages, v_pages, cu_new=cu)
    pages_fork(shape, src, dst, table, lens, refs, copies)      # n answers to one prompt
    pages_copy(shape, copies, k_pages, v_pages)                 # every layer
    pages_reserve(shape, ones, table, lens, refs)               # each step: a page where one is needed,
    paged_append(shape, k_new, v_new, table, lens, k_pages, v_pages)
    paged_attend(shape, q, k_pages, v_pages, table, lens, max_len, out, lse, workspace)
    pages_free(shape, ended, table, lens, refs)

A prompt into the cache of the sampled decode, ``[batch, kv heads, capacity, d]``, which is one page of ``capacity``
tokens a sequence (``n_pages=batch, page_size=capacity, max_pages=1`` and a table of 0, 1, ..)::

    prompt_attend(prompt_shape, q, k, v, cu, out, lse)
    paged_append(one_page_each, k, v, table, lens, k_cache, v_cache, cu_new=cu)
    hash_keys(shape, k_cache, W, longest, codes)
    append_token(...); decode_attend(...)                       # each step; paged_attend reads the same cache exactly
"""
from ._binding import (  # noqa: F401
    MagicPIGError,
    PagesShape,
    PromptShape,
    Shape,
    append_token,
    append_token_q8,
    auto_planes,
    codes_bytes,
    codes_shape,
    decode_attend,
    decode_attend_noalloc,
    decode_attend_q8,
    decode_workspace_bytes,
    hash_keys,
    hash_keys_range,
    hash_queries,
    library,
    library_path,
    paged_append,
    paged_attend,
    paged_workspace_bytes,
    pages_compact,
    pages_copy,
    pages_fork,
    pages_free,
    pages_reserve,
    prompt_attend,
    quantize_keys,
    read_status,
    status_string,
    MP_OK,
    MP_ERR_ARG,
    MP_ERR_SHAPE,
    MP_ERR_ALIGN,
    MP_ERR_CAPACITY,
    MP_ERR_WORKSPACE,
    MP_ERR_CUDA,
    MP_ERR_TOO_LARGE,
    MP_CODES_AUTO,
    MP_CODES_BYTES,
    MP_CODES_PLANES,
    MP_CODES_AUTO_PLANES_MIN,
    Q8_ROW_BYTES,
    MP_PATH_AUTO,
    MP_PATH_SPLIT,
    MP_PATH_FUSED,
    MP_PATH_TC,
)

__all__ = [
    "MagicPIGError", "Shape", "append_token", "append_token_q8", "auto_planes", "codes_bytes", "codes_shape", "decode_attend",
    "decode_attend_noalloc", "decode_attend_q8", "quantize_keys",
    "decode_workspace_bytes", "hash_keys", "hash_keys_range", "hash_queries", "library", "library_path", "read_status",
    "status_string", "PagesShape", "PromptShape", "paged_append", "paged_attend", "paged_workspace_bytes",
    "pages_compact", "pages_copy", "pages_fork", "pages_free", "pages_reserve", "prompt_attend",
]
