"""Paged KV-cache attention, prompts and decode, for GB300 (sm_103a).

The compute lives in ``lib/libpkv.so`` (hand-written CUDA behind the C ABI in
``include/pkv.h``); this package is a thin ctypes binding over it, plus the
seeded workload generator used by the tests and the benchmark.  Build the
library with ``python -m paged_kv_cache_268_gb300.build``.
"""
from ._binding import (  # noqa: F401
    BlockManager,
    PkvError,
    copy_blocks,
    alloc_workspace,
    chunk_shape,
    chunk_workspace_bytes,
    decode_plan,
    decode_shape,
    decode_step,
    get_device_error,
    kv4_append,
    kv4_attn_decode,
    kv4_cache,
    kv4_decode_plan,
    kv4_decode_shape,
    kv4_gather,
    kv4_workspace_bytes,
    kv_cache_append,
    launch_count,
    load_library,
    paged_attn_chunk,
    paged_attn_decode,
    prompt_attn,
    prompt_shape,
    prompt_workspace_bytes,
    rope_append,
    rope_table,
    selftest_wait_timeout,
    set_workspace,
    workspace_bytes,
)
