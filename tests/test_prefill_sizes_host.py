"""Chunk and prompt attention: sizes that the waits of the kernel do not bear are
refused (no call here reaches a GPU)."""
import ctypes

import pytest

from paged_kv_cache_268_gb300 import _binding as B
from paged_kv_cache_268_gb300 import build

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.load_library()


def test_very_many_sequences_are_refused(lib):
    n = ctypes.c_size_t(0)
    for B_, code in ((1 << 24, 0), ((1 << 24) + 1, -3)):
        shape = B.make_shape(num_seqs=B_, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16, num_blocks=64,
                             max_blocks_per_seq=8, max_context_len=100, dtype=0)
        # (no rows: nothing to do)
        assert lib.pkv_paged_attn_chunk(ctypes.byref(shape), FAKE, 0, 0, FAKE, FAKE, FAKE, FAKE, FAKE, 0.1, FAKE, None,
                                        0, None) == code
        prompt = B.Prompt(B_, 8, 2, 128, 0, 5, 0, 1, 0, 0, 0, 0)
        assert lib.pkv_prompt_attn(ctypes.byref(prompt), FAKE, FAKE, FAKE, FAKE, FAKE, 0.1, FAKE, None, 0, None) == code
        if code:
            assert lib.pkv_chunk_workspace_bytes(ctypes.byref(shape), 5, ctypes.byref(n)) == code
            assert lib.pkv_prompt_workspace_bytes(ctypes.byref(prompt), ctypes.byref(n)) == code
