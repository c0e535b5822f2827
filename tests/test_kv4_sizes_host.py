"""Sizes that the C structs could not hold, and tables of an odd width, are refused."""
import pytest
import torch

from paged_kv_cache_268_gb300 import _binding as B
from test_kv4_host import _args, _c


@pytest.mark.parametrize("kw", [dict(max_context_len=2 ** 32 + 20), dict(max_context_len=2 ** 31),
                                dict(max_context_len=20, split_tokens=2 ** 32 + 16), dict(max_context_len=-2 ** 32 + 20)])
def test_sizes_past_32_bits_are_refused(kw):
    a = _args(True)
    call = dict(q=_c(3, 4, 64), k_cache=a["k_cache"], block_tables=_c(3, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        B.kv4_decode_shape(**call, **kw)
    good = B.kv4_decode_shape(**call, max_context_len=20, split_tokens=16)
    assert (good.max_context_len, good.split_tokens) == (20, 16)


def test_rope_table_refuses_an_odd_width():
    for rot in (15, 1, -2):
        with pytest.raises(ValueError):
            B.rope_table(8, rot, device="cpu")
    assert B.rope_table(8, 16, device="cpu").shape == (8, 16) and B.rope_table(8, 0, device="cpu").shape == (8, 0)
