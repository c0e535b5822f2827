"""copy_blocks takes uint8 pools only where they are 4-bit caches."""
import pytest
import torch

from paged_kv_cache_268_gb300 import _binding as B
from test_kv4_host import _c


def _copy(*shapes, dtype=torch.uint8):
    B.copy_blocks(*(_c(*s, dtype=dtype) for s in shapes), _c(1, 2, dtype=torch.int32))


@pytest.mark.parametrize("shape", [
    (4, 2, 16, 64), (4, 2, 16, 128), (4, 2, 16, 82), (4, 2, 16, 41), (4, 2, 16, 20), (4, 2, 16, 320),   # no 5D/8
    (4, 2, 8, 80), (4, 2, 64, 80), (4, 2, 1, 1280),                                                     # no block size
])
def test_other_bytes_are_refused(shape):
    with pytest.raises(ValueError):
        _copy(*[shape] * 4)


def test_pools_that_do_not_fit_are_refused():
    a = (4, 2, 16, 80)
    for bad in ((4, 3, 16, 80), (4, 2, 32, 80), (4, 2, 16, 40), (4, 2, 1280)):
        for i in range(4):
            with pytest.raises(ValueError):
                _copy(*[bad if j == i else a for j in range(4)])
    with pytest.raises(ValueError):
        B.copy_blocks(_c(*a, dtype=torch.uint8), _c(*a, dtype=torch.uint8), _c(4, 2, 16, 80), _c(4, 2, 16, 80),
                      _c(1, 2, dtype=torch.int32))


@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("W", [40, 80, 160])
def test_a_block_is_one_row_of_16_bit_elements(W, bs):
    pool = torch.arange(3 * 2 * bs * W).to(torch.uint8).view(3, 2, bs, W)
    rows = B._kv4_as_rows(pool)
    assert rows.shape == (3, 2, 1, bs * W // 2) and rows.data_ptr() == pool.data_ptr()
    assert torch.equal(rows.view(torch.uint8).flatten(), pool.flatten())
