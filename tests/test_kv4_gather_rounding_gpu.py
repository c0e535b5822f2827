"""kv4_gather's values: s (n + z) rounded once in FP32, and from there to the 16-bit
type, bit for bit."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv4_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [300, 5003])                     # both forms of the kernel
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("low", [1e-5, 1e-3, 0.02, -0.02, 3.0])
def test_values_are_rounded_once_in_fp32(pkv, T, dtype, low):
    """Groups whose smallest value lies just off zero: n + z has up to 28 bits."""
    Hkv, D, bs = 16, 128, 16
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.rand((2, T, Hkv, D), generator=g, device="cuda") * (1 + torch.rand((2, T, Hkv, 1), generator=g, device="cuda"))
    x = (x + low * torch.rand((2, T, Hkv, 1), generator=g, device="cuda")).to(dtype)
    x[..., ::32] = (low * torch.rand((2, T, Hkv, D // 32), generator=g, device="cuda")).to(dtype)
    NB = T // bs + 1
    kc, vc = pkv.kv4_cache(NB, Hkv, bs, D), pkv.kv4_cache(NB, Hkv, bs, D)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    pkv.kv4_append(None, x[0], x[1], None, None, slots, kc, vc)
    for got, cache, values in zip(pkv.kv4_gather(kc, vc, slots, dtype), (kc, vc), (False, True)):
        # the 64-bit values are exact: s has 11 bits, n + z at most 28
        want = R.load(cache.cpu().numpy(), np.arange(T), values).astype(np.float32)
        assert torch.equal(got.cpu(), torch.from_numpy(want).to(dtype))
    assert pkv.get_device_error() == 0
