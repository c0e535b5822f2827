"""Chunk and prompt attention with values at bfloat16's end."""
import pytest
import torch

import prefill_ref as R

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("split", [0, 128])
@pytest.mark.parametrize("later", [0.0, 2.0, 5.4])
def test_values_at_the_types_end(pkv, D, split, later):
    """A few later keys above the first ones by less than makes the reference follow:
    results are finite where the weights' sum (the largest as 1) times the values is."""
    g = torch.Generator().manual_seed(D)
    n, L, hq, hkv = 40, 700, 4, 2
    q, k = torch.zeros((n, hq, D)), torch.zeros((L, hkv, D))
    q[..., 3] = 1
    k[..., 3] = -9.0
    k[:5, :, 3] = 0.0
    k[[300, 301, 460, 555, 600, 640], :, 3] = later
    v = 3e37 * (1 - 0.1 * torch.rand((L, hkv, D), generator=g))
    q, k, v = q.to(BF16).cuda(), k.to(BF16).cuda(), v.to(BF16).cuda()
    out = pkv.prompt_attn(q, k, v, _i32([0, n]), 1.0, key_starts=_i32([0, L]), split_tokens=split)
    ref, bound = R.attend(q, k, v, 1.0)
    R.check(out, ref, bound)
