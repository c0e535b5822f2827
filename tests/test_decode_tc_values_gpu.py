"""The tcgen05 decode kernel with values at bfloat16's end."""
import pytest
import torch

import prefill_ref as R

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.mark.parametrize("G", [8, 16, 32])
@pytest.mark.parametrize("split", [0, 128])
@pytest.mark.parametrize("later", [0.0, 2.0, 5.4])
@pytest.mark.parametrize("kernel", [0, 3])
def test_values_at_the_types_end(pkv, G, split, later, kernel):
    """A few later keys above the first ones by less than makes the maximum follow:
    results are finite where the weights' sum (the largest as 1) times the values is."""
    g = torch.Generator().manual_seed(G)
    L, hkv, D, bs = 240, 2, 128, 16
    q, k = torch.zeros((1, G * hkv, D)), torch.zeros((L, hkv, D))
    q[..., 3] = 1
    k[..., 3] = -30.0
    k[:5, :, 3] = 0.0
    k[[150, 151, 170, 190, 201, 230], :, 3] = later
    v = 3e36 * (1 - 0.1 * torch.rand((L, hkv, D), generator=g))
    q, k, v = q.to(BF16).cuda(), k.to(BF16).cuda(), v.to(BF16).cuda()
    kc, vc, tables = R.paged(k, v, [L], bs, g)
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    out = pkv.paged_attn_decode(q, kc.cuda(), vc.cuda(), tables.cuda(), lens, 1.0, split_tokens=split, kernel=kernel)
    ref, bound = R.attend(q, k, v, 1.0)
    assert pkv.get_device_error() == 0
    R.check(out, ref, bound)
