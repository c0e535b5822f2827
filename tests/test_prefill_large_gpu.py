"""Chunk and prompt attention with logits of any size that FP32 holds."""
import pytest
import torch

import prefill_ref as R

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("log2", [12, 20, 27, 31, 38, 60, 120])
@pytest.mark.parametrize("split", [0, 128])
def test_the_largest_logit_takes_all(pkv, D, dt, log2, split):
    """A logit is one product, exact in FP32, and two of them are equal or at least
    2^log2 / 2^11 apart: a row is the mean of the values of its largest, as far as
    their roundings let it be (one of the weights, one of the sum, one of the store)."""
    if dt is F16 and log2 > 31:
        pytest.skip("past binary16's products")
    g = torch.Generator().manual_seed(D + log2)
    n, L, hq, hkv = 70, 900, 6, 2
    up = log2 // 2 if dt is F16 else log2 - 4
    q, k = torch.zeros((n, hq, D)), torch.zeros((L, hkv, D))
    q[..., 5] = 2.0 ** min(up, 15 if dt is F16 else up)
    step = 2.0 ** log2 / q[0, 0, 5] / 128                              # 8 bits of a key at most: exact in both types
    k[..., 5] = torch.randint(1, 128, (L, hkv), generator=g).float() * step
    v = torch.randn((L, hkv, D), generator=g)
    q, k, v = q.to(dt).cuda(), k.to(dt).cuda(), v.to(dt).cuda()
    out = pkv.prompt_attn(q, k, v, _i32([0, n]), 1.0, key_starts=_i32([0, L]), split_tokens=split).double()
    assert pkv.get_device_error() == 0
    a = k[:, :, 5].double().repeat_interleave(hq // hkv, 1)            # [L, hq]
    seen = torch.arange(L, device="cuda")[None] <= L - n + torch.arange(n, device="cuda")[:, None]
    a = torch.where(seen[..., None], a[None], -1.0)                    # [n, L, hq]
    w = (a == a.amax(1, keepdim=True)).double()
    w /= w.sum(1, keepdim=True)
    vv = v.double().repeat_interleave(hq // hkv, 1)
    ref, A = torch.einsum("nlh,lhd->nhd", w, vv), torch.einsum("nlh,lhd->nhd", w, vv.abs())
    u = R.HALF[dt]
    assert bool(((out - ref).abs() <= u * ref.abs() + A * (u + 2.0 ** -18) + 2.0 ** -24).all())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("far", [300.0, 680.0, 720.0, 2000.0, -720.0, -20000.0])
def test_logits_far_from_zero(pkv, D, dt, far):
    """All logits of a row lie about one far value: what tells them apart is a few
    units of it.  Cut and whole."""
    g = torch.Generator().manual_seed(D)
    n, L, hq, hkv = 60, 1500, 4, 2
    q, k, v = (torch.randn((m, h, D), generator=g) for m, h in ((n, hq), (L, hkv), (L, hkv)))
    q[..., 0], k[..., 0] = 32.0, far * D ** 0.5 / 32
    k[..., 0] += (torch.arange(L) // 128 % 3)[:, None] * 0.25          # the key tiles differ
    q, k, v = q.to(dt).cuda(), k.to(dt).cuda(), v.to(dt).cuda()
    ref, bound = R.attend(q, k, v, D ** -0.5)
    for split in (0, 128):
        out = pkv.prompt_attn(q, k, v, _i32([0, n]), D ** -0.5, key_starts=_i32([0, L]), split_tokens=split)
        R.check(out, ref, bound)
    assert pkv.get_device_error() == 0
