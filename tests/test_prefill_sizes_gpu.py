"""Chunk and prompt attention at the longest sequence that they take, and past it."""
import pytest
import torch

import prefill_ref as R

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
MOST = 1 << 24


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_the_longest_chunk(pkv):
    """A context of one block over and over: attention over that block's keys.  A CTA
    has a 152nd of them, under 2^17, in steps of 16 that are off by two units each in
    FP32: 2^-9 of the weighted values, and as much for all else."""
    g = torch.Generator().manual_seed(1)
    D, bs, n = 64, 32, 3
    q, k, v = (torch.randn((m, h, D), generator=g).to(BF16).cuda() for m, h in ((2 * n, 4), (bs, 1), (bs, 1)))
    kc, vc = (x.transpose(0, 1).unsqueeze(0).contiguous() for x in (k, v))
    tables = torch.zeros((2, MOST // bs + 1), dtype=torch.int32, device="cuda")
    ref, bound = R.attend(q, k, v, 0.2, causal=False)
    bound = bound + 2.0 ** -8 * v.double().abs().amax()
    for lens, code in (([MOST, MOST - 32], 0), ([MOST + 1, MOST], 2), ([MOST, MOST + 32], 2)):
        out = torch.full_like(q, 7.0)
        pkv.paged_attn_chunk(q, kc, vc, tables, _i32(lens), _i32([0, n, 2 * n]), 0.2, out)
        assert pkv.get_device_error() == code
        for i, L in enumerate(lens):
            rows = slice(i * n, i * n + n)
            if L > MOST:
                assert bool((out[rows] == 7).all())
            else:
                R.check(out[rows], ref[rows], bound[rows])


@pytest.mark.parametrize("causal", [True, False])
def test_the_longest_prompt(pkv, causal):
    g = torch.Generator().manual_seed(2)
    D, n, bs = 64, 2, 32
    q, k, v = (torch.randn((m, h, D), generator=g).to(BF16).cuda() for m, h in ((2 * n, 2), (bs, 1), (bs, 1)))
    kk, vv = (x.repeat(MOST // bs + 1, 1, 1) for x in (k, v))
    ref, bound = R.attend(q, k, v, 0.2, causal=False)
    bound = bound + 2.0 ** -8 * v.double().abs().amax()
    for L, code in ((MOST, 0), (MOST + 1, 6)):
        out = torch.full_like(q, 7.0)
        pkv.prompt_attn(q, kk, vv, _i32([0, n, 2 * n]), 0.2, out, key_starts=_i32([0, L, L]), causal=causal)
        assert pkv.get_device_error() == code
        if code:
            assert bool((out[:n] == 7).all())
        else:
            R.check(out[:n], ref[:n], bound[:n])
        assert not bool(out[n:].any())                                # (the second sequence has no keys)
