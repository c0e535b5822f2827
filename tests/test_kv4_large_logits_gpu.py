"""kv4_attn_decode with logits of any size that FP32 holds."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv4_ref as R
from kv4_bound import attention_and_bound
from test_kv4_decode_values_gpu import HALF_SUBNORMAL
from test_kv4_gpu import EPS, batch, device

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("Hq,D", [(2, 128), (8, 128), (24, 128), (8, 64), (2, 256)])
@pytest.mark.parametrize("mag", [10.0, 1e3, 3e4])
def test_large_logits(pkv, dtype, Hq, D, mag):
    """Queries and keys of ``mag``, logits up to 10^11: the tokens whose logits are
    the largest beyond FP32's rounding share the weight."""
    b = batch([700, 33, 1], Hq, 2, D, 16, dtype, seed=int(mag) + D + Hq, k_mul=mag)
    b["q"] = (b["q"].float() * mag).clamp(-6e4, 6e4).to(dtype)
    for split in (0, 64):
        out = pkv.kv4_attn_decode(**device(b), split_tokens=split)
        assert pkv.get_device_error() == 0
        got = R.to_np(out).astype(np.float64)
        assert np.isfinite(got).all()
        for i, L in enumerate(b["lens"]):
            t = np.arange(L)
            slots = b["tables"][i, t // 16].astype(np.int64) * 16 + t % 16
            k, v = R.load(b["kc"], slots, False), R.load(b["vc"], slots, True)
            size = R._magnitudes(b["kc"], slots)
            for h in range(Hq):
                q, g = R.to_np(b["q"][i, h]).astype(np.float64), h // (Hq // 2)
                a = b["scale"] * (k[:, g] @ q)
                # FP32's error of a logit (kv4_ref.attention's steps), from which the
                # others must be further apart than the bits of a weight
                off = b["scale"] * (D / 8 + 8) * 2.0 ** -24 * (size[:, g] @ np.abs(q)).max()
                near = a >= a.max() - 2 * off - 30
                if near.sum() > 1:
                    lo, hi = v[near, g].min(0), v[near, g].max(0)
                else:
                    lo = hi = v[near, g][0]
                room = 2.0 ** -8 * np.abs(v[near, g]).max(0) + 2.0 ** -9 * np.abs(v[:, g]).max()
                assert np.all(got[i, h] >= lo - room) and np.all(got[i, h] <= hi + room)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("Hq,D", [(1, 128), (4, 128), (8, 64), (16, 128), (3, 256)])
@pytest.mark.parametrize("span", [20.0, 400.0, 4000.0])
def test_logits_that_grow_along_a_sequence(pkv, dtype, Hq, D, span):
    """The reference moves at nearly every stage, or at the first alone."""
    L = 3000
    for down in (False, True):
        b = batch([L, 45], Hq, 1, D, 16, dtype, seed=Hq + D)
        t = np.arange(L)
        slots = b["tables"][0, t // 16].astype(np.int64) * 16 + t % 16
        x = (t[::-1] if down else t) / L * span - 0.7 * span + np.random.default_rng(1).standard_normal(L)
        k = np.broadcast_to((x / (b["scale"] * D))[:, None, None], (L, 1, D))
        R.store(b["kc"], k.astype(np.float32), slots, False)
        b["q"][0] = 1
        for split in (0, 1024):
            out = pkv.kv4_attn_decode(**device(b), split_tokens=split)
            want, bound = attention_and_bound(b, EPS[dtype], HALF_SUBNORMAL[dtype])
            assert np.all(np.abs(R.to_np(out).astype(np.float64) - want) <= bound)
