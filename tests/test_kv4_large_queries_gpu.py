"""kv4_attn_decode with queries up to bfloat16's largest: logits that FP32 holds
give their softmax, not NaN."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv4_ref as R
from test_kv4_gpu import batch, check, device

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,D", [(2, 128), (6, 128), (16, 128), (4, 64), (8, 256)])
@pytest.mark.parametrize("mag", [1e30, 3e36, 3e38])
@pytest.mark.parametrize("sign", [1, -1])
def test_large_queries(pkv, Hq, D, mag, sign):
    L = 300
    b = batch([L, 40], Hq, 2, D, 16, torch.bfloat16, seed=Hq + D)
    b["scale"] *= sign
    t = np.arange(L)
    slots = b["tables"][0, t // 16].astype(np.int64) * 16 + t % 16
    small = torch.from_numpy(np.random.default_rng(0).standard_normal((1, Hq, D)).astype(np.float32)).bfloat16()
    # all keys zero: the values' mean, whatever the query
    R.store(b["kc"], np.zeros((L, 2, D), np.float32), slots, False)
    b["q"][0], b["q"][1] = 0, small[0]
    mean = check(pkv, b)
    b["q"][0] = mag
    assert torch.equal(check(pkv, b), mean)
    # one key of small channels takes all the weight (or none, where the scale is negative)
    k = np.zeros((L, 2, D), np.float32)
    k[123] = 1e-5
    R.store(b["kc"], k, slots, False)
    out = check(pkv, b)
    v = torch.from_numpy(R.load(b["vc"], slots, True)[123].repeat(Hq // 2, 0)).to(out.device)
    if sign > 0:
        assert bool(((out[0].double() - v).abs() <= 2.0 ** -8 * v.abs() + 1e-30).all())
    # ordinary heads beside a large one keep their results
    b["q"][0] = small[0]
    good = check(pkv, b)
    d = device(b)
    d["q"][0, 1] = mag
    got = pkv.kv4_attn_decode(**d)
    assert bool(torch.isfinite(got).all())
    rest = [h for h in range(Hq) if h != 1]
    assert torch.equal(got[:, rest], good[:, rest])


@pytest.mark.parametrize("mag", [1e-38, 1e-30])
def test_small_queries_with_a_large_scale(pkv, mag):
    """The scale times the query's power of two leaves FP32's normal numbers only where both are small."""
    b = batch([200], 4, 1, 128, 16, torch.bfloat16, seed=1)
    b["q"] = (b["q"].float() * mag).to(torch.bfloat16)
    b["scale"] = float(np.float32(0.1 / mag))
    check(pkv, b)
    b["q"] = (b["q"].float() * 1e-6).to(torch.bfloat16)      # weights all alike
    b["scale"] = 2.0 ** -100
    check(pkv, b)
