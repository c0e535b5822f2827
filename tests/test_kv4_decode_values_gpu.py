"""kv4_attn_decode over values of any magnitude: small ones, and small beside
large ones, keep their weights.  The bound has no absolute floor, so an output
of zeros is outside of it."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv4_ref as R
from kv4_bound import attention_and_bound
from test_kv4_gpu import EPS, batch, device

pytestmark = pytest.mark.gpu

HALF_SUBNORMAL = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def within(pkv, b, **kw):
    """The result is within the bound, and a zero would not be."""
    out = pkv.kv4_attn_decode(**device(b), **kw)
    assert pkv.get_device_error() == 0
    dtype = b["q"].dtype
    want, bound = attention_and_bound(b, EPS[dtype], HALF_SUBNORMAL[dtype])
    err = np.abs(R.to_np(out).astype(np.float64) - want)
    assert np.all(err <= bound), f"{(err > bound).sum()} of {err.size} out of tolerance, worst {(err / bound).max():.1f} of it"
    live = np.asarray(b["lens"]) > 0
    assert (np.abs(want[live]) > bound[live]).mean() > 0.75
    return out


def diffuse(L, Hq, Hkv, D, bs, dtype, values, *, ratio=13.3, every=128, seed=0):
    """Every warp of every partition of 128 tokens or more has a strong token and
    many that weigh 2^-ratio of it; ``values(rng, L, Hkv, D)`` are the value rows."""
    b = batch([L], Hq, Hkv, D, bs, dtype, seed=seed)
    rng = np.random.default_rng(seed + 1)
    t = np.arange(L)
    slots = b["tables"][0, t // bs].astype(np.int64) * bs + t % bs
    # all channels of a key alike: with a query of ones a logit is scale * D * x
    x = np.where(t % every < 128, np.where(t % 32 == 5, 1.0, 0.0), 0.0) * ratio * np.log(2) / (b["scale"] * D)
    R.store(b["kc"], np.broadcast_to(x[:, None, None], (L, Hkv, D)).astype(np.float32), slots, False)
    R.store(b["vc"], values(rng, L, Hkv, D).astype(np.float32), slots, True)
    b["q"] = torch.ones((1, Hq, D), dtype=dtype)
    return b


@pytest.mark.parametrize("mag", [1e-2, 1e-3, 1e-4, 1e-5, 1e-6, 2e-7])
@pytest.mark.parametrize("Hq,D,bs", [(1, 128, 16), (4, 64, 16), (8, 128, 32), (16, 64, 32), (5, 256, 16)])
def test_small_values_keep_their_weights(pkv, mag, Hq, D, bs):
    for L, every, split in ((4096, 128, 4096), (4096, 4096, 4096), (4001, 1024, 1024)):
        b = diffuse(L, Hq, 1, D, bs, torch.bfloat16, lambda r, *n: mag * (1 + 0.3 * r.standard_normal(n)), every=every)
        within(pkv, b, split_tokens=split)


@pytest.mark.parametrize("mag", [1e-1, 1e-2, 1e-3])
def test_small_binary16_values_keep_their_weights(pkv, mag):
    b = diffuse(4096, 4, 1, 128, 16, torch.float16, lambda r, *n: mag * (1 + 0.3 * r.standard_normal(n)), every=4096)
    within(pkv, b, split_tokens=4096)


@pytest.mark.parametrize("Hq,D", [(1, 128), (4, 128), (8, 128), (16, 128), (4, 64), (8, 256)])
def test_channel_groups_of_different_magnitudes(pkv, Hq, D):
    """One group's scale says nothing about another's."""
    def values(r, L, H, D):
        by = np.repeat(np.logspace(3, -6, D // 32), 32)
        return by * (1 + 0.3 * r.standard_normal((L, H, D)))
    for flip in (False, True):
        b = diffuse(4096, Hq, 1, D, 16, torch.bfloat16,
                    (lambda *a: values(*a)[..., ::-1]) if flip else values, every=4096)
        within(pkv, b, split_tokens=4096)


@pytest.mark.parametrize("magnitudes", [(1e4, 1e-5), (1e-5, 1e4), (1e-6, 1.0, 1e-6), (3e4, 1e-3, 10.0, 1e-6)])
@pytest.mark.parametrize("Hq", [2, 8, 16])
def test_stretches_of_different_magnitudes(pkv, magnitudes, Hq):
    """A stretch of large values whose weights are next to nothing takes nothing
    from a stretch of small ones before or behind it."""
    L, D = 4096, 128
    n = len(magnitudes)
    which = np.arange(L) * n // L
    b = diffuse(L, Hq, 1, D, 16, torch.bfloat16,
                lambda r, *s: np.array(magnitudes)[which][:, None, None] * (1 + 0.3 * r.standard_normal(s)), every=4096)
    # the tokens of all but the smallest magnitude: weights of about 2^-58 of the others'
    t = np.arange(L)
    slots = b["tables"][0, t // 16].astype(np.int64) * 16 + t % 16
    k = R.load(b["kc"], slots, False)
    k[np.array(magnitudes)[which] > min(magnitudes)] -= 40.0 / (b["scale"] * D)
    R.store(b["kc"], k.astype(np.float32), slots, False)
    within(pkv, b, split_tokens=4096)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("Hq,Hkv,D,bs", [(8, 2, 128, 16), (2, 2, 256, 32), (10, 1, 64, 16)])
def test_random_batches_within_the_bound(pkv, dtype, Hq, Hkv, D, bs):
    for v_mul in (1.0, 1e-3, 300.0):
        within(pkv, batch([70, 0, 1300, 33, 1], Hq, Hkv, D, bs, dtype, seed=int(D + Hq), v_mul=v_mul))


def test_rows_of_zeros_among_values(pkv):
    """Zero rows (scale 2^-24) in a stage, stages of them, and groups that are always zero."""
    def values(r, L, H, D):
        v = 0.5 * r.standard_normal((L, H, D))
        v[::3] = 0
        v[700:900] = 0
        v[..., 32:64] = 0
        return v
    b = diffuse(2000, 4, 1, 128, 16, torch.bfloat16, values, ratio=3.0, every=2048)
    out = pkv.kv4_attn_decode(**device(b), split_tokens=2048)
    want, bound = attention_and_bound(b, EPS[torch.bfloat16], 2.0 ** -134)
    assert np.all(np.abs(R.to_np(out).astype(np.float64) - want) <= bound) and not bool(out[..., 32:64].any())
