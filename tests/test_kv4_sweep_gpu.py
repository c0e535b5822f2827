"""The rotation append and the 4-bit cache over seeded random shapes, head_dim 64
and 256 over long contexts, and rows at the ends of their type's range."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv4_ref as R
from kv4_bound import attention_and_bound
from test_kv4_decode_values_gpu import HALF_SUBNORMAL, within
from test_kv4_gpu import EPS, batch, reference_append
from test_rope_append_gpu import assert_rounded, turned

pytestmark = pytest.mark.gpu


# the ring's stages are refilled several times from 600 tokens on, also where a
# partition is cut for each of many CTAs; several partitions run the reduce
@pytest.mark.parametrize("D,bs", [(64, 32), (64, 16), (256, 16), (256, 32), (128, 16)])
@pytest.mark.parametrize("G", [1, 2, 9, 16])
@pytest.mark.parametrize("split", [0, 1024, 4096])
def test_long_contexts(pkv, D, bs, G, split):
    for dtype in (torch.float16, torch.bfloat16):
        b = batch([1, 2999, 640, 0, 1025], G, 1, D, bs, dtype, seed=D + G)
        within(pkv, b, split_tokens=split, max_context_len=3000)


@pytest.mark.parametrize("seed", range(40))
def test_random_session(pkv, seed):
    """Sequences of random lengths appended in chunks of tokens in any order, read
    back, and attended over: 4-bit bytes and 16-bit rows as their references have
    them, values bit for bit, attention within its bound."""
    r = np.random.default_rng(1000 + seed)
    D, bs = int(r.choice([64, 128, 256])), int(r.choice([16, 32]))
    dtype = (torch.float16, torch.bfloat16)[int(r.integers(2))]
    Hkv, G = int(r.choice([1, 2, 3, 5, 8])), int(r.choice([1, 2, 3, 4, 6, 7, 8, 11, 16, 20, 32]))
    while Hkv * G > 64:
        G = max(1, G // 2)
    Hq = Hkv * G
    rot = int(r.choice([0, 16, 48, D // 2, D]))
    inter = bool(r.integers(2))
    lens = np.exp(r.uniform(0, np.log(900), int(r.integers(1, 7)))).astype(np.int32)
    lens[r.random(len(lens)) < 0.2] = 0
    nblk = -(-lens // bs)
    NB = int(nblk.sum()) + int(r.integers(1, 5))
    MB = max(1, int(nblk.max(initial=0)) + int(r.integers(0, 3)))
    perm, at = r.permutation(NB).astype(np.int32), 0
    tables = np.full((len(lens), MB), -1, np.int32)
    slots, pos = [], []
    for i, n in enumerate(nblk):
        tables[i, :n] = perm[at:at + n]
        at += n
        t = np.arange(lens[i])
        slots.append(tables[i, t // bs] * bs + t % bs)
        pos.append(t)
    pads = int(r.integers(0, 9))
    slots = np.concatenate(slots + [np.full(pads, -1 - int(r.integers(0, 1 << 30)))]).astype(np.int32)
    pos = np.concatenate(pos + [np.zeros(pads)]).astype(np.int32)
    order = r.permutation(len(slots))
    slots, pos = slots[order], pos[order]
    table = pkv.rope_table(1000, rot) if rot else None
    g = torch.Generator(device="cuda").manual_seed(seed)
    k4, v4 = (torch.randint(0, 256, (NB, Hkv, bs, D * 5 // 8), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2))
    k16, v16 = (torch.randn((NB, Hkv, bs, D), generator=g, device="cuda").to(dtype) for _ in range(2))
    ek, ev = k4.cpu().numpy(), v4.cpu().numpy()
    before = k16.clone(), v16.clone()
    mul = float(2.0 ** r.integers(-6, 5))
    extra = int(r.choice([0, 8, 24])) if r.integers(2) else None       # channels behind each token's row, or dense rows
    cuts = np.sort(r.integers(0, len(slots) + 1, 2))
    for part in np.split(np.arange(len(slots)), cuts):
        T = len(part)
        w = (Hq + 2 * Hkv) * D
        buf = torch.randn((T, w + (extra or 0)), generator=g, device="cuda").mul_(mul).to(dtype)
        q, k, v = buf[:, :w].unflatten(1, (Hq + 2 * Hkv, D)).split([Hq, Hkv, Hkv], 1)
        if extra is None:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        a = dict(q=q, k=k, v=v, positions=torch.from_numpy(pos[part]).cuda() if rot else None, cos_sin=table,
                 slot_mapping=torch.from_numpy(slots[part]).cuda())
        q4 = pkv.kv4_append(**a, k_cache=k4, v_cache=v4, interleaved=inter)
        q16 = pkv.rope_append(**a, k_cache=k16, v_cache=v16, interleaved=inter)
        assert torch.equal(q4, q16)
        if T == 0:
            continue
        assert_rounded(R.to_np(q16), turned(q, a, inter), R.to_np(q), dtype, "q")
        reference_append(a, ek, ev, inter)
        live = part[slots[part] >= 0]
        s, here = slots[live], np.isin(part, live)
        assert_rounded(R.to_np(k16)[s // bs, :, s % bs], turned(k, a, inter)[here], R.to_np(k)[here], dtype, "k")
        assert np.array_equal(R.to_np(v16)[s // bs, :, s % bs], R.to_np(v)[here])
    assert pkv.get_device_error() == 0
    assert np.array_equal(k4.cpu().numpy(), ek) and np.array_equal(v4.cpu().numpy(), ev)
    rest = torch.ones(NB * bs, dtype=torch.bool, device="cuda")
    rest[torch.from_numpy(slots[slots >= 0].astype(np.int64)).cuda()] = False
    for now, was in ((k16, before[0]), (v16, before[1])):
        assert torch.equal(now.transpose(1, 2).flatten(0, 1)[rest], was.transpose(1, 2).flatten(0, 1)[rest])
    k, v = pkv.kv4_gather(k4, v4, torch.from_numpy(slots).cuda(), dtype)
    live = slots >= 0
    for got, cache, values in ((k, ek, False), (v, ev, True)):
        want = R.load(cache, slots[live], values).astype(np.float32)
        assert torch.equal(got[torch.from_numpy(live).cuda()].cpu(), torch.from_numpy(want).to(dtype))
        assert not bool(got[torch.from_numpy(~live).cuda()].any())
    q = torch.randn((len(lens), Hq, D), generator=g, device="cuda").div_(mul).to(dtype)
    scale = float(np.float32(D ** -0.5)) * (-1 if r.random() < 0.1 else 1)
    split = int(r.choice([0, 0, 16, 200, 1000]))
    out = pkv.kv4_attn_decode(q, k4, v4, torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda(), scale,
                              max_context_len=int(lens.max(initial=1)) or 1, split_tokens=split)
    assert pkv.get_device_error() == 0
    b = dict(q=q.cpu(), kc=ek, vc=ev, tables=tables, lens=lens, scale=scale)
    want, bound = attention_and_bound(b, EPS[dtype], HALF_SUBNORMAL[dtype])
    assert np.all(np.abs(R.to_np(out).astype(np.float64) - want) <= bound)


@pytest.mark.parametrize("dtype,top", [(torch.float16, 65504.0), (torch.bfloat16, 3.38e38), (torch.bfloat16, 5e5)])
@pytest.mark.parametrize("rot", [0, 128])
def test_append_at_the_type_ends(pkv, dtype, top, rot):
    """Groups that span the type from end to end (scales near and at their limit),
    that lie at one end of it, and of its smallest numbers."""
    T, Hkv, D, bs = 40, 2, 128, 16
    r = np.random.default_rng(int(rot))
    x = r.uniform(-1, 1, (2, T, Hkv, D)) * top
    x[:, 0::5, 0] = top * np.sign(r.standard_normal((2, 8, D)))
    x[:, 1::5, 1] = -top
    x[:, 2::5] = top * r.uniform(0.97, 1, (2, 8, Hkv, D))
    x[:, 3::5] = r.integers(-3, 4, (2, 8, Hkv, D)) * (2.0 ** -24 if dtype == torch.float16 else 2.0 ** -133)
    k, v = (torch.from_numpy(y).to(dtype).cuda() for y in x)
    a = dict(q=None, k=k, v=v, cos_sin=pkv.rope_table(64, rot) if rot else None,
             positions=torch.arange(T, dtype=torch.int32, device="cuda") if rot else None,
             slot_mapping=torch.from_numpy(r.permutation(4 * bs)[:T].astype(np.int32)).cuda())
    kc, vc = pkv.kv4_cache(4, Hkv, bs, D), pkv.kv4_cache(4, Hkv, bs, D)
    ek, ev = kc.cpu().numpy(), vc.cpu().numpy()
    with np.errstate(all="ignore"):
        reference_append(a, ek, ev, False)
    pkv.kv4_append(**a, k_cache=kc, v_cache=vc)
    s = a["slot_mapping"].cpu().numpy()
    for got, want, values in ((kc, ek, False), (vc, ev, True)):
        got, want = (R.load(c, s, values) for c in (got.cpu().numpy(), want))
        assert np.array_equal(got, want, equal_nan=True)
        if not (rot and top > 1e38):           # (rotated bfloat16 ends leave FP32, and read as NaN)
            assert np.isfinite(want).all()
