"""GPU parity of rope_append (rotation and append into the 16-bit cache) against
the definition in 64 bits, with untouched slots bit-exact."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv4_ref as R

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def make(T, Hq, Hkv, D, bs, dtype, rot, *, seed=0, fused=False, base=0, pad=0):
    """Inputs on the GPU: rows, positions in any order, distinct slots."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    x = torch.randn((T, Hq + 2 * Hkv, D), generator=g).to(dtype).cuda()
    q, k, v = x.split([Hq, Hkv, Hkv], 1)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    NB = (T + bs - 1) // bs + 3
    slots = rng.permutation(NB * bs)[:T].astype(np.int32)
    if pad:
        slots[rng.permutation(T)[:pad]] = -1 - rng.integers(0, 9)
    pos = (base + rng.permutation(T)).astype(np.int32)
    from paged_kv_cache_268_gb300 import rope_table
    table = rope_table(base + T, rot, device="cuda") if rot else None
    return dict(q=q, k=k, v=v, positions=torch.from_numpy(pos).cuda() if rot else None, cos_sin=table,
                slot_mapping=torch.from_numpy(slots).cuda()), NB


def turned(x, a, inter):
    """The rows rotated in 64 bits."""
    if a["cos_sin"] is None:
        return R.to_np(x).astype(np.float64)
    return R.rotate(R.to_np(x), a["cos_sin"].cpu().numpy(), a["positions"].cpu().numpy(), inter, np.float64)


def assert_rounded(got, want, x, dtype, what):
    """One rounding to dtype (half a step of the result, or half of binary16's
    smallest step) after two products and a sum in FP32 of magnitude at most
    |a| + |b| <= 2 max |row|: 2^-24 each, relative."""
    top = np.abs(x).max(-1, keepdims=True)
    bound = HALF_STEP[dtype] * np.abs(want) + 2.0 ** -25 + 3 * 2.0 ** -24 * 2 * top
    bad = np.abs(got - want) > bound
    assert not bad.any(), f"{what}: {bad.sum()} elements out of tolerance"


CASES = [
    # T, Hq, Hkv, D, bs, dtype, rot, interleaved, fused, base, pad
    (1, 1, 1, 64, 16, torch.float16, 64, False, False, 0, 0),
    (1, 8, 2, 128, 16, torch.bfloat16, 128, True, True, 7, 0),
    (2, 5, 5, 256, 32, torch.float16, 256, False, False, 0, 1),
    (7, 3, 1, 64, 32, torch.bfloat16, 16, False, True, 0, 2),
    (33, 32, 8, 128, 16, torch.float16, 128, False, True, 100000, 5),
    (33, 32, 8, 128, 16, torch.bfloat16, 48, False, False, 0, 0),
    (33, 7, 7, 128, 32, torch.bfloat16, 64, True, True, 0, 33),
    (130, 16, 16, 256, 16, torch.float16, 80, True, False, 3, 11),
    (1500, 12, 3, 64, 16, torch.float16, 32, False, True, 0, 100),
    (1025, 9, 1, 128, 32, torch.bfloat16, 112, False, True, 0, 0),
    (40, 4, 4, 128, 16, torch.float16, 0, False, True, 0, 3),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,bs,dtype,rot,inter,fused,base,pad", CASES)
def test_rotation_and_append(pkv, T, Hq, Hkv, D, bs, dtype, rot, inter, fused, base, pad):
    a, NB = make(T, Hq, Hkv, D, bs, dtype, rot, seed=T, fused=fused, base=base, pad=pad)
    kc = torch.full((NB, Hkv, bs, D), float("nan"), dtype=dtype, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    before = kc.view(torch.int16).cpu().numpy().copy()
    inputs = [t.clone() for t in (a["q"], a["k"], a["v"])]
    q = pkv.rope_append(**a, k_cache=kc, v_cache=vc, interleaved=inter)
    assert pkv.get_device_error() == 0
    assert all(torch.equal(t, u) for t, u in zip(inputs, (a["q"], a["k"], a["v"])))
    assert_rounded(R.to_np(q), turned(a["q"], a, inter), R.to_np(a["q"]), dtype, "q")
    slots = a["slot_mapping"].cpu().numpy()
    live = slots >= 0
    s = slots[live]
    k_want = turned(a["k"], a, inter)[live]
    assert_rounded(R.to_np(kc)[s // bs, :, s % bs], k_want, R.to_np(a["k"])[live], dtype, "k")
    vb = a["v"].contiguous().view(torch.int16).cpu().numpy()
    for cache, rows in ((kc, None), (vc, vb[live])):
        got = cache.view(torch.int16).cpu().numpy()
        if rows is not None:
            assert np.array_equal(got[s // bs, :, s % bs], rows)       # values: bit for bit
        rest = np.ones((NB, bs), bool)
        rest[s // bs, s % bs] = False
        assert np.array_equal(got.swapaxes(1, 2)[rest], before.swapaxes(1, 2)[rest])
    if rot == 0:
        assert torch.equal(q, a["q"])


def test_in_place_and_given_output(pkv):
    a, NB = make(19, 8, 2, 128, 16, torch.bfloat16, 128, seed=3)
    kc = torch.zeros((NB, 2, 16, 128), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    want = pkv.rope_append(**a, k_cache=kc, v_cache=vc)
    out = torch.empty_like(want)
    assert pkv.rope_append(**a, k_cache=kc, v_cache=vc, q_out=out) is out and torch.equal(out, want)
    q = a["q"].clone()
    assert pkv.rope_append(**dict(a, q=q), k_cache=kc, v_cache=vc, q_out=q) is q and torch.equal(q, want)
    k0 = kc.clone()
    assert pkv.rope_append(**dict(a, q=None), k_cache=kc.zero_(), v_cache=vc) is None
    assert torch.equal(kc, k0)                                          # keys only


def test_bad_positions_and_slots(pkv):
    a, NB = make(6, 4, 2, 64, 16, torch.float16, 64, seed=1)
    kc = torch.zeros((NB, 2, 16, 64), dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc)
    good = pkv.rope_append(**a, k_cache=kc, v_cache=vc)
    k0 = kc.clone()
    for bad in (-1, 6, 2 ** 31 - 1, -2 ** 31):
        pos = a["positions"].clone()
        pos[2] = bad
        q_out = torch.full_like(good, 7.0)
        kc.zero_()
        pkv.rope_append(**dict(a, positions=pos), k_cache=kc, v_cache=vc, q_out=q_out)
        assert pkv.get_device_error() == 5
        s = int(a["slot_mapping"][2])
        assert not kc[s // 16, :, s % 16].any() and bool((q_out[2] == 7).all())
        keep = torch.tensor([0, 1, 3, 4, 5], device="cuda")
        assert torch.equal(q_out[keep], good[keep])
    for bad in (NB * 16, 2 ** 31 - 1):
        slots = a["slot_mapping"].clone()
        slots[1] = bad
        kc.zero_()
        q = pkv.rope_append(**dict(a, slot_mapping=slots), k_cache=kc, v_cache=vc)
        assert pkv.get_device_error() == 3
        s = int(a["slot_mapping"][1])
        assert torch.equal(q, good) and not kc[s // 16, :, s % 16].any()
        k1 = k0.clone()
        k1[s // 16, :, s % 16] = 0
        assert torch.equal(kc, k1)
    empty = {n: t[:0] if n != "cos_sin" else t for n, t in a.items()}
    assert pkv.rope_append(**empty, k_cache=kc, v_cache=vc).shape == (0, 4, 64)


@pytest.mark.parametrize("T", [5, 2000])
def test_graph_replay_and_other_stream(pkv, T):
    a, NB = make(T, 8, 4, 128, 16, torch.float16, 64, seed=9, fused=True)
    kc = torch.zeros((NB, 4, 16, 128), dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc)
    want = pkv.rope_append(**a, k_cache=kc, v_cache=vc)
    k0 = kc.clone()
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.rope_append(**a, k_cache=kc, v_cache=vc, q_out=out)
    kc.zero_()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(kc, k0)
    st = torch.cuda.Stream()
    kc.zero_()
    st.wait_stream(torch.cuda.current_stream())
    got = pkv.rope_append(**a, k_cache=kc, v_cache=vc, stream=st)
    st.synchronize()
    assert torch.equal(got, want) and torch.equal(kc, k0)


def test_same_rows_as_kv_cache_append_without_rotation(pkv):
    """rot_dim 0 stores what kv_cache_append stores."""
    a, NB = make(300, 8, 4, 64, 32, torch.bfloat16, 0, seed=5, pad=20)
    caches = [torch.zeros((NB, 4, 32, 64), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    pkv.rope_append(**a, k_cache=caches[0], v_cache=caches[1])
    pkv.kv_cache_append(a["k"], a["v"], a["slot_mapping"], caches[2], caches[3])
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])


def test_pool_past_32_bit_offsets(pkv):
    """A pool of more than 2^32 bytes: the last block of it."""
    NB, Hkv, bs, D = 40000, 16, 32, 128                    # 5.2 GB a cache
    kc = torch.zeros((NB, Hkv, bs, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    a, _ = make(bs, 16, Hkv, D, bs, torch.bfloat16, 128, seed=2)
    a["slot_mapping"] = torch.arange((NB - 1) * bs, NB * bs, dtype=torch.int32, device="cuda")
    pkv.rope_append(**a, k_cache=kc, v_cache=vc)
    assert torch.equal(vc[-1], a["v"].transpose(0, 1))
    assert_rounded(R.to_np(kc[-1].transpose(0, 1)), turned(a["k"], a, False), R.to_np(a["k"]),
                   torch.bfloat16, "k")
    assert not bool(kc[:64].any()) and not bool(vc[:64].any())
