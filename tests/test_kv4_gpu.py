"""GPU parity of the 4-bit cache: kv4_append byte for byte against the format's
reference, kv4_gather against its values, kv4_attn_decode against attention in
64 bits over the same bytes."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv4_ref as R
from test_rope_append_gpu import CASES, HALF_STEP, make

pytestmark = pytest.mark.gpu

EPS = {torch.float16: 2.0 ** -10, torch.bfloat16: 2.0 ** -7}


# ---------------------------------------------------------------- append
def reference_append(a, kc, vc, inter):
    k = R.to_np(a["k"])
    if a["cos_sin"] is not None:
        k = R.rotate(k, a["cos_sin"].cpu().numpy(), a["positions"].cpu().numpy(), inter)
    slots = a["slot_mapping"].cpu().numpy()
    R.store(kc, k, slots, False)
    R.store(vc, R.to_np(a["v"]), slots, True)


@pytest.mark.parametrize("T,Hq,Hkv,D,bs,dtype,rot,inter,fused,base,pad", CASES)
def test_append_writes_the_format_byte_for_byte(pkv, T, Hq, Hkv, D, bs, dtype, rot, inter, fused,
                                                base, pad):
    a, NB = make(T, Hq, Hkv, D, bs, dtype, rot, seed=T + 1, fused=fused, base=base, pad=pad)
    g = torch.Generator(device="cuda").manual_seed(T)
    kc, vc = (torch.randint(0, 256, (NB, Hkv, bs, D * 5 // 8), generator=g, device="cuda", dtype=torch.uint8)
              for _ in range(2))
    ek, ev = kc.cpu().numpy(), vc.cpu().numpy()
    reference_append(a, ek, ev, inter)
    q = pkv.kv4_append(**a, k_cache=kc, v_cache=vc, interleaved=inter)
    assert pkv.get_device_error() == 0
    assert np.array_equal(kc.cpu().numpy(), ek)
    assert np.array_equal(vc.cpu().numpy(), ev)
    c16 = torch.zeros((NB, Hkv, bs, D), dtype=dtype, device="cuda")
    assert torch.equal(q, pkv.rope_append(**a, k_cache=c16, v_cache=c16.clone(), interleaved=inter))


@pytest.mark.parametrize("what", ["small", "large", "offset", "constant", "zero", "nan", "inf", "huge"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_append_of_extreme_rows(pkv, what, dtype):
    a, NB = make(50, 4, 4, 128, 16, dtype, 128, seed=8)
    for n in ("k", "v"):
        x = a[n]
        if what == "small":
            x *= 2.0 ** -15
        elif what == "large":
            x *= 8000.0
        elif what == "offset":
            x += 50.0
        elif what == "constant":
            x.fill_(-3.25)
        elif what == "zero":
            x.zero_()
        elif what in ("nan", "inf"):
            x[::3, 1, ::37] = float(what)
            x[1::3, 2, 5] = -float(what)
        elif dtype == torch.bfloat16:
            x *= 1e37
    kc = torch.zeros((NB, 4, 16, 80), dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    ek, ev = kc.cpu().numpy(), vc.cpu().numpy()
    with np.errstate(all="ignore"):
        reference_append(a, ek, ev, False)
    pkv.kv4_append(**a, k_cache=kc, v_cache=vc)
    for got, want, values in ((kc, ek, False), (vc, ev, True)):
        # the NaN's own bits may be any: compare what the bytes stand for
        s = a["slot_mapping"].cpu().numpy()
        assert np.array_equal(R.load(got.cpu().numpy(), s, values), R.load(want, s, values), equal_nan=True)


def test_append_refuses_on_the_device(pkv):
    a, NB = make(6, 4, 2, 64, 16, torch.float16, 64, seed=1)
    kc = pkv.kv4_cache(NB, 2, 16, 64)
    vc = pkv.kv4_cache(NB, 2, 16, 64)
    pos = a["positions"].clone()
    pos[0] = 6
    pkv.kv4_append(**dict(a, positions=pos), k_cache=kc, v_cache=vc)
    assert pkv.get_device_error() == 5
    slots = a["slot_mapping"].clone()
    slots.fill_(NB * 16)
    kc.zero_()
    pkv.kv4_append(**dict(a, slot_mapping=slots), k_cache=kc, v_cache=vc)
    assert pkv.get_device_error() == 3 and not bool(kc.any())


# ---------------------------------------------------------------- gather
@pytest.mark.parametrize("T,Hkv,D,bs,dtype", [
    (1, 1, 64, 16, torch.float16), (3, 5, 256, 32, torch.bfloat16), (129, 8, 128, 16, torch.bfloat16),
    (1000, 3, 64, 32, torch.float16), (77, 16, 128, 32, torch.float16), (40, 2, 256, 16, torch.bfloat16),
    # enough rows for the form of four tokens a CTA
    (19467, 3, 64, 16, torch.bfloat16), (3895, 20, 128, 32, torch.float16), (6491, 5, 256, 16, torch.float16)])
def test_gather(pkv, T, Hkv, D, bs, dtype):
    a, NB = make(T, 1, Hkv, D, bs, dtype, 0, seed=T, pad=T // 5)
    kc, vc = pkv.kv4_cache(NB, Hkv, bs, D), pkv.kv4_cache(NB, Hkv, bs, D)
    pkv.kv4_append(**dict(a, q=None), k_cache=kc, v_cache=vc)
    slots = a["slot_mapping"].cpu().numpy()
    k, v = pkv.kv4_gather(kc, vc, a["slot_mapping"], dtype)
    assert pkv.get_device_error() == 0
    for got, cache, values in ((k, kc, False), (v, vc, True)):
        got, live = R.to_np(got).astype(np.float64), slots >= 0
        want = R.load(cache.cpu().numpy(), slots[live], values)
        # the product is rounded once in FP32 and once to 16 bits
        assert np.all(np.abs(got[live] - want) <= (HALF_STEP[dtype] + 2.0 ** -23) * np.abs(want) + 2.0 ** -25)
        assert not got[~live].any()
    # repeated slots, another order, given outputs
    twice = torch.cat([a["slot_mapping"].flip(0), a["slot_mapping"]])
    k2, v2 = torch.empty((2 * T, Hkv, D), dtype=dtype, device="cuda"), torch.empty((2 * T, Hkv, D), dtype=dtype, device="cuda")
    r = pkv.kv4_gather(kc, vc, twice, dtype, k2, v2)
    assert r[0] is k2 and r[1] is v2
    assert torch.equal(k2, torch.cat([k.flip(0), k])) and torch.equal(v2, torch.cat([v.flip(0), v]))
    bad = a["slot_mapping"].clone()
    bad[0] = NB * bs
    k3, _ = pkv.kv4_gather(kc, vc, bad, dtype)
    assert pkv.get_device_error() == 3 and not bool(k3[0].any()) and torch.equal(k3[1:], k[1:])


# ---------------------------------------------------------------- decode
def batch(lens, Hq, Hkv, D, bs, dtype, *, seed=0, k_mul=1.0, v_mul=1.0, v_add=0.0, poison=True):
    """A decode batch over 4-bit caches whose other bytes are noise (their
    scales decode to anything, NaN among it)."""
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int32)
    nblk = -(-lens // bs)
    NB = int(nblk.sum()) + 5
    MB = max(1, int(nblk.max(initial=1))) + 1
    tables, perm, at = np.full((len(lens), MB), -1, np.int32), rng.permutation(NB), 0
    for i, n in enumerate(nblk):
        tables[i, :n] = perm[at:at + n]
        at += n
    shape = (NB, Hkv, bs, D * 5 // 8)
    kc = rng.integers(0, 256, shape, dtype=np.uint8) if poison else np.zeros(shape, np.uint8)
    vc = rng.integers(0, 256, shape, dtype=np.uint8) if poison else np.zeros(shape, np.uint8)
    for i, L in enumerate(lens):
        t = np.arange(L)
        slots = tables[i, t // bs] * bs + t % bs
        R.store(kc, (rng.standard_normal((L, Hkv, D)) * k_mul).astype(np.float32), slots, False)
        R.store(vc, (rng.standard_normal((L, Hkv, D)) * v_mul + v_add).astype(np.float32), slots, True)
    q = torch.from_numpy(rng.standard_normal((len(lens), Hq, D)).astype(np.float32)).to(dtype)
    return dict(q=q, kc=kc, vc=vc, tables=tables, lens=lens, scale=float(np.float32(D ** -0.5)))


def device(b):
    return dict(q=b["q"].cuda(), k_cache=torch.from_numpy(b["kc"]).cuda(), v_cache=torch.from_numpy(b["vc"]).cuda(),
                block_tables=torch.from_numpy(b["tables"]).cuda(), context_lens=torch.from_numpy(b["lens"]).cuda(),
                scale=b["scale"])


def check(pkv, b, d=None, **kw):
    d = d or device(b)
    out = pkv.kv4_attn_decode(**d, **kw)
    assert pkv.get_device_error() == 0
    want, mag, low, smag = R.attention(R.to_np(b["q"]), b["kc"], b["vc"], b["tables"], b["lens"], b["scale"])
    got = R.to_np(out).astype(np.float64)
    assert np.all(np.isfinite(got))
    err = np.abs(got - want)
    bound = R.attention_bound(want, mag, low, smag, EPS[b["q"].dtype])
    assert np.all(err <= bound), f"{(err > bound).sum()} out of tolerance, worst {(err / bound).max():.2f} of it"
    return out


@pytest.mark.parametrize("D,bs", [(64, 16), (64, 32), (128, 16), (128, 32), (256, 16), (256, 32)])
@pytest.mark.parametrize("G", [1, 2, 5, 8, 9, 16, 17, 32])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_decode_groups(pkv, D, bs, G, dtype):
    check(pkv, batch([1, 15, 16, 17, 33, 150], 2 * G, 2, D, bs, dtype, seed=G))


@pytest.mark.parametrize("lens", [[1], [0, 5, 0], [31, 32, 33, 63, 64, 65], [127, 128, 129, 2047, 2048, 2049],
                                  [5000, 1, 0, 700], [0, 0]])
@pytest.mark.parametrize("split", [0, 16, 32, 100, 256, 1000])
def test_decode_lengths_and_splits(pkv, lens, split):
    for dtype, bs in ((torch.float16, 16), (torch.bfloat16, 32)):
        check(pkv, batch(lens, 6, 2, 128, bs, dtype, seed=len(lens)), split_tokens=split,
              max_context_len=max(max(lens), 1))


@pytest.mark.parametrize("B,max_len,Hq,D,bs,splits", [(75, 1024, 8, 128, 16, (1024, 1)), (75, 1600, 16, 64, 32, (1024, 2)),
                                                      (40, 2048, 72, 128, 16, (1024, 2))])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_decode_whose_last_sequences_are_cut_finer(pkv, B, max_len, Hq, D, bs, splits, dtype):
    """Both regions of the grid with lengths at their partitions' edges, empty
    sequences, one partition and several; nothing outside the workspace."""
    last = -(-B // 8)
    edge = [0, 1, 511, 512, 513, 1023, 1024, max_len - 1, max_len]
    lens = [edge[i % 9] if i % 5 == 0 else i for i in range(B - last)]
    lens += [edge[(4 * i + 8) % 9] for i in range(last)]
    b = batch(lens, Hq, 8, D, bs, dtype, seed=B)
    d = device(b)
    shape = pkv.kv4_decode_shape(d["q"], d["k_cache"], d["block_tables"], max_len)
    p = pkv.kv4_decode_plan(shape)
    assert (p.split_tokens, p.num_splits) == splits
    assert p.grid_ctas % 8 == 0 and p.grid_ctas > B * 8 * p.num_splits
    n = pkv.kv4_workspace_bytes(shape)
    ws = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    got = check(pkv, b, d, max_context_len=max_len, workspace=ws[4096:4096 + n])
    assert bool((ws[:4096] == 0xA5).all()) and bool((ws[4096 + n:] == 0xA5).all())
    assert torch.equal(got, pkv.kv4_attn_decode(**d, max_context_len=max_len))
    one = check(pkv, b, d, max_context_len=max_len, split_tokens=p.split_tokens)
    assert torch.equal(got[:B - last], one[:B - last])


@pytest.mark.parametrize("k_mul,v_mul,v_add", [(1, 1e-4, 0), (1, 6000, 0), (1, 1, 300), (1, 1e-7, 0), (30, 1, 0),
                                               (1e-3, 1, 0), (1, 3, -2e4)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_decode_magnitudes(pkv, k_mul, v_mul, v_add, dtype):
    check(pkv, batch([70, 1300], 8, 2, 128, 16, dtype, seed=4, k_mul=k_mul, v_mul=v_mul, v_add=v_add))


def test_decode_value_scales_that_grow_along_a_sequence(pkv):
    """Value rows from 1e-3 to 2e4 in order of position, and back."""
    for down in (False, True):
        b = batch([900], 4, 1, 128, 16, torch.bfloat16, seed=6)
        rng = np.random.default_rng(7)
        mul = np.logspace(-3, 4.3, 900)[::-1 if down else 1, None, None]
        slots = b["tables"][0, np.arange(900) // 16] * 16 + np.arange(900) % 16
        R.store(b["vc"], (rng.standard_normal((900, 1, 128)) * mul).astype(np.float32), slots, True)
        check(pkv, b)


@pytest.mark.parametrize("mul", [1e-6, 200.0])
def test_decode_query_magnitudes(pkv, mul):
    b = batch([40, 333], 8, 2, 64, 16, torch.bfloat16, seed=2)
    b["q"] = (b["q"].float() * mul).to(torch.bfloat16)
    b["scale"] /= max(mul, 1.0)
    check(pkv, b)


def test_decode_zero_query_averages_the_values(pkv):
    b = batch([77], 4, 1, 128, 16, torch.float16, seed=3)
    b["q"].zero_()
    check(pkv, b)


@pytest.mark.parametrize("scale", [-0.125, 0.0, 3.0])
@pytest.mark.parametrize("Hq", [2, 6, 14])
def test_decode_any_scale(pkv, scale, Hq):
    b = batch([50, 1, 700], Hq, 2, 128, 16, torch.float16, seed=8)
    b["scale"] = scale
    check(pkv, b)


@pytest.mark.parametrize("Hq,D", [(2, 64), (2, 128), (6, 128), (16, 128), (24, 64), (4, 256)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_decode_queries_that_are_no_numbers(pkv, Hq, D, bad):
    """A NaN or infinity in one head's query makes that head NaN and no other."""
    b = batch([50, 3], Hq, 2, D, 16, torch.float16, seed=8)
    d = device(b)
    good = pkv.kv4_attn_decode(**d)
    d["q"][0, 1, D // 2 + 5] = bad
    out = pkv.kv4_attn_decode(**d)
    assert bool(out[0, 1].isnan().all())
    rest = torch.ones((2, Hq), dtype=torch.bool, device="cuda")
    rest[0, 1] = False
    assert torch.equal(out[rest], good[rest])


def test_decode_nan_rows_stay_in_their_sequence(pkv):
    """A cached NaN reaches its own sequence's heads and no other; a NaN past
    a sequence's end reaches nothing."""
    b = batch([40, 40, 37], 4, 2, 64, 16, torch.float16, seed=5)
    x = np.full((1, 2, 64), 1.0, np.float32)
    x[0, 0, 3] = np.nan
    R.store(b["kc"], x, [int(b["tables"][1, 1]) * 16 + 2], False)
    R.store(b["vc"], x, [int(b["tables"][2, 2]) * 16 + 5], True)      # position 37 of length 37
    d = device(b)
    out = R.to_np(pkv.kv4_attn_decode(**d))
    assert np.isnan(out[1, :2]).all() and np.isfinite(out[1, 2:]).all()
    assert np.isfinite(out[0]).all() and np.isfinite(out[2]).all()


def test_decode_is_deterministic_and_padding_rows_are_zero(pkv):
    b = batch([300, 0, 1200, 0], 16, 2, 128, 16, torch.bfloat16, seed=1)
    d = device(b)
    out = torch.full((4, 16, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    first = pkv.kv4_attn_decode(**d, out=out, max_context_len=1200).clone()
    for _ in range(3):
        assert torch.equal(pkv.kv4_attn_decode(**d, max_context_len=1200), first)
    assert not bool(first[1].any()) and not bool(first[3].any())


def test_decode_device_errors(pkv):
    b = batch([100, 100, 100], 8, 2, 128, 16, torch.float16, seed=1)
    d = device(b)
    good = pkv.kv4_attn_decode(**d, max_context_len=100)
    for i, bad in ((0, -1), (1, 101), (2, 2 ** 31 - 1)):
        lens = d["context_lens"].clone()
        lens[i] = bad
        out = torch.full_like(good, 7.0)
        pkv.kv4_attn_decode(**dict(d, context_lens=lens), out=out, max_context_len=100)
        assert pkv.get_device_error() == 2
        assert bool((out[i] == 7).all())
        rest = [j for j in range(3) if j != i]
        assert torch.equal(out[rest], good[rest])
    for bad in (-1, b["kc"].shape[0], 2 ** 31 - 1):
        tables = d["block_tables"].clone()
        tables[1, 3] = bad
        out = pkv.kv4_attn_decode(**dict(d, block_tables=tables), max_context_len=100)
        assert pkv.get_device_error() == 1
        assert torch.equal(out[[0, 2]], good[[0, 2]])
    assert pkv.kv4_attn_decode(d["q"][:0], d["k_cache"], d["v_cache"], d["block_tables"][:0],
                               d["context_lens"][:0], 1.0).shape == (0, 8, 128)


@pytest.mark.parametrize("split", [0, 64])
def test_writes_stay_inside_their_buffers(pkv, split):
    b = batch([500, 64, 0, 333], 24, 2, 128, 16, torch.bfloat16, seed=2)
    d = device(b)
    buf = torch.full((4 * 24 * 128 + 8192,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[4096:-4096].view(4, 24, 128)
    shape = pkv.kv4_decode_shape(d["q"], d["k_cache"], d["block_tables"], 500, split)
    n = pkv.kv4_workspace_bytes(shape)
    wbuf = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    caches = [d["k_cache"].clone(), d["v_cache"].clone()]
    check(pkv, b, d, out=out, max_context_len=500, split_tokens=split, workspace=wbuf[4096:4096 + n] if n else None)
    assert bool((buf[:4096] == 7).all()) and bool((buf[-4096:] == 7).all())
    assert bool((wbuf[:4096] == 0xA5).all()) and bool((wbuf[4096 + n:] == 0xA5).all())
    assert torch.equal(caches[0], d["k_cache"]) and torch.equal(caches[1], d["v_cache"])


def test_workspace_rules(pkv):
    b = batch([1000], 8, 1, 128, 16, torch.float16, seed=2)
    d = device(b)
    shape = pkv.kv4_decode_shape(d["q"], d["k_cache"], d["block_tables"], 1000, 64)
    n = pkv.kv4_workspace_bytes(shape)
    assert n > 0
    kw = dict(max_context_len=1000, split_tokens=64)
    want = check(pkv, b, d, **kw)
    with pytest.raises(pkv.PkvError) as e:
        pkv.kv4_attn_decode(**d, **kw, workspace=torch.empty(n - 16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == -5
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    pkv.set_workspace(ws)
    try:
        assert torch.equal(pkv.kv4_attn_decode(**d, **kw), want)
        pkv.set_workspace(ws[:n - 16])
        with pytest.raises(pkv.PkvError):
            pkv.kv4_attn_decode(**d, **kw)
    finally:
        pkv.set_workspace(None)


@pytest.mark.parametrize("split", [0, 128])
def test_two_graphs_share_a_workspace_and_another_stream(pkv, split):
    """Replayed one after the other, two captured calls may share a workspace."""
    bs = [batch([900, 30], 8, 2, 128, 16, torch.float16, seed=s) for s in (1, 2)]
    ds = [device(b) for b in bs]
    want = [check(pkv, b, d, split_tokens=split) for b, d in zip(bs, ds)]
    n = max(16, *(pkv.kv4_workspace_bytes(pkv.kv4_decode_shape(d["q"], d["k_cache"], d["block_tables"], None, split)) for d in ds))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    outs, graphs = [torch.zeros_like(w) for w in want], []
    torch.cuda.synchronize()
    for d, o in zip(ds, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv.kv4_attn_decode(**d, out=o, split_tokens=split, workspace=ws)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = [pkv.kv4_attn_decode(**d, split_tokens=split, stream=st) for d in ds]
    st.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(got, want))


def test_graph_replayed_with_other_lengths(pkv):
    """A captured call reads its lengths when it runs: rows that were one
    partition become several and the other way round, in both grid regions."""
    B, max_len = 75, 1600
    rng = np.random.default_rng(5)
    full = rng.integers(1000, max_len + 1, B)
    b = batch(full, 8, 8, 64, 16, torch.float16, seed=9)
    d = device(b)
    p = pkv.kv4_decode_plan(pkv.kv4_decode_shape(d["q"], d["k_cache"], d["block_tables"], max_len))
    assert (p.split_tokens, p.num_splits) == (1024, 2)
    out = torch.zeros_like(d["q"])
    pkv.kv4_attn_decode(**d, out=out, max_context_len=max_len)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.kv4_attn_decode(**d, out=out, max_context_len=max_len)
    for lens in (full, np.minimum(full, rng.integers(0, 700, B)), full // 2, np.where(np.arange(B) % 3, full, 0)):
        d["context_lens"].copy_(torch.from_numpy(lens.astype(np.int32)))
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        want = check(pkv, dict(b, lens=lens.astype(np.int32)), d, max_context_len=max_len)
        assert torch.equal(got, want)


def test_cache_past_32_bit_offsets(pkv):
    """A 4-bit pool of more than 2^32 bytes: append to, gather from and attend
    over its last blocks."""
    NB, Hkv, bs, D, L = 60000, 32, 32, 128, 70              # 4.9 GB a cache
    kc, vc = pkv.kv4_cache(NB, Hkv, bs, D), pkv.kv4_cache(NB, Hkv, bs, D)
    a, _ = make(L, 32, Hkv, D, bs, torch.bfloat16, 128, seed=2)
    blocks = np.array([NB - 1, NB - 3, NB - 2], np.int32)
    slots = blocks[np.arange(L) // bs].astype(np.int64) * bs + np.arange(L) % bs
    a["slot_mapping"] = torch.from_numpy(slots.astype(np.int32)).cuda()
    q = pkv.kv4_append(**a, k_cache=kc, v_cache=vc)
    ek, ev = (np.zeros((3, Hkv, bs, 80), np.uint8) for _ in range(2))
    b = dict(a, slot_mapping=torch.from_numpy((slots - (NB - 3) * bs).astype(np.int32)))
    reference_append(b, ek, ev, False)
    assert np.array_equal(kc[-3:].cpu().numpy(), ek) and np.array_equal(vc[-3:].cpu().numpy(), ev)
    assert not bool(kc[:60].any())
    k, _ = pkv.kv4_gather(kc, vc, a["slot_mapping"], torch.bfloat16)
    k2, _ = pkv.kv4_gather(kc[-3:].contiguous(), vc[-3:].contiguous(), b["slot_mapping"].cuda(), torch.bfloat16)
    assert torch.equal(k, k2)
    batch_ = dict(q=q[-1:].cpu(), kc=ek, vc=ev, tables=blocks[None] - (NB - 3), lens=np.array([L], np.int32),
                  scale=float(np.float32(D ** -0.5)))
    d = dict(q=q[-1:].contiguous(), k_cache=kc, v_cache=vc, block_tables=torch.from_numpy(blocks[None]).cuda(),
             context_lens=torch.tensor([L], dtype=torch.int32, device="cuda"), scale=batch_["scale"])
    check(pkv, batch_, d)


# ---------------------------------------------------------------- together
def test_serving_session(pkv):
    """Prompts appended in chunks, their prefix read back, decode steps by the
    block manager's slots, a fork with copy-on-write, a swap out and in: the
    caches stay the reference's byte for byte, attention within its bound."""
    Hq, Hkv, D, bs, dtype = 8, 2, 128, 16, torch.bfloat16
    NB, rng = 40, np.random.default_rng(0)
    bm = pkv.BlockManager(NB, 24, bs)
    kc, vc = pkv.kv4_cache(NB, Hkv, bs, D), pkv.kv4_cache(NB, Hkv, bs, D)
    kh, vh = (torch.zeros((24, Hkv, bs, D * 5 // 8), dtype=torch.uint8).pin_memory() for _ in range(2))
    ek, ev = kc.cpu().numpy(), vc.cpu().numpy()
    table = pkv.rope_table(256, D)
    scale = float(np.float32(D ** -0.5))

    def rows(T):
        x = torch.from_numpy(rng.standard_normal((T, Hq + 2 * Hkv, D)).astype(np.float32)).to(dtype).cuda()
        return x.split([Hq, Hkv, Hkv], 1)

    def append(slots, positions):
        q, k, v = rows(len(slots))
        a = dict(q=q, k=k, v=v, positions=torch.tensor(positions, dtype=torch.int32, device="cuda"), cos_sin=table,
                 slot_mapping=torch.tensor(slots, dtype=torch.int32, device="cuda"))
        reference_append(a, ek, ev, False)
        return pkv.kv4_append(**a, k_cache=kc, v_cache=vc)

    prompt = {0: 37, 1: 64, 2: 5}
    for i, n in prompt.items():
        bm.add_sequence(i, n)
        tables, _ = bm.block_tables([i], 8)
        slots = [int(tables[0, t // bs]) * bs + t % bs for t in range(n)]
        for lo in range(0, n, 20):
            append(slots[lo:lo + 20], list(range(lo, min(n, lo + 20))))
        k, v = pkv.kv4_gather(kc, vc, torch.tensor(slots, dtype=torch.int32, device="cuda"), dtype)
        assert np.abs(R.to_np(k) - R.load(ek, slots, False)).max() <= 2.0 ** -8 * np.abs(R.to_np(k)).max()
    bm.fork(0, 3)
    ids = [0, 1, 2, 3]
    for step in range(20):
        if step == 8:                               # sequence 1 leaves the GPU and comes back
            pairs = bm.swap_out(1, 0)
            pkv.copy_blocks(kc, vc, kh, vh, torch.from_numpy(pairs).cuda())
            torch.cuda.synchronize()
            back = bm.swap_in(1)
            pkv.copy_blocks(kh, vh, kc, vc, torch.from_numpy(back).cuda())
            keep = ek.copy(), ev.copy()
            to = dict(pairs.tolist())
            for c, g in back.tolist():
                src = next(s for s, d in to.items() if d == c)
                ek[g], ev[g] = keep[0][src], keep[1][src]
        slots, positions = [], []
        for i in ids:
            slot, src, dst = bm.append_token(i)
            if src >= 0:
                pkv.copy_blocks(kc, vc, kc, vc, torch.tensor([[src, dst]], dtype=torch.int32, device="cuda"))
                ek[dst], ev[dst] = ek[src], ev[src]
            slots.append(slot)
            positions.append(bm.seq_info(i)[0] - 1)
        q = append(slots + [-1], positions + [0])   # one padding row behind the batch
        tables, lens = bm.block_tables(ids, 8)
        tables, lens = np.vstack([tables, np.full((1, 8), -1, np.int32)]), np.append(lens, 0).astype(np.int32)
        b = dict(q=q.cpu(), kc=ek, vc=ev, tables=tables, lens=lens, scale=scale)
        check(pkv, b, dict(q=q, k_cache=kc, v_cache=vc, block_tables=torch.from_numpy(tables).cuda(),
                           context_lens=torch.from_numpy(lens).cuda(), scale=scale))
    assert np.array_equal(kc.cpu().numpy(), ek) and np.array_equal(vc.cpu().numpy(), ev)
    bm.close()
