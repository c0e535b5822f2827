"""The rotation append and the 4-bit cache on the CPU: the format's reference
against its own error bound, and every refusal of the C ABI and the binding
(no call here reaches a GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import kv4_ref as R
from paged_kv_cache_268_gb300 import _binding as B
from paged_kv_cache_268_gb300 import build

FAKE = 0x10000  # 16-byte aligned non-null address; never dereferenced on the host


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.load_library()


# ---------------------------------------------------------------- the format
@pytest.mark.parametrize("make", [
    lambda r: r.standard_normal((64, 2, 128)),
    lambda r: r.standard_normal((64, 2, 64)) * 1e-3,
    lambda r: r.standard_normal((64, 1, 256)) * 3e4,
    lambda r: r.standard_normal((64, 1, 128)) + 40,          # an offset far from zero
    lambda r: np.full((4, 1, 64), -7.25),                     # no spread at all
    lambda r: np.zeros((4, 1, 64)),
    lambda r: r.standard_normal((8, 1, 64)) * 1e-8,           # below binary16's smallest step
], ids=["normal", "small", "large", "offset", "constant", "zero", "tiny"])
def test_values_are_within_half_a_step(make):
    x = make(np.random.default_rng(0)).astype(np.float32)
    n, s, z = R.quantise(x)
    s, z = s.astype(np.float64)[..., None], z.astype(np.float64)[..., None]
    got = (s * (n + z)).reshape(x.shape)
    # half a step, plus what rounding z (2^-11 of it, or half of binary16's
    # smallest subnormal step) moves the span's ends by, plus FP32's rounding
    # of the quotient x / s (2^-23 of it)
    bound = s * (0.5 + np.abs(z) * 2.0 ** -11 + 2.0 ** -25) + np.abs(x.reshape(n.shape)) * 2.0 ** -22
    assert np.all(np.abs(got - x).reshape(n.shape) <= bound)
    assert np.all(np.abs(z) <= 1025) and n.max() <= 15


def test_a_group_with_a_nan_or_infinity_reads_as_nan():
    x = np.ones((3, 1, 64), np.float32)
    x[0, 0, 5], x[1, 0, 40], x[2, 0, 40] = np.nan, np.inf, -np.inf
    n, s, z = R.quantise(x)
    assert np.isnan(s[0, 0, 0]) and not np.isnan(s[0, 0, 1])
    assert np.isnan(s[1, 0, 1]) and np.isnan(s[2, 0, 1]) and not np.isnan(s[1, 0, 0])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("values", [False, True])
def test_every_byte_of_a_tile_belongs_to_one_row(D, bs, values):
    off = R.row_offsets(bs, D, values)
    assert sorted(off.ravel()) == list(range(bs * D * 5 // 8))
    # eight rows' 16-byte pieces of one group lie in eight different 16-byte
    # columns of 128 bytes (what reads without bank conflicts want)
    for g in range(D // 32):
        for r0 in range(0, bs, 8):
            assert len({off[r, 16 * g] % 128 // 16 for r in range(r0, r0 + 8)}) == 8


def test_store_then_load():
    rng = np.random.default_rng(1)
    cache = rng.integers(0, 256, (5, 3, 16, 80), dtype=np.uint8)
    x = rng.standard_normal((7, 3, 128)).astype(np.float32)
    slots = np.array([3, 79, -1, 16, 33, 40, 0])
    before = cache.copy()
    R.store(cache, x, slots, True)
    n, s, z = R.quantise(x)
    want = (s.astype(np.float64)[..., None] * (n + z.astype(np.float64)[..., None])).reshape(x.shape)
    keep = slots >= 0
    assert np.array_equal(R.load(cache, slots[keep], True), want[keep])
    assert (cache != before).any(-1).any(-1).sum() <= 5 * 3


# ---------------------------------------------------------------- C ABI refusals
def _shape(**kw):
    base = dict(num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16,
                num_blocks=64, max_blocks_per_seq=8, max_context_len=100, dtype=0)
    base.update(kw)
    return B.make_shape(**base)


def _append(lib, fn, shape=None, rope=(128, 0, 100, 0, 0, 0), T=2, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, pos=FAKE, cs=FAKE, slots=FAKE, q_out=FAKE, kc=FAKE, vc=FAKE)
    a.update(kw)
    shape, rope = shape or _shape(), B.Rope(*rope)
    return getattr(lib, fn)(ctypes.byref(shape), ctypes.byref(rope), a["q"], a["k"], a["v"],
                            a["pos"], a["cs"], a["slots"], T, a["q_out"], a["kc"], a["vc"], None)


@pytest.mark.parametrize("fn", ["pkv_rope_append", "pkv_kv4_append"])
@pytest.mark.parametrize("kw,code", [
    (dict(shape=dict(head_dim=96)), -3),
    (dict(shape=dict(block_size=8)), -3),
    (dict(shape=dict(dtype=2)), -3),
    (dict(shape=dict(num_kv_heads=0)), -2),
    (dict(shape=dict(num_q_heads=0)), -2),
    (dict(shape=dict(num_blocks=1 << 24, num_kv_heads=8)), -3),
    (dict(rope=(136, 0, 100, 0, 0, 0)), -2),              # more channels than a head has
    (dict(rope=(-16, 0, 100, 0, 0, 0)), -2),
    (dict(rope=(24, 0, 100, 0, 0, 0)), -3),               # not a multiple of 16
    (dict(rope=(64, 0, 0, 0, 0, 0)), -2),                 # an empty table
    (dict(rope=(64, 0, 9, 1016, 0, 0)), -2),              # q rows overlap
    (dict(rope=(64, 0, 9, 0, 248, 0)), -2),
    (dict(rope=(64, 0, 9, 0, 0, -256)), -2),
    (dict(rope=(64, 0, 9, 1028, 0, 0)), -4),              # q rows not 16-byte aligned
    (dict(rope=(64, 0, 9, 2048, 0, 0)), -2),              # strided q, rotated "in place"
    (dict(T=-1), -2),
    (dict(k=None), -1), (dict(v=None), -1), (dict(slots=None), -1), (dict(kc=None), -1),
    (dict(vc=None), -1), (dict(q_out=None), -1), (dict(pos=None), -1), (dict(cs=None), -1),
    (dict(q=FAKE + 8), -4), (dict(k=FAKE + 2), -4), (dict(cs=FAKE + 4), -4),
    (dict(pos=FAKE + 2), -4), (dict(vc=FAKE + 8), -4),
    (dict(T=0, k=None, v=None), 0),                       # no tokens: no-op
    (dict(), -6),                                         # all good: no device here
    (dict(q=None, q_out=None, shape=dict(num_q_heads=0)), -6),
    (dict(rope=(0, 0, 0, 0, 0, 0), pos=None, cs=None), -6),
])
def test_append_refusals(lib, fn, kw, code):
    kw = dict(kw)
    if "shape" in kw:
        kw["shape"] = _shape(**kw["shape"])
    assert _append(lib, fn, **kw) == code
    assert lib.pkv_launch_count() == 0


def test_append_refuses_null_structs(lib):
    s, r = _shape(), B.Rope()
    for fn in ("pkv_rope_append", "pkv_kv4_append"):
        f = getattr(lib, fn)
        assert f(None, ctypes.byref(r), *[FAKE] * 6, 1, FAKE, FAKE, FAKE, None) == -1
        assert f(ctypes.byref(s), None, *[FAKE] * 6, 1, FAKE, FAKE, FAKE, None) == -1


@pytest.mark.parametrize("kw,args,code", [
    (dict(head_dim=32), {}, -3), (dict(), dict(T=-1), -2), (dict(), dict(T=0, k=None), 0),
    (dict(), dict(k=None), -1), (dict(), dict(slots=None), -1), (dict(), dict(kc=FAKE + 4), -4),
    (dict(), dict(slots=FAKE + 1), -4), (dict(), {}, -6),
])
def test_gather_refusals(lib, kw, args, code):
    a = dict(kc=FAKE, vc=FAKE, slots=FAKE, T=3, k=FAKE, v=FAKE)
    a.update(args)
    s = _shape(**kw)
    assert lib.pkv_kv4_gather(ctypes.byref(s), a["kc"], a["vc"], a["slots"], a["T"], a["k"],
                              a["v"], None) == code


@pytest.mark.parametrize("kw,args,code", [
    (dict(num_q_heads=6, num_kv_heads=4), {}, -2), (dict(num_q_heads=66), {}, -3),
    (dict(max_context_len=129), {}, -2), (dict(max_context_len=0), {}, -2),
    (dict(split_tokens=-1), {}, -2), (dict(kernel=1), {}, -3), (dict(kernel=3), {}, -3),
    (dict(head_dim=80), {}, -3), (dict(num_seqs=0), dict(q=None), 0),
    (dict(), dict(q=None), -1), (dict(), dict(cl=None), -1), (dict(), dict(out=FAKE + 8), -4),
    (dict(), dict(bt=FAKE + 2), -4), (dict(), {}, -6),
])
def test_decode_refusals(lib, kw, args, code):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, cl=FAKE, out=FAKE)
    a.update(args)
    s = _shape(**kw)
    assert lib.pkv_kv4_attn_decode(ctypes.byref(s), a["q"], a["kc"], a["vc"], a["bt"], a["cl"],
                                   0.1, a["out"], None, 0, None) == code


def test_plan_refusals(lib):
    p, n = B.Plan(), ctypes.c_size_t()
    s = _shape()
    assert lib.pkv_kv4_decode_plan(None, 152, ctypes.byref(p)) == -1
    assert lib.pkv_kv4_decode_plan(ctypes.byref(s), -1, ctypes.byref(p)) == -2
    assert lib.pkv_kv4_decode_plan(ctypes.byref(_shape(kernel=2)), 152, ctypes.byref(p)) == -3
    assert lib.pkv_kv4_decode_plan(ctypes.byref(s), 152, ctypes.byref(p)) == 0 and p.variant == 3
    assert lib.pkv_kv4_workspace_bytes(ctypes.byref(s), None) == -1
    with pytest.raises(ValueError):
        B.kv4_decode_plan(s, num_sms=0)


def test_sizes_past_the_counters_are_refused(lib):
    big = (1 << 30) + 1
    assert _append(lib, "pkv_rope_append", T=big) == -3
    assert _append(lib, "pkv_kv4_append", T=big) == -3
    s = _shape()
    assert lib.pkv_kv4_gather(ctypes.byref(s), FAKE, FAKE, FAKE, big, FAKE, FAKE, None) == -3
    heads = _shape(num_kv_heads=1 << 26, num_blocks=1)
    assert lib.pkv_kv4_gather(ctypes.byref(heads), FAKE, FAKE, FAKE, 1, FAKE, FAKE, None) == -3
    many = _shape(num_seqs=1 << 30, num_q_heads=8, num_kv_heads=8)
    p = B.Plan()
    assert lib.pkv_kv4_decode_plan(ctypes.byref(many), 152, ctypes.byref(p)) == -3


# ---------------------------------------------------------------- the planner
def columns(D, G):
    return 2 if G <= 2 and D > 64 else (4 if G <= 4 else 8)


def tiles(D, G):
    return 2 if D <= 128 and G > 8 else 1


def resident(D, G):
    nt = tiles(D, G)
    if D * nt == 64 or (D * nt == 128 and columns(D, G) < 8):
        return 4
    return 3 if D * nt == 128 else 2


def restated_plan(B_, Hq, Hkv, D, bs, maxL, split, sms):
    G = Hq // Hkv
    heads = columns(D, G) * tiles(D, G)
    units = B_ * Hkv * -(-G // heads)
    if split > 0:
        P = -(-split // bs) * bs
    else:
        slots = sms * resident(D, G)
        per_slot = units * maxL // slots
        P = 2048 if per_slot >= 6000 else (1024 if per_slot >= 1000 else per_slot // 2)
        if B_ <= 4 and 0 < units < slots:
            S = slots // units
            P = -(-maxL // S)
        P = max(P, 128 if 256 < maxL <= 2048 else 256)
        P = -(-P // 128) * 128
        least = -(-maxL // 1024)
        if P < least:
            P = -(-least // 128) * 128
    P = min(P, 256 * bs)
    if P > maxL:
        P = -(-maxL // bs) * bs
    P = max(P, bs)
    S = -(-maxL // P)
    last, S2 = 0, S                      # the sequences dispatched last, finer
    if split == 0 and P >= 1024 and B_ > 4:
        last = -(-B_ // 8)
        S2 = -(-maxL // min(P, max(512, -(-least // 128) * 128)))
    grid = units // B_ * ((B_ - last) * S + last * S2) if B_ else 0
    rows = (B_ - last) * S * (S > 1) + last * S2 * (S2 > 1)
    return P, S, grid, rows * Hq * (4 * D + 8)


@pytest.mark.parametrize("sms", [1, 16, 152])
@pytest.mark.parametrize("D,bs", [(64, 16), (128, 32), (128, 16), (256, 16)])
def test_plan_follows_its_rule(lib, sms, D, bs):
    for B_ in (0, 1, 3, 4, 5, 64, 300):
        for Hkv, G in ((1, 1), (8, 4), (32, 1), (2, 8), (8, 16), (3, 5), (1, 32)):
            for maxL in (1, 16, 200, 256, 257, 1100, 2048, 5000, 40000, 700001):
                for split in (0, 1, 100, 4096, 100000):
                    s = B.make_shape(num_seqs=B_, num_q_heads=Hkv * G, num_kv_heads=Hkv, head_dim=D, block_size=bs,
                                     num_blocks=4096, max_blocks_per_seq=-(-maxL // bs), max_context_len=maxL,
                                     dtype=1, split_tokens=split)
                    p = B.kv4_decode_plan(s, num_sms=sms)
                    P, S, grid, ws = restated_plan(B_, Hkv * G, Hkv, D, bs, maxL, split, sms)
                    assert (p.split_tokens, p.num_splits, p.grid_ctas, p.workspace_bytes) == (P, S, grid, ws)
                    assert p.split_tokens % bs == 0 and (p.num_splits - 1) * p.split_tokens < maxL
                    assert p.variant == 3 and p.schedule == 0 and p.warps_per_cta == 4


@pytest.mark.parametrize("maxL", [600_000, 4_194_304, 5_000_000, 100_000_000, 2 ** 31 - 16])
@pytest.mark.parametrize("bs", [16, 32])
def test_plan_of_very_long_contexts(lib, maxL, bs):
    """A partition's block ids always fit its CTA (256), whatever the length."""
    for B_ in (1, 5, 8):
        s = B.make_shape(num_seqs=B_, num_q_heads=4, num_kv_heads=1, head_dim=128, block_size=bs, num_blocks=4096,
                         max_blocks_per_seq=-(-maxL // bs), max_context_len=maxL, dtype=1)
        p = B.kv4_decode_plan(s, num_sms=152)
        P, S, grid, ws = restated_plan(B_, 4, 1, 128, bs, maxL, 0, 152)
        assert (p.split_tokens, p.num_splits, p.grid_ctas, p.workspace_bytes) == (P, S, grid, ws)
        last = -(-B_ // 8) if B_ > 4 else 0
        assert p.split_tokens <= 256 * bs
        if last:
            late = (p.grid_ctas - (B_ - last) * S) // last
            assert late * 256 * bs >= maxL and late >= S


def test_plan_worked_examples(lib):
    def plan(B_, Hq, Hkv, D, bs, maxL):
        s = B.make_shape(num_seqs=B_, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, block_size=bs, num_blocks=65536,
                         max_blocks_per_seq=-(-maxL // bs), max_context_len=maxL, dtype=1)
        p = B.kv4_decode_plan(s, num_sms=152)
        return p.split_tokens, p.num_splits, p.grid_ctas

    assert plan(64, 32, 32, 128, 16, 4096) == (2048, 2, 56 * 64 + 8 * 256)
    assert plan(4, 64, 8, 128, 32, 32768) == (2432, 14, 448)        # one wave of three CTAs per SM
    assert plan(256, 32, 8, 128, 16, 2048) == (2048, 1, 224 * 8 + 32 * 32)
    assert plan(4, 8, 8, 64, 16, 200) == (208, 1, 32)                # no split of up to 256 tokens


# ---------------------------------------------------------------- binding refusals
class _Cuda(torch.Tensor):
    """A host tensor that says it is on a GPU: reaches the binding's checks."""
    is_cuda = True
    device = torch.device("cuda", 0)


def _c(*shape, dtype=torch.float16):
    return torch.zeros(shape, dtype=dtype).as_subclass(_Cuda)


def _args(kv4, T=3, Hq=4, Hkv=2, D=64, bs=16, NB=4):
    cache = (lambda: _c(NB, Hkv, bs, D * 5 // 8, dtype=torch.uint8)) if kv4 else (lambda: _c(NB, Hkv, bs, D))
    return dict(q=_c(T, Hq, D), k=_c(T, Hkv, D), v=_c(T, Hkv, D), positions=_c(T, dtype=torch.int32),
                cos_sin=_c(9, D, dtype=torch.float32), slot_mapping=_c(T, dtype=torch.int32),
                k_cache=cache(), v_cache=cache())


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("bad", [
    dict(q=_c(3, 4, 128)), dict(q=_c(2, 4, 64)), dict(q=_c(3, 256)), dict(k=_c(3, 3, 64)), dict(k=_c(3, 128)),
    dict(v=_c(3, 2, 64, dtype=torch.bfloat16)), dict(q=_c(3, 4, 64, dtype=torch.float32)),
    dict(k=_c(3, 2, 128)[..., ::2]), dict(k=_c(3, 4, 64)[:, ::2]),
    dict(k=_c(1, 2, 64).expand(3, 2, 64)),
    dict(slot_mapping=_c(4, dtype=torch.int32)), dict(slot_mapping=_c(3, dtype=torch.int64)),
    dict(positions=_c(2, dtype=torch.int32)), dict(positions=_c(3, dtype=torch.int64)), dict(positions=None),
    dict(cos_sin=None), dict(cos_sin=_c(9, 64)), dict(cos_sin=_c(64, dtype=torch.float32)),
    dict(q_out=_c(3, 4, 128)), dict(q_out=_c(3, 4, 64, dtype=torch.bfloat16)), dict(q=None, q_out=_c(3, 4, 64)),
    dict(v_cache=_c(4, 2, 32, 64)), dict(k_cache=_c(4, 2, 1024)), dict(slot_mapping=torch.zeros(3, dtype=torch.int32)),
])
def test_binding_refuses(kv4, bad):
    a = _args(kv4)
    a.update(bad)
    with pytest.raises(ValueError):
        (B.kv4_append if kv4 else B.rope_append)(**a)


def test_binding_refuses_other_caches():
    a = _args(True)
    for bad in (_c(4, 2, 16, 64), _c(4, 2, 16, 42, dtype=torch.uint8), _c(4, 2, 640, dtype=torch.uint8)):
        with pytest.raises(ValueError):
            B.kv4_append(**dict(a, k_cache=bad, v_cache=bad))
        with pytest.raises(ValueError):
            B.kv4_gather(bad, bad, a["slot_mapping"], torch.float16)
    with pytest.raises(ValueError):
        B.kv4_gather(a["k_cache"], a["v_cache"], a["slot_mapping"], torch.float32)
    with pytest.raises(ValueError):
        B.kv4_gather(a["k_cache"], a["v_cache"], a["slot_mapping"], torch.float16, k=_c(3, 2, 128))
    q, bt, cl = _c(3, 4, 64), _c(3, 2, dtype=torch.int32), _c(3, dtype=torch.int32)
    for kw in (dict(q=_c(3, 4, 128)), dict(block_tables=_c(2, 2, dtype=torch.int32)),
               dict(context_lens=_c(3, dtype=torch.int64)), dict(out=_c(3, 4, 32)),
               dict(q=_c(3, 4, 64, dtype=torch.float32)), dict(context_lens=_c(2, dtype=torch.int32))):
        d = dict(q=q, k_cache=a["k_cache"], v_cache=a["v_cache"], block_tables=bt, context_lens=cl)
        d.update(kw)
        with pytest.raises(ValueError):
            B.kv4_attn_decode(d.pop("q"), scale=1.0, **d)


def test_rope_table_is_worked_out_in_64_bits():
    t = B.rope_table(131072, 32, device="cpu")
    assert t.shape == (131072, 32) and t.dtype == torch.float32
    p = np.array([0, 1, 77, 131071])
    ang = p[:, None] * 10000.0 ** (-np.arange(0, 32, 2) / 32)
    want = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    # one rounding of a number of at most 1, plus a 64-bit angle's own error
    assert np.abs(t.numpy()[p] - want).max() <= 2.0 ** -24
    assert B.kv4_cache(3, 2, 16, 128, device="cpu").shape == (3, 2, 16, 80)
