"""The rotation appends with positions of several axes.  A token's angles are
those of a table row made up of its axes' rows, so the call has to equal, bit
for bit, the one-axis call on such a table (which has its own tests), and the
rotated rows have to be the formula's in 64 bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _case(T, hq, hkv, D, bs, dt, sections, seed=0, fused=False, far=4096):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, hq + 2 * hkv, D), generator=g).to(dt).cuda()
    q, k, v = x.split([hq, hkv, hkv], 1)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pos = torch.randint(0, far, (len(sections), T), generator=g, dtype=torch.int32).cuda()
    NB = T // bs + 3
    slots = torch.randperm(NB * bs, generator=g)[:T].int().cuda()
    if T > 3:
        slots[T // 2] = -1
    return q, k, v, pos, slots, NB


def _merged(table, pos, sections):
    """[T, R]: each token's own table row."""
    half = sum(sections)
    axis = torch.arange(len(sections)).repeat_interleave(torch.tensor(sections)).cuda()
    p, i = pos.long()[axis].T, torch.arange(half, device="cuda")
    return torch.cat([table[p, i], table[p, half + i]], 1).contiguous()


SECTIONS = [(64, (16, 8, 8)), (64, (11, 13, 8)), (128, (16, 24, 24)), (128, (1, 62, 1)), (128, (0, 40, 24)),
            (128, (10, 20, 30, 4)), (128, (64,)), (128, (63, 1)), (256, (32, 48, 48)), (256, (5, 100, 23)),
            (256, (24, 24, 24, 56)), (128, (8, 4, 4)), (256, (0, 0, 0, 8))]


@pytest.mark.parametrize("D,sections", SECTIONS)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
def test_equals_the_merged_table(pkv, D, sections, inter, dt):
    rot = 2 * sum(sections)
    table = pkv.rope_table(4096, rot)
    for T, hq, hkv, bs, fused in ((1, 4, 1, 16, False), (37, 8, 2, 16, True), (700, 5, 5, 32, False)):
        q, k, v, pos, slots, NB = _case(T, hq, hkv, D, bs, dt, sections, seed=T, fused=fused)
        own, arange = _merged(table, pos, sections), torch.arange(T, dtype=torch.int32, device="cuda")
        a, b = ([torch.full((NB, hkv, bs, D), 3.0, dtype=dt, device="cuda") for _ in range(2)] for _ in range(2))
        got = pkv.rope_append(q, k, v, pos, table, slots, *a, interleaved=inter, sections=sections)
        want = pkv.rope_append(q, k, v, arange, own, slots, *b, interleaved=inter)
        assert torch.equal(got, want) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        a, b = ([pkv.kv4_cache(NB, hkv, bs, D) for _ in range(2)] for _ in range(2))
        got = pkv.kv4_append(q, k, v, pos, table, slots, *a, interleaved=inter, sections=list(sections))
        want = pkv.kv4_append(q, k, v, arange, own, slots, *b, interleaved=inter)
        assert torch.equal(got, want) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        # the formula in 64 bits: two products and a sum in FP32 (each off by half a step of a
        # number of at most |a| + |b|), one rounding to 16 bits
        c, s = own.double()[:, None].chunk(2, -1)
        x = q.double()
        x, y = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
        half = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[dt]
        ref = torch.stack([x * c - y * s, y * c + x * s], -1)
        z = got.double()
        z = torch.stack([z[..., 0:rot:2], z[..., 1:rot:2]] if inter else [z[..., :rot // 2], z[..., rot // 2:rot]], -1)
        bound = half * ref.abs() + (x.abs() + y.abs())[..., None] * 2.0 ** -22 + 2.0 ** -25
        assert bool(((z - ref).abs() <= bound).all()) and torch.equal(got[..., rot:], q[..., rot:])
    assert pkv.get_device_error() == 0


def test_equal_axes_are_one(pkv):
    """Text counts on in every axis: the same as a single position."""
    T, D = 50, 128
    q, k, v, pos, slots, NB = _case(T, 8, 2, D, 16, torch.bfloat16, (16, 24, 24))
    pos = pos[:1].expand(3, T).contiguous()
    table = pkv.rope_table(4096, D)
    a, b = ([torch.zeros((NB, 2, 16, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(2))
    got = pkv.rope_append(q, k, v, pos, table, slots, *a, sections=(16, 24, 24))
    want = pkv.rope_append(q, k, v, pos[0].contiguous(), table, slots, *b)
    assert torch.equal(got, want) and torch.equal(a[0], b[0])


def test_keys_only_and_in_place(pkv):
    T, D = 33, 64
    q, k, v, pos, slots, NB = _case(T, 8, 2, D, 16, torch.float16, (8, 12, 12))
    table = pkv.rope_table(4096, D)
    a, b = ([torch.zeros((NB, 2, 16, D), dtype=torch.float16, device="cuda") for _ in range(2)] for _ in range(2))
    want = pkv.rope_append(q, k, v, pos, table, slots, *a, sections=(8, 12, 12))
    assert pkv.rope_append(None, k, v, pos, table, slots, *b, sections=(8, 12, 12)) is None
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    pkv.rope_append(q, k, v, pos, table, slots, *b, q_out=q, sections=(8, 12, 12))
    assert torch.equal(q, want)


@pytest.mark.parametrize("axis", [0, 1, 2])
@pytest.mark.parametrize("bad", [-1, 4096])
def test_a_bad_position_of_any_axis_skips_the_token(pkv, axis, bad):
    T, D = 20, 128
    q, k, v, pos, slots, NB = _case(T, 8, 2, D, 16, torch.float16, (16, 24, 24))
    table = pkv.rope_table(4096, D)
    a, b = ([torch.zeros((NB, 2, 16, D), dtype=torch.float16, device="cuda") for _ in range(2)] for _ in range(2))
    want = pkv.rope_append(q, k, v, pos, table, slots, *a, sections=(16, 24, 24))
    pos[axis, 7] = bad
    out = torch.full_like(q, 9.0)
    pkv.rope_append(q, k, v, pos, table, slots, *b, q_out=out, sections=(16, 24, 24))
    assert pkv.get_device_error() == 5
    s = int(slots[7])
    assert bool((out[7] == 9).all()) and not bool(b[0][s // 16, :, s % 16].any())
    keep = torch.arange(T) != 7
    assert torch.equal(out[keep], want[keep])
    a[0][s // 16, :, s % 16] = 0
    assert torch.equal(a[0], b[0])


def test_positions_of_an_axis_without_pairs_do_not_matter(pkv):
    T, D = 20, 128
    q, k, v, pos, slots, NB = _case(T, 8, 2, D, 16, torch.float16, (0, 40, 24))
    table = pkv.rope_table(4096, D)
    a, b = ([torch.zeros((NB, 2, 16, D), dtype=torch.float16, device="cuda") for _ in range(2)] for _ in range(2))
    want = pkv.rope_append(q, k, v, pos, table, slots, *a, sections=(0, 40, 24))
    pos[0] = -1
    got = pkv.rope_append(q, k, v, pos, table, slots, *b, sections=(0, 40, 24))
    assert torch.equal(got, want) and torch.equal(a[0], b[0]) and pkv.get_device_error() == 0


def test_refusals(pkv):
    T, D = 4, 64
    q, k, v, pos, slots, NB = _case(T, 8, 2, D, 16, torch.float16, (8, 12, 12))
    table = pkv.rope_table(64, D)
    kc, vc = (torch.zeros((NB, 2, 16, D), dtype=torch.float16, device="cuda") for _ in range(2))
    for sections, p in (((8, 12), pos), ((8, 12, 11), pos), ((8, -4, 28), pos), ((4, 4, 8, 8, 8), pos),
                        ((8, 12, 12), pos[0]), ((8, 12, 12), pos.T.contiguous()), ((), pos), ((8.0, 12, 12), pos),
                        (None, pos)):
        with pytest.raises(ValueError):
            pkv.rope_append(q, k, v, p, table, slots, kc, vc, sections=sections)
    with pytest.raises(ValueError):
        pkv.rope_append(q, k, v, None, None, slots, kc, vc, sections=(8, 12, 12))
