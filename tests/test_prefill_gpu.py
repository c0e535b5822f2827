"""Chunk and prompt attention against the plain 64-bit forms."""
import pytest
import torch

import prefill_ref as R

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def _rows(T, hq, hkv, D, dt, g, fused=False):
    x = torch.randn((T, hq + 2 * hkv, D), generator=g).to(dt).cuda()
    q, k, v = x.split([hq, hkv, hkv], 1)
    return (q, k, v) if fused else (q.contiguous(), k.contiguous(), v.contiguous())


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _chunk(pkv, new, ctx, hq, hkv, D, bs, dt, seed=0, scale=None, fused=False, spare=2, **kw):
    g = torch.Generator().manual_seed(seed)
    scale = D ** -0.5 if scale is None else scale
    lens = [n + c for n, c in zip(new, ctx)]
    q = _rows(sum(new), hq, hkv, D, dt, g, fused)[0]
    _, k, v = _rows(sum(lens), hq, hkv, D, dt, g)
    kc, vc, tables = R.paged(k, v, lens, bs, g, spare=spare)
    out = pkv.paged_attn_chunk(q, kc.cuda(), vc.cuda(), tables.cuda(), _i32(lens), _i32(R.starts(new)), scale,
                               max_context_len=max(max(lens), 1), **kw)
    ref, bound = R.packed(q, k, v, R.starts(new), R.starts(lens), scale)
    assert pkv.get_device_error() == 0
    R.check(out, ref, bound)


# around the ends of row tiles and key tiles, sequences without new tokens or without any
LENS = {
    "single": ([1], [0]),
    "one-after": ([1, 1, 1], [0, 127, 128]),
    "mixed": ([3, 1, 0, 40, 1, 2], [0, 300, 77, 5, 0, 1022]),
    "edges": ([127, 128, 129], [1, 0, 128]),
    "long": ([300, 1], [700, 1500]),
    "none": ([2, 0, 5], [0, 0, 0]),
}


@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("D,bs", [(64, 16), (64, 32), (128, 16), (128, 32), (256, 16), (256, 32)])
@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
def test_chunk_lengths(pkv, lens, D, bs, dt):
    new, ctx = LENS[lens]
    _chunk(pkv, new, ctx, 8, 2, D, bs, dt, seed=D + bs)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 6, 7, 8, 9, 12, 16, 17, 24, 31, 32])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunk_groups(pkv, G, D):
    _chunk(pkv, [1, 45, 130], [200, 17, 0], 2 * G, 2, D, 16, BF16 if G % 2 else F16, seed=G)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("split", [1, 128, 300])
def test_chunk_partitions(pkv, D, split):
    _chunk(pkv, [1, 8, 300, 0, 2], [1200, 900, 500, 40, 0], 12, 3, D, 32, F16, seed=split, split_tokens=split)


def test_chunk_strided_queries_and_many_sequences(pkv):
    g = torch.Generator().manual_seed(5)
    new = torch.randint(0, 4, (150,), generator=g).tolist()
    ctx = torch.randint(0, 200, (150,), generator=g).tolist()
    _chunk(pkv, new, ctx, 8, 2, 128, 16, BF16, fused=True)


def test_chunk_long_contexts(pkv):
    for D, bs in ((128, 16), (64, 32), (256, 16)):
        _chunk(pkv, [4, 1, 6], [9000, 20000, 5], 8, 2, D, bs, BF16)


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0, 40.0])
def test_chunk_scales(pkv, scale):
    for D in (64, 128, 256):
        _chunk(pkv, [70, 1], [300, 200], 6, 2, D, 16, F16, scale=scale)


def test_a_scale_that_is_no_number(pkv):
    x = torch.randn((9, 2, 64), device="cuda").half()
    assert bool(pkv.prompt_attn(x, x, x, _i32([0, 9]), float("nan")).isnan().all())


def _prompt(pkv, nq, nk, hq, hkv, D, dt, causal, seed=0, fused=False, scale=None, **kw):
    g = torch.Generator().manual_seed(seed)
    scale = D ** -0.5 if scale is None else scale
    q, k, v = _rows(sum(nq), hq, hkv, D, dt, g, fused)
    ks = None
    if nk != nq:
        _, k, v = _rows(sum(nk), hq, hkv, D, dt, g, fused)
        ks = _i32(R.starts(nk))
    out = pkv.prompt_attn(q, k, v, _i32(R.starts(nq)), scale, key_starts=ks, causal=causal, **kw)
    ref, bound = R.packed(q, k, v, R.starts(nq), R.starts(nk), scale, causal)
    assert pkv.get_device_error() == 0
    R.check(out, ref, bound)


PROMPTS = {
    "one": ([1], [1]),
    "short": ([5, 40, 1, 17], [5, 40, 1, 17]),
    "edges": ([128, 127, 0, 257, 64], [128, 127, 0, 257, 64]),
    "prefix": ([3, 100, 1], [300, 129, 128]),
    "fewer-keys": ([50, 200, 7], [20, 64, 0]),     # rows before the first key see none
    "long": ([700], [700]),
}


@pytest.mark.parametrize("lens", list(PROMPTS))
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
def test_prompt_lengths(pkv, lens, causal, D, dt):
    nq, nk = PROMPTS[lens]
    _prompt(pkv, nq, nk, 6, 2, D, dt, causal, seed=D, fused=nq == nk)


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 7, 8, 11, 16, 32])
def test_prompt_groups(pkv, G):
    _prompt(pkv, [150, 3, 260], [150, 3, 260], 3 * G, 3, 128, F16 if G % 2 else BF16, True, fused=True)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_partitions(pkv, D, causal):
    _prompt(pkv, [40, 300, 0, 9], [900, 700, 5, 64], 8, 2, D, BF16, causal, split_tokens=128)
    _prompt(pkv, [600, 30], [600, 30], 8, 4, D, F16, causal, split_tokens=200)


def test_prompt_scales(pkv):
    for scale in (0.0, -0.5, 20.0):
        _prompt(pkv, [150, 30], [150, 30], 4, 2, 128, BF16, True, scale=scale)


# ---------------------------------------------------------------- what must not matter
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["k", "v"])
def test_a_bad_token_reaches_only_the_rows_that_see_it(pkv, D, bad, where):
    """A token that is no number: earlier rows of its sequence and other
    sequences know nothing of it."""
    g = torch.Generator().manual_seed(3)
    n = [90, 200, 40]
    q, k, v = _rows(sum(n), 4, 2, D, F16, g)
    ref, bound = R.packed(q, k, v, R.starts(n), R.starts(n), D ** -0.5)
    for at in (89, 90, 100, 217, 218, 289, 290):
        kk, vv = k.clone(), v.clone()
        (kk if where == "k" else vv)[at, 1, 3] = bad
        out = pkv.prompt_attn(q, kk, vv, _i32(R.starts(n)), D ** -0.5)
        seq = next(i for i in range(3) if at < R.starts(n)[i + 1])
        rows = torch.ones(sum(n), dtype=torch.bool)
        rows[at:R.starts(n)[seq + 1]] = False
        R.check(out[rows], ref[rows], bound[rows])
        if where == "v":
            R.check(out[:, :2], ref[:, :2], bound[:, :2])              # the other key head's rows
            ref2, bound2 = R.packed(q, kk, vv, R.starts(n), R.starts(n), D ** -0.5)
            R.check(out, ref2, bound2)


def test_rows_of_no_sequence_stay(pkv):
    g = torch.Generator().manual_seed(4)
    for D in (64, 128, 256):
        q, k, v = _rows(40, 8, 2, D, BF16, g)
        out = torch.full_like(q, 7.0)
        pkv.prompt_attn(q, k, v, _i32([3, 20, 20, 31]), D ** -0.5, out)
        ref, bound = R.packed(q, k, v, [3, 20, 20, 31], [3, 20, 20, 31], D ** -0.5)
        R.check(out[3:31], ref, bound)
        assert bool((out[:3] == 7).all()) and bool((out[31:] == 7).all())


def test_nothing_to_do(pkv):
    q, k, v = (torch.empty((0, h, 128), dtype=F16, device="cuda") for h in (8, 2, 2))
    assert pkv.prompt_attn(q, k, v, _i32([0]), 1.0).shape == q.shape
    assert pkv.prompt_attn(q, k, v, _i32([0, 0, 0]), 1.0).shape == q.shape
    q = torch.randn((5, 8, 128), device="cuda").half()
    assert not bool(pkv.prompt_attn(q, k, v, _i32([0, 3, 5]), 1.0, key_starts=_i32([0, 0, 0])).any())
    cache = torch.full((4, 2, 16, 128), float("nan"), dtype=F16, device="cuda")
    out = pkv.paged_attn_chunk(q, cache, cache, _i32([[-1], [-1]]), _i32([0, 0]), _i32([0, 3, 5]), 1.0)
    assert not bool(out.any()) and pkv.get_device_error() == 0


def test_rows_before_the_first_key_are_zero(pkv):
    """More query rows than cached tokens: the first ones stand before them all."""
    g = torch.Generator().manual_seed(6)
    for D in (64, 128, 256):
        q, k, v = _rows(200, 8, 2, D, F16, g)
        kc, vc, tables = R.paged(k, v, [30], 16, g)
        out = pkv.paged_attn_chunk(q, kc.cuda(), vc.cuda(), tables.cuda(), _i32([30]), _i32([0, 200]), D ** -0.5)
        assert not bool(out[:170].any()) and bool(out[170:].any(-1).all())
        ref, bound = R.attend(q, k[:30], v[:30], D ** -0.5)
        R.check(out, ref, bound)


def test_bad_device_values_are_reported_and_harmless(pkv):
    g = torch.Generator().manual_seed(7)
    D, lens = 128, [100, 60, 200]
    q, k, v = _rows(30, 8, 2, D, F16, g)
    _, k, v = _rows(sum(lens), 8, 2, D, F16, g)
    kc, vc, tables = R.paged(k, v, lens, 16, g)
    kc, vc, st = kc.cuda(), vc.cuda(), [0, 10, 20, 30]
    ref, bound = R.packed(q, k, v, st, R.starts(lens), 0.1)

    def run(tables, lens, st):
        out = torch.full_like(q, 7.0)
        pkv.paged_attn_chunk(q, kc, vc, tables.cuda(), _i32(lens), _i32(st), 0.1, out, max_context_len=208)
        return out, pkv.get_device_error()
    out, code = run(tables, lens, st)
    assert code == 0
    R.check(out, ref, bound)
    bad = tables.clone()
    bad[1, 2] = kc.shape[0]
    out, code = run(bad, lens, st)
    assert code == 1
    R.check(out[:10], ref[:10], bound[:10])
    R.check(out[20:], ref[20:], bound[20:])
    for wrong in (-1, 209):
        out, code = run(tables, [100, wrong, 200], st)
        assert code == 2 and bool((out[10:20] == 7).all())
        R.check(out[:10], ref[:10], bound[:10])
        R.check(out[20:], ref[20:], bound[20:])
    out, code = run(tables, lens, [0, 10, 20, 31])
    assert code == 6 and bool((out[20:] == 7).all())
    R.check(out[:20], ref[:20], bound[:20])
    out, code = run(tables, lens, [-1, 10, 20, 30])
    assert code == 6 and bool((out[:10] == 7).all())
    R.check(out[10:], ref[10:], bound[10:])
    x = torch.full_like(q, 7.0)
    pkv.prompt_attn(q, k, v, _i32([0, 20, 10, 30]), 0.1, x, key_starts=_i32([0, 100, 50, 361]))
    assert pkv.get_device_error() == 6
    # starts that fall: rows would be several sequences', nothing is done
    assert bool((x == 7).all())
    many = torch.randint(-5, 40, (200,), generator=g).tolist()
    pkv.prompt_attn(q, k, v, _i32(many), 0.1, x, key_starts=_i32([0] * 100 + [360] * 100))
    assert pkv.get_device_error() == 6 and bool((x == 7).all())
    # keys that fall leave out their sequence only
    pkv.prompt_attn(q, k, v, _i32([0, 10, 20, 30]), 0.1, x, key_starts=_i32([0, 100, 50, 360]))
    assert pkv.get_device_error() == 6 and bool((x[10:20] == 7).all())
    ref, bound = R.attend(q[:10], k[:100], v[:100], 0.1)
    R.check(x[:10], ref, bound)
    ref, bound = R.attend(q[20:], k[50:], v[50:], 0.1)
    R.check(x[20:], ref, bound)


def test_lengths_counted_in_64_bits(pkv):
    """A bound of the lengths that is far above them: the work is counted in 64
    bits, the rows are the same."""
    g = torch.Generator().manual_seed(13)
    for D, new, lens in ((128, [300, 1, 40], [900, 3000, 40]), (256, [70, 9], [400, 1500]), (64, [500], [600])):
        q = _rows(sum(new), 8, 2, D, F16, g)[0]
        _, k, v = _rows(sum(lens), 8, 2, D, F16, g)
        kc, vc, tables = R.paged(k, v, lens, 32, g)
        wide = torch.full((len(new), 1 << 23), -1, dtype=torch.int32)
        wide[:, :tables.shape[1]] = tables
        out = pkv.paged_attn_chunk(q, kc.cuda(), vc.cuda(), wide.cuda(), _i32(lens), _i32(R.starts(new)), 0.1)
        ref, bound = R.packed(q, k, v, R.starts(new), R.starts(lens), 0.1)
        assert pkv.get_device_error() == 0
        R.check(out, ref, bound)


def test_offsets_past_32_bits(pkv):
    """Blocks, rows and outputs that lie more than 2^32 bytes into their arrays."""
    g = torch.Generator().manual_seed(8)
    D, hkv, bs = 128, 8, 32
    NB = (1 << 32) // (hkv * bs * D * 2) * 2 + 64           # 8 GB a cache
    k, v = (torch.randn((300, hkv, D), generator=g).to(BF16).cuda() for _ in range(2))
    q = torch.randn((60, 16, D), generator=g).to(BF16).cuda()
    kc, vc = (torch.empty((NB, hkv, bs, D), dtype=BF16, device="cuda") for _ in range(2))
    blocks = torch.tensor([NB - 1, 3, NB - 7, NB // 2 + 1, NB - 20, 0, NB - 3, NB - 2, NB - 11, NB - 40], device="cuda")
    for c, x in ((kc, k), (vc, v)):
        c[blocks] = torch.cat([x, torch.full((20, hkv, D), float("nan"), dtype=BF16, device="cuda")]).view(10, bs, hkv, D).transpose(1, 2)
    out = pkv.paged_attn_chunk(q, kc, vc, blocks.int()[None], _i32([300]), _i32([0, 60]), 0.1)
    ref, bound = R.attend(q, k, v, 0.1)
    R.check(out, ref, bound)
    del kc, vc
    # packed rows of a wide projection, the sequence at its end
    T, stride = 300, 1 << 23                                # 16 MB a token row: 4.9 GB
    x = torch.empty((T, stride), dtype=BF16, device="cuda")
    qkv = x[:, stride - 4 * D:].unflatten(1, (4, D))
    qkv.copy_(torch.randn((T, 4, D), generator=g))
    q, k, v = qkv.split([2, 1, 1], 1)
    out = pkv.prompt_attn(q, k, v, _i32([0, 10, 300]), 0.1)
    ref, bound = R.packed(q, k, v, [0, 10, 300], [0, 10, 300], 0.1)
    R.check(out, ref, bound)


def test_the_same_call_gives_the_same_bits(pkv):
    g = torch.Generator().manual_seed(9)
    q, k, v = _rows(700, 8, 2, 128, BF16, g)
    st = _i32([0, 300, 700])
    one = pkv.prompt_attn(q, k, v, st, 0.1, split_tokens=128)
    for _ in range(3):
        assert torch.equal(one, pkv.prompt_attn(q, k, v, st, 0.1, split_tokens=128))


# many items a CTA: one row tile and two in turn, some without keys
@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_short_items(pkv, D):
    g = torch.Generator().manual_seed(11)
    new = torch.randint(0, 4, (1200,), generator=g).tolist()
    ctx = torch.randint(0, 9, (1200,), generator=g).tolist()
    _chunk(pkv, new, ctx, 16, 16, D, 16, F16)


@pytest.mark.parametrize("hq,hkv", [(24, 24), (24, 8)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_ragged_prompts(pkv, hq, hkv, D):
    g = torch.Generator().manual_seed(12)
    nq = torch.randint(0, 420, (48,), generator=g).tolist()
    nk = [max(0, n + d) for n, d in zip(nq, torch.randint(-60, 150, (48,), generator=g).tolist())]
    _prompt(pkv, nq, nk, hq, hkv, D, BF16, True, seed=D)


# rows that begin at 16 bytes, not at 32
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("split", [0, 128])
def test_output_at_16_bytes(pkv, D, split):
    g = torch.Generator().manual_seed(13)
    q, k, v = _rows(333, 6, 2, D, F16, g)
    st = _i32([0, 33, 333])
    one = pkv.prompt_attn(q, k, v, st, 0.1, split_tokens=split)
    room = torch.full((q.numel() + 32,), 7.0, dtype=F16, device="cuda")
    out = room[8:8 + q.numel()].view_as(q)
    assert out.data_ptr() % 32 == 16
    pkv.prompt_attn(q, k, v, st, 0.1, out, split_tokens=split)
    assert torch.equal(one, out)
    assert bool((room[:8] == 7).all()) and bool((room[8 + q.numel():] == 7).all())


# ---------------------------------------------------------------- streams, graphs, workspaces
def test_on_another_stream(pkv):
    g = torch.Generator().manual_seed(10)
    q, k, v = _rows(400, 8, 2, 128, F16, g)
    st = _i32([0, 150, 400])
    want = pkv.prompt_attn(q, k, v, st, 0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pkv.prompt_attn(q, k, v, st, 0.1, stream=side)
    with torch.cuda.stream(side):
        also = pkv.prompt_attn(q, k, v, st, 0.1)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(also, want)


def test_a_captured_chunk_replayed_with_other_lengths(pkv):
    g = torch.Generator().manual_seed(11)
    D, MB = 128, 40
    kc, vc = (torch.randn((3 * MB, 2, 16, D), generator=g).half().cuda() for _ in range(2))
    tables = torch.randperm(3 * MB, generator=g).int().view(3, MB).cuda()
    q = torch.randn((64, 8, D), generator=g).half().cuda()
    lens, st, out = _i32([640, 100, 9]), _i32([0, 30, 50, 59]), torch.zeros_like(q)
    ws = torch.empty(pkv.chunk_workspace_bytes(pkv.chunk_shape(q, kc, tables), 64) + 16, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pkv.paged_attn_chunk(q, kc, vc, tables, lens, st, 0.1, out, workspace=ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pkv.paged_attn_chunk(q, kc, vc, tables, lens, st, 0.1, out, workspace=ws)
    for L, s in (([640, 100, 9], [0, 30, 50, 59]), ([1, 0, 640], [0, 1, 1, 64]), ([5, 640, 7], [0, 0, 40, 40])):
        lens.copy_(_i32(L))
        st.copy_(_i32(s))
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        want = torch.full_like(out, 7)
        pkv.paged_attn_chunk(q, kc, vc, tables, lens, st, 0.1, want)
        assert torch.equal(out, want)
        assert bool((out[s[-1]:] == 7).all())
    assert pkv.get_device_error() == 0


def test_a_set_workspace_serves(pkv):
    g = torch.Generator().manual_seed(12)
    q, k, v = _rows(300, 8, 2, 128, F16, g)
    st = _i32([0, 300])
    want = pkv.prompt_attn(q, k, v, st, 0.1, split_tokens=128)
    n = pkv.prompt_workspace_bytes(pkv.prompt_shape(q, k, v, st, split_tokens=128))
    ws = torch.empty(n + 16, dtype=torch.uint8, device="cuda")
    pkv.set_workspace(ws)
    try:
        assert torch.equal(pkv.prompt_attn(q, k, v, st, 0.1, split_tokens=128), want)
        if n:
            pkv.set_workspace(ws[:16])
            with pytest.raises(pkv.PkvError) as e:
                pkv.prompt_attn(q, k, v, st, 0.1, split_tokens=128)
            assert e.value.code == -5
    finally:
        pkv.set_workspace(None)
