"""The prompt side as it is used: prompts that enter the cache in chunks, mixed
steps, prefixes from a 4-bit cache, forks, several streams and graphs; and
seeded batches of every kind against the plain 64-bit forms."""
import random

import pytest
import torch

import prefill_ref as R

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("D,sections", [(64, None), (128, (16, 24, 24)), (256, (32, 48, 48))])
@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
def test_a_prompt_in_chunks_then_decode(pkv, D, sections, dt):
    """rope_append and paged_attn_chunk, chunk by chunk, with two prompts that
    advance at different rates; then one decode step.  The rows are those of
    prompt_attn on the whole prompts, and the decode's those of a chunk of one."""
    g = torch.Generator().manual_seed(D)
    hq, hkv, bs, lens = 8, 2, 16, [431, 150]
    rows = [torch.randn((n + 1, hq + 2 * hkv, D), generator=g).to(dt).cuda() for n in lens]
    pos = [torch.arange(n + 1, dtype=torch.int32) for n in lens]
    if sections:
        pos = [torch.stack([p, p // 7, p % 7]) for p in pos]
    pos = [p.cuda() for p in pos]
    table, MB = pkv.rope_table(1024, D), 40
    tables = torch.randperm(2 * MB + 5, generator=g)[:2 * MB].int().view(2, MB).cuda()
    kc, vc = (torch.full((2 * MB + 5, hkv, bs, D), float("nan"), dtype=dt, device="cuda") for _ in range(2))
    kw = dict(sections=sections) if sections else {}
    done, outs, qs = [0, 0], [[], []], [[], []]
    for step in ([100, 1], [17, 60], [300, 0], [14, 89]):
        part = [r[d:d + n] for r, d, n in zip(rows, done, step)]
        x, p = torch.cat(part), torch.cat([q[..., d:d + n] for q, d, n in zip(pos, done, step)], -1).contiguous()
        q, k, v = x.split([hq, hkv, hkv], 1)
        t = [torch.arange(d, d + n, device="cuda") for d, n in zip(done, step)]
        slots = torch.cat([tables[i, a // bs] * bs + a % bs for i, a in enumerate(t)]).int()
        turned = pkv.rope_append(q, k, v, p, table, slots, kc, vc, **kw)
        done = [d + n for d, n in zip(done, step)]
        out = pkv.paged_attn_chunk(turned, kc, vc, tables, _i32(done), _i32(R.starts(step)), D ** -0.5)
        for i, (o, z) in enumerate(zip(out.split(step), turned.split(step))):
            outs[i].append(o)
            qs[i].append(z)
    assert done == lens and pkv.get_device_error() == 0
    # the keys as the cache holds them
    t = [torch.arange(n, device="cuda") for n in lens]
    k, v = (torch.cat([c[tables[i, a // bs].long(), :, a % bs] for i, a in enumerate(t)]) for c in (kc, vc))
    q, st = torch.cat([torch.cat(x) for x in qs]), R.starts(lens)
    ref, bound = R.packed(q, k, v, st, st, D ** -0.5)
    R.check(torch.cat([torch.cat(x) for x in outs]), ref, bound)
    R.check(pkv.prompt_attn(q, k, v, _i32(st), D ** -0.5), ref, bound)
    # one decode step, and the same as a chunk of one token each
    x = torch.stack([r[-1] for r in rows])
    p = torch.stack([q[..., -1] for q in pos], -1).contiguous()
    slots = torch.stack([tables[i, n // bs] * bs + n % bs for i, n in enumerate(lens)]).int()
    q, k, v = x.split([hq, hkv, hkv], 1)
    turned = pkv.rope_append(q, k, v, p, table, slots, kc, vc, **kw)
    L = _i32([n + 1 for n in lens])
    a = pkv.paged_attn_decode(turned, kc, vc, tables, L, D ** -0.5)
    b = pkv.paged_attn_chunk(turned, kc, vc, tables, L, _i32([0, 1, 2]), D ** -0.5)
    t = [torch.arange(n + 1, device="cuda") for n in lens]
    k, v = (torch.cat([c[tables[i, a_ // bs].long(), :, a_ % bs] for i, a_ in enumerate(t)]) for c in (kc, vc))
    ref, bound = R.packed(turned, k, v, [0, 1, 2], R.starts([n + 1 for n in lens]), D ** -0.5)
    R.check(a, ref, bound + 2 * R.HALF[dt] * ref.abs().amax())     # (the decode kernels' own roundings)
    R.check(b, ref, bound)


@pytest.mark.parametrize("D,bs", [(64, 16), (128, 32), (256, 16)])
def test_a_chunk_after_a_4_bit_prefix(pkv, D, bs):
    """kv4_append, kv4_gather and prompt_attn: the chunk attends over the rows as
    the 4-bit cache holds them, and its last row is what decode gives."""
    g = torch.Generator().manual_seed(D)
    hq, hkv, back, n, dt = 8, 4, 333, 90, F16
    x = torch.randn((back + n, hq + 2 * hkv, D), generator=g).to(dt).cuda()
    pos = torch.arange(back + n, dtype=torch.int32, device="cuda")
    NB = (back + n) // bs + 4
    blocks = torch.randperm(NB, generator=g).int().cuda()
    slots = blocks[pos.long() // bs] * bs + pos % bs
    table = pkv.rope_table(1024, D)
    k4, v4 = pkv.kv4_cache(NB, hkv, bs, D), pkv.kv4_cache(NB, hkv, bs, D)
    q, k, v = x.split([hq, hkv, hkv], 1)
    pkv.kv4_append(None, k[:back], v[:back], pos[:back], table, slots[:back], k4, v4)
    turned = pkv.kv4_append(q[back:], k[back:], v[back:], pos[back:], table, slots[back:], k4, v4)
    rk, rv = pkv.kv4_gather(k4, v4, slots, dt)
    out = pkv.prompt_attn(turned, rk, rv, _i32([0, n]), D ** -0.5, key_starts=_i32([0, back + n]))
    ref, bound = R.attend(turned, rk, rv, D ** -0.5)
    R.check(out, ref, bound)
    one = pkv.kv4_attn_decode(turned[-1:].contiguous(), k4, v4, blocks[None].contiguous(), _i32([back + n]), D ** -0.5)
    # (the decode reads the cache's values before their rounding to 16 bits)
    assert float((one.double() - ref[-1:]).abs().max()) < 8 * R.HALF[dt] * float(rv.abs().max())
    assert pkv.get_device_error() == 0


def test_forked_sequences_share_their_prompt(pkv):
    """A prompt, two forks of it that go on differently: copy-on-write of the last
    block, then one step with drafted tokens for all three."""
    g = torch.Generator().manual_seed(1)
    D, bs, hq, hkv, n, dt = 128, 16, 8, 2, 75, BF16
    bm = pkv.BlockManager(64, 0, bs)
    bm.add_sequence(0, n)
    x = torch.randn((n, hq + 2 * hkv, D), generator=g).to(dt).cuda()
    kc, vc = (torch.full((64, hkv, bs, D), float("nan"), dtype=dt, device="cuda") for _ in range(2))
    table, lens = pkv.rope_table(256, D), [n]
    tables = torch.from_numpy(bm.block_tables([0], 16)[0]).cuda()
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    slots = (tables[0, (pos // bs).long()] * bs + pos % bs).int()
    q, k, v = x.split([hq, hkv, hkv], 1)
    turned = pkv.rope_append(q, k, v, pos, table, slots, kc, vc)
    first = pkv.paged_attn_chunk(turned, kc, vc, tables, _i32([n]), _i32([0, n]), D ** -0.5)
    bm.fork(0, 1)
    bm.fork(0, 2)
    new = [3, 1, 6]
    slots, pairs = [], []
    for i, m in enumerate(new):
        for _ in range(m):
            slot, src, dst = bm.append_token(i)
            slots.append(slot)
            if src >= 0:
                pairs.append((src, dst))
    pkv.copy_blocks(kc, vc, kc, vc, _i32(pairs).view(-1, 2))
    x = torch.randn((sum(new), hq + 2 * hkv, D), generator=g).to(dt).cuda()
    q, k, v = x.split([hq, hkv, hkv], 1)
    pos = torch.cat([torch.arange(n, n + m) for m in new]).int().cuda()
    turned = pkv.rope_append(q, k, v, pos, table, _i32(slots), kc, vc)
    tables, lens = bm.block_tables([0, 1, 2], 16)
    out = pkv.paged_attn_chunk(turned, kc, vc, torch.from_numpy(tables).cuda(), _i32(lens.tolist()),
                               _i32(R.starts(new)), D ** -0.5)
    assert lens.tolist() == [n + m for m in new] and pkv.get_device_error() == 0
    tables = torch.from_numpy(tables).long().cuda()
    t = [torch.arange(m, device="cuda") for m in lens.tolist()]
    k, v = (torch.cat([c[tables[i, a // bs], :, a % bs] for i, a in enumerate(t)]) for c in (kc, vc))
    ref, bound = R.packed(turned, k, v, R.starts(new), R.starts(lens.tolist()), D ** -0.5)
    R.check(out, ref, bound)
    assert bool(first.isfinite().all())


# ---------------------------------------------------------------- streams, graphs, memory
def test_two_calls_at_once(pkv):
    """Two streams, each with its own workspace."""
    g = torch.Generator().manual_seed(2)
    x = [torch.randn((1500, 12, 128), generator=g).to(BF16).cuda() for _ in range(2)]
    st = _i32([0, 1300, 1500])
    parts = [t.split([8, 2, 2], 1) for t in x]
    want = [pkv.prompt_attn(*p, st, 0.1, split_tokens=128) for p in parts]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = []
        for s, p in zip(streams, parts):
            with torch.cuda.stream(s):
                got.append(pkv.prompt_attn(*p, st, 0.1, split_tokens=128))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_graphs_share_a_workspace(pkv):
    """Captured once, replayed in turn on one stream: nothing of one is left for the other."""
    g = torch.Generator().manual_seed(3)
    x = [torch.randn((n, 12, 128), generator=g).half().cuda() for n in (900, 1400)]
    parts = [t.split([8, 2, 2], 1) for t in x]
    st = [_i32([0, 900]), _i32([0, 700, 700, 1400])]
    want = [pkv.prompt_attn(*p, s, 0.1, split_tokens=128) for p, s in zip(parts, st)]
    need = max(pkv.prompt_workspace_bytes(pkv.prompt_shape(*p, s, split_tokens=128)) for p, s in zip(parts, st))
    ws = torch.randint(0, 256, (need + 16,), dtype=torch.uint8, device="cuda")
    outs, graphs, side = [torch.zeros_like(w) for w in want], [], torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for p, s, o in zip(parts, st, outs):
        with torch.cuda.stream(side):
            pkv.prompt_attn(*p, s, 0.1, o, split_tokens=128, workspace=ws)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            pkv.prompt_attn(*p, s, 0.1, o, split_tokens=128, workspace=ws)
        graphs.append(graph)
    for i in (0, 1, 1, 0, 1):
        outs[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], want[i])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_out_on_a_16_byte_boundary(pkv, D):
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn((210, h, D), generator=g).half().cuda() for h in (6, 2, 2))
    st = _i32([0, 33, 210])
    want = pkv.prompt_attn(q, k, v, st, 0.1)
    buf = torch.full((q.numel() + 32,), 7.0, dtype=F16, device="cuda")
    for off in (8, 16, 24):
        out = buf[off:off + q.numel()].view_as(q)
        assert torch.equal(pkv.prompt_attn(q, k, v, st, 0.1, out), want)
        assert bool((buf[:off] == 7).all()) and bool((buf[off + q.numel():] == 7).all())
        buf.fill_(7)


def test_refusals_on_the_gpu(pkv):
    q, k = torch.zeros((8, 4, 64), dtype=F16, device="cuda"), torch.zeros((8, 2, 64), dtype=F16, device="cuda")
    st = _i32([0, 8])
    for kw in (dict(q=q[:, :3]), dict(q=q.bfloat16()), dict(k=k.bfloat16()), dict(q=q.transpose(0, 1)),
               dict(q=q[..., ::2]), dict(st=st.long()), dict(st=st[None]), dict(k=k[:, :1]),
               dict(q=torch.zeros((8, 66, 64), dtype=F16, device="cuda")),
               dict(q=torch.zeros(8 * 4 * 64 + 2, dtype=F16, device="cuda")[1:-1].view(8, 4, 64)),
               dict(q=torch.zeros(8, 4 * 64 + 4, dtype=F16, device="cuda")[:, :256].unflatten(1, (4, 64)))):
        a = dict(q=q, k=k, st=st)
        a.update(kw)
        v = torch.zeros_like(k)
        with pytest.raises((ValueError, pkv.PkvError)):
            pkv.prompt_attn(a["q"], a["k"], v, a["st"], 1.0)
    with pytest.raises(pkv.PkvError):
        pkv.prompt_attn(q, k, k, st, 1.0, split_tokens=-1)
    with pytest.raises(ValueError):
        pkv.prompt_attn(q, k, k, st, 1.0, key_starts=_i32([0, 4, 8]))


# ---------------------------------------------------------------- values
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("grow", [0.03, 0.5, -0.5])
def test_logits_that_grow_along_the_keys(pkv, D, dt, grow):
    """The running maximum moves at nearly every key tile (or never again)."""
    g = torch.Generator().manual_seed(5)
    n, L = 150, 1100
    q, k, v = (torch.randn((m, h, D), generator=g) for m, h in ((n, 4), (L, 2), (L, 2)))
    along = torch.arange(L).float() * grow
    q = q.sign()
    k = (0.1 * k + along[:, None, None] / D * q[0, 0])      # q . k grows by `grow` a key for the first row
    q, k, v = q.to(dt).cuda(), k.to(dt).cuda(), v.to(dt).cuda()
    out = pkv.prompt_attn(q, k, v, _i32([0, n]), 1.0, key_starts=_i32([0, L]))
    ref, bound = R.attend(q, k, v, 1.0)
    R.check(out, ref, bound)
    assert torch.equal(out, pkv.prompt_attn(q, k, v, _i32([0, n]), 1.0, key_starts=_i32([0, L])))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_far_weights_keep_their_share(pkv, D):
    """One key far above 4000 equal others in binary16: their small weights add up."""
    L, gap = 4096, 13.0
    q = torch.zeros((1, 1, D), dtype=F16, device="cuda")
    k = torch.zeros((L, 1, D), dtype=F16, device="cuda")
    q[..., 0], k[7, 0, 0] = 1, gap
    v = torch.ones((L, 1, D), dtype=F16, device="cuda")
    v[7] = -1
    out = pkv.prompt_attn(q, k, v, _i32([0, 1]), 1.0, key_starts=_i32([0, L]))
    ref, bound = R.attend(q, k, v, 1.0)
    R.check(out, ref, bound)
    assert abs(float(ref[0, 0, 0]) + 1) > 1e-2               # (their share shows)


def test_large_values(pkv):
    """Values at the type's ends, logits in the thousands."""
    g = torch.Generator().manual_seed(6)
    for dt, most in ((F16, 60000.0), (BF16, 3e38)):
        q, k, v = (torch.randn((130, h, 128), generator=g) for h in (4, 2, 2))
        out = pkv.prompt_attn((30 * q).to(dt).cuda(), (30 * k).to(dt).cuda(), (v.clamp(-1, 1) * most).to(dt).cuda(),
                              _i32([0, 130]), 1.0)
        ref, bound = R.attend((30 * q).to(dt).cuda(), (30 * k).to(dt).cuda(), (v.clamp(-1, 1) * most).to(dt).cuda(), 1.0)
        fine = ref.abs() + bound < most
        assert bool(((out.double() - ref).abs() <= bound)[fine].all())


# ---------------------------------------------------------------- seeded batches of every kind
@pytest.mark.parametrize("seed", range(40))
def test_seeded_batches(pkv, seed):
    rng, g = random.Random(seed), torch.Generator().manual_seed(seed)
    D, dt = rng.choice([64, 128, 256]), rng.choice([F16, BF16])
    hkv, G = rng.choice([1, 2, 3, 4]), rng.choice([1, 2, 3, 4, 5, 8, 13, 16, 32])
    while hkv * G > 48:
        G = max(1, G // 2)
    B = rng.choice([1, 2, 3, 7, 33, 70])
    top = rng.choice([1, 9, 300]) if B > 5 else rng.choice([1, 9, 300, 900])
    far = rng.choice([0, 40, 700]) if B > 5 else rng.choice([0, 40, 700, 3000])
    new = [rng.randrange(0, top + 1) for _ in range(B)]
    lens = [n + rng.randrange(0, far + 1) for n in new]
    if sum(new) == 0:
        new[0], lens[0] = 1, max(1, lens[0])
    causal, split = rng.random() < 0.7, rng.choice([0, 0, 1, 200, 4000])
    scale = rng.choice([D ** -0.5, D ** -0.5, 0.5, -0.2])
    x = torch.randn((sum(new), hkv * (G + 2), D), generator=g).to(dt).cuda()
    q = x[:, :hkv * G] if rng.random() < 0.5 else x[:, :hkv * G].contiguous()
    k, v = (torch.randn((sum(lens), hkv, D), generator=g).to(dt).cuda() for _ in range(2))
    st = R.starts(new)
    if rng.random() < 0.5:
        bs = rng.choice([16, 32])
        kc, vc, tables = R.paged(k, v, lens, bs, g)
        out = pkv.paged_attn_chunk(q, kc.cuda(), vc.cuda(), tables.cuda(), _i32(lens), _i32(st), scale, split_tokens=split)
        causal = True
    else:
        out = pkv.prompt_attn(q, k, v, _i32(st), scale, key_starts=_i32(R.starts(lens)), causal=causal, split_tokens=split)
    assert pkv.get_device_error() == 0
    ref, bound = R.packed(q, k, v, st, R.starts(lens), scale, causal)
    R.check(out, ref, bound)


def test_very_many_sequences(pkv):
    g = torch.Generator().manual_seed(7)
    new = torch.randint(0, 3, (3001,), generator=g).tolist()
    lens = [n + m for n, m in zip(new, torch.randint(0, 30, (3001,), generator=g).tolist())]
    q, k, v = (torch.randn((n, h, 64), generator=g).half().cuda() for n, h in ((sum(new), 4), (sum(lens), 2), (sum(lens), 2)))
    out = pkv.prompt_attn(q, k, v, _i32(R.starts(new)), 0.125, key_starts=_i32(R.starts(lens)))
    # a plain form over all pairs, the other sequences' keys masked
    seq_q = torch.repeat_interleave(torch.arange(3001), torch.tensor(new)).cuda()
    seq_k = torch.repeat_interleave(torch.arange(3001), torch.tensor(lens)).cuda()
    end = torch.tensor(R.starts(lens)[1:], device="cuda")
    last = torch.cat([torch.arange(b - n, b) for n, b in zip(new, R.starts(lens)[1:])]).cuda() if sum(new) else None
    for at in range(0, sum(new), 500):
        s = slice(at, at + 500)
        seen = (seq_q[s, None] == seq_k[None]) & (torch.arange(sum(lens), device="cuda")[None] <= last[s, None])
        a = torch.einsum("nhd,thd->hnt", q[s].double(), k.double().repeat_interleave(2, 1)) * 0.125
        w = torch.softmax(a.masked_fill(~seen, float("-inf")), -1)
        ref = torch.einsum("hnt,thd->nhd", w, v.double().repeat_interleave(2, 1))
        A = torch.einsum("hnt,thd->nhd", w, v.double().abs().repeat_interleave(2, 1))
        assert bool(((out[s].double() - ref).abs() <= 2.0 ** -11 * ref.abs() + A * (2.0 ** -11 + 2.0 ** -14) + 2.0 ** -18).all())
    assert end.numel() == 3001 and pkv.get_device_error() == 0
