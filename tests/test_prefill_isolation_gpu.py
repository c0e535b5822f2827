"""A row of a chunk or a prompt is its own sequence's alone: its bits stay the
same whatever the rows beside it in a tile, the cache's unwritten slots and the
calls before it hold."""
import pytest
import torch

import prefill_ref as R

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _randn(shape, g, dt, by=1.0):
    return (by * torch.randn(shape, generator=g)).to(dt).cuda()


@pytest.mark.parametrize("G", [3, 5, 6, 7, 9, 12])
@pytest.mark.parametrize("D,dt", [(64, F16), (128, BF16), (128, F16), (256, BF16)])
def test_calls_before_leave_nothing(pkv, G, D, dt):
    """Groups that fill no row tile: the tile's last rows are what was in shared memory."""
    g = torch.Generator().manual_seed(G + D)
    n, L = 150, 2300
    q, k, v = (_randn((m, h, D), g, dt) for m, h in ((n, 2 * G), (L, 2), (L, 2)))
    big = [_randn((600, 8, D), g, dt, by) for by in (40.0, 0.01)]
    st, ks = _i32([0, n]), _i32([0, L])
    outs = []
    for x in big * 2:
        pkv.prompt_attn(x, x, x, _i32([0, 600]), 1.0, causal=False)
        outs.append(pkv.prompt_attn(q, k, v, st, D ** -0.5, key_starts=ks))
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


@pytest.mark.parametrize("D,bs,G,dt", [(64, 16, 1, F16), (128, 16, 4, BF16), (128, 32, 3, F16), (256, 16, 2, BF16)])
def test_neighbours_and_unwritten_slots_leave_nothing(pkv, D, bs, G, dt):
    """Few new tokens a sequence: most rows of a tile are other sequences' queries,
    which would see past the sequence's end."""
    g = torch.Generator().manual_seed(G + D)
    new, lens = [1, 3, 2, 1], [2049 - 5, 1501, 700, 2049]
    k, v = (_randn((sum(lens), 2, D), g, dt) for _ in range(2))
    q = _randn((sum(new), 2 * G, D), g, dt)
    kc, vc, tables = R.paged(k, v, lens, bs, g, fill=0.0)
    st, cl, tables = _i32(R.starts(new)), _i32(lens), tables.cuda()
    empty = torch.ones(kc.shape[:3:2], dtype=torch.bool)              # [NB, bs]: slots that no token has
    for i, n in enumerate(lens):
        t = torch.arange(n)
        empty[tables[i].cpu().long()[t // bs], t % bs] = False
    kc, vc = kc.cuda(), vc.cuda()
    want = pkv.paged_attn_chunk(q, kc, vc, tables, cl, st, D ** -0.5)
    for by in (50.0, -50.0, float("nan"), float("inf")):
        for c in (kc, vc):
            c.transpose(1, 2)[empty.cuda()] = by
        assert torch.equal(pkv.paged_attn_chunk(q, kc, vc, tables, cl, st, D ** -0.5), want)
    # every sequence but one gets other queries
    for i in range(len(new)):
        rows = torch.zeros(sum(new), dtype=torch.bool)
        rows[R.starts(new)[i]:R.starts(new)[i + 1]] = True
        for by in (60.0, float("nan")):
            other = q.clone()
            other[~rows] = other[~rows] * by
            got = pkv.paged_attn_chunk(other, kc, vc, tables, cl, st, D ** -0.5)
            assert torch.equal(got[rows], want[rows])
