"""Keys and values that are no numbers, among the new tokens of a chunk: in pieces
of cut items (partial rows) and through a block table.  A row that sees one has it,
the others know nothing of it."""
import pytest
import torch

import prefill_ref as R

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
NAN, INF = float("nan"), float("inf")


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _batch(D, dt, seed=0):
    """Two sequences that are cut: 150 and 9 new tokens after 700 and 1200."""
    g = torch.Generator().manual_seed(seed + D)
    new, lens = [150, 9], [850, 1209]
    q, k, v = (torch.randn((sum(m), h, D), generator=g).to(dt).cuda() for m, h in ((new, 6), (lens, 2), (lens, 2)))
    return g, new, lens, q, k, v


# tokens by the packed rows' numbers: the first and last new ones, a key tile's ends, both sequences
PLACES = [(700,), (701, 767, 768), (849,), (760, 800, 2050), (850 + 1200, 850 + 1208), (699, 2049)]


@pytest.mark.parametrize("D,bs,dt", [(64, 16, F16), (64, 32, BF16), (128, 16, BF16), (128, 32, F16), (256, 16, BF16), (256, 32, F16)])
@pytest.mark.parametrize("split", [0, 128])
@pytest.mark.parametrize("paged", [False, True])
def test_values_that_are_no_numbers(pkv, D, bs, dt, split, paged):
    g, new, lens, q, k, v = _batch(D, dt)
    st, ks = R.starts(new), R.starts(lens)
    for places in PLACES:
        for n, bads in enumerate(([NAN], [INF], [-INF], [INF, -INF])):
            bad = v.clone()
            for i, t in enumerate(places):
                bad[t, 1, (7 * i + n) % D] = bads[i % len(bads)]
                bad[t, 0, 5] = bads[i % len(bads)]                    # the same channel: they meet
            ref, bound = R.packed(q, k, bad, st, ks, D ** -0.5)
            if paged:
                kc, vc, tables = R.paged(k, bad, lens, bs, g)
                shape = pkv.chunk_shape(q, kc, tables, max(lens), split)
                assert split == 0 or pkv.chunk_workspace_bytes(shape, sum(new)) > 0
                out = pkv.paged_attn_chunk(q, kc.cuda(), vc.cuda(), tables.cuda(), _i32(lens), _i32(st), D ** -0.5,
                                           max_context_len=max(lens), split_tokens=split)
            else:
                out = pkv.prompt_attn(q, k, bad, _i32(st), D ** -0.5, key_starts=_i32(ks), split_tokens=split)
            assert pkv.get_device_error() == 0
            R.check(out, ref, bound)


@pytest.mark.parametrize("D,dt", [(64, F16), (128, BF16), (256, F16)])
@pytest.mark.parametrize("split", [0, 128])
def test_keys_that_are_no_numbers(pkv, D, dt, split):
    g, new, lens, q, k, v = _batch(D, dt)
    st, ks = R.starts(new), R.starts(lens)
    for places in PLACES:
        bad = k.clone()
        for t in places:
            bad[t, 1, t % D] = NAN
        ref, bound = R.packed(q, bad, v, st, ks, D ** -0.5)
        # (the plain form's weights of a row are all NaN where one is)
        kc, vc, tables = R.paged(bad, v, lens, 16, g)
        out = pkv.paged_attn_chunk(q, kc.cuda(), vc.cuda(), tables.cuda(), _i32(lens), _i32(st), D ** -0.5, split_tokens=split)
        R.check(out, ref, bound)
        R.check(pkv.prompt_attn(q, bad, v, _i32(st), D ** -0.5, key_starts=_i32(ks), split_tokens=split), ref, bound)
    assert pkv.get_device_error() == 0
