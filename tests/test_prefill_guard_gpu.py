"""Chunk and prompt attention write their out rows and at most the stated bytes of
workspace: both lie in larger allocations whose margins hold a pattern."""
import pytest
import torch

import prefill_ref as R

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
PAD, PATTERN = 4096, 0xA5                  # bytes on each side


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _guarded(nbytes, shift):
    buf = torch.full((nbytes + 2 * PAD + 16,), PATTERN, dtype=torch.uint8, device="cuda")
    return buf[PAD + shift:PAD + shift + nbytes], buf


def _margins(buf, shift, nbytes):
    return bool((buf[:PAD + shift] == PATTERN).all()) and bool((buf[PAD + shift + nbytes:] == PATTERN).all())


@pytest.mark.parametrize("shift", [0, 16])               # on a 32-byte boundary, and not
@pytest.mark.parametrize("D,G,dt", [(64, 1, F16), (64, 5, BF16), (128, 4, BF16), (128, 32, F16), (256, 3, F16), (256, 8, BF16)])
@pytest.mark.parametrize("new,ctx", [([300], [0]), ([3, 1, 0, 40, 9], [1700, 300, 77, 5, 2500]), ([700, 1], [3000, 9000]), ([1] * 40, [333] * 40)])
def test_writes_stay_inside_their_buffers(pkv, D, G, dt, new, ctx, shift):
    g = torch.Generator().manual_seed(D + G)
    lens = [n + c for n, c in zip(new, ctx)]
    q, k, v = (torch.randn((m, h, D), generator=g).to(dt).cuda() for m, h in ((sum(new), 2 * G), (sum(lens), 2), (sum(lens), 2)))
    kc, vc, tables = (x.cuda() for x in R.paged(k, v, lens, 16, g))
    st, ks, cl = _i32(R.starts(new)), _i32(R.starts(lens)), _i32(lens)
    nout = q.numel() * 2
    for split in (0, 128, 1000):
        for paged in (False, True):
            if paged:
                shape = pkv.chunk_shape(q, kc, tables, max(lens), split)
                need = pkv.chunk_workspace_bytes(shape, sum(new))
            else:
                need = pkv.prompt_workspace_bytes(pkv.prompt_shape(q, k, v, st, split_tokens=split))
            ws, wbuf = _guarded(need, shift)
            o, obuf = _guarded(nout, shift)
            out = o.view(dt).view(q.shape)
            kw = dict(split_tokens=split, workspace=ws if need else None)
            if paged:
                pkv.paged_attn_chunk(q, kc, vc, tables, cl, st, 0.1, out, max_context_len=max(lens), **kw)
                want = pkv.paged_attn_chunk(q, kc, vc, tables, cl, st, 0.1, max_context_len=max(lens), split_tokens=split)
            else:
                pkv.prompt_attn(q, k, v, st, 0.1, out, key_starts=ks, **kw)
                want = pkv.prompt_attn(q, k, v, st, 0.1, key_starts=ks, split_tokens=split)
            assert pkv.get_device_error() == 0
            assert torch.equal(out, want)
            assert _margins(wbuf, shift, need) and _margins(obuf, shift, nout)
            if need:                                      # one byte less is refused, before anything runs
                with pytest.raises(pkv.PkvError) as e:
                    if paged:
                        pkv.paged_attn_chunk(q, kc, vc, tables, cl, st, 0.1, out, max_context_len=max(lens),
                                             split_tokens=split, workspace=ws[:-1])
                    else:
                        pkv.prompt_attn(q, k, v, st, 0.1, out, key_starts=ks, split_tokens=split, workspace=ws[:-1])
                assert e.value.code == -5
