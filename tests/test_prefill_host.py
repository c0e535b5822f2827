"""Chunk and prompt attention and the rotation of several axes on the CPU: the
refusals of the C ABI and of the binding, and how the work is cut over the CTAs
(no call here reaches a GPU)."""
import ctypes

import pytest
import torch

from paged_kv_cache_268_gb300 import _binding as B
from paged_kv_cache_268_gb300 import build

FAKE = 0x10000  # 16-byte aligned non-null address; never dereferenced on the host


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.load_library()


def _shape(**kw):
    base = dict(num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16, num_blocks=64,
                max_blocks_per_seq=8, max_context_len=100, dtype=0)
    base.update(kw)
    return B.make_shape(**base)


def _chunk(lib, shape, q=FAKE, stride=0, T=5, st=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, cl=FAKE, out=FAKE):
    return lib.pkv_paged_attn_chunk(None if shape is None else ctypes.byref(shape), q, stride, T, st, kc, vc, bt,
                                    cl, 0.1, out, None, 0, None)


@pytest.mark.parametrize("kw,code", [
    (dict(num_q_heads=6, num_kv_heads=4), -2), (dict(num_kv_heads=0), -2), (dict(num_seqs=-1), -2),
    (dict(max_context_len=0), -2), (dict(max_context_len=129), -2), (dict(split_tokens=-1), -2),
    (dict(head_dim=96), -3), (dict(block_size=8), -3), (dict(dtype=5), -3), (dict(kernel=1), -3),
    (dict(kernel=3), -3), (dict(num_q_heads=66), -3),
    (dict(max_blocks_per_seq=1 << 27, max_context_len=(1 << 30) + 1), -3),
])
def test_chunk_rejects_bad_shapes(lib, kw, code):
    assert _chunk(lib, _shape(**kw)) == code


def test_chunk_rejects_bad_arguments(lib):
    assert _chunk(lib, None) == -1
    for name in ("q", "st", "kc", "vc", "bt", "cl", "out"):
        assert _chunk(lib, _shape(), **{name: None}) == -1
        assert _chunk(lib, _shape(), **{name: FAKE + 2}) == -4
    assert _chunk(lib, _shape(), T=-1) == -2
    assert _chunk(lib, _shape(), T=(1 << 30) + 1) == -3
    assert _chunk(lib, _shape(), stride=8 * 128 - 8) == -2
    assert _chunk(lib, _shape(), stride=8 * 128 + 4) == -4
    assert _chunk(lib, _shape(), stride=1 << 39) == -3
    assert _chunk(lib, _shape(num_seqs=0), q=None) == 0        # nothing to do
    assert _chunk(lib, _shape(), T=0, q=None) == 0
    assert lib.pkv_launch_count() == 0


def _prompt(**kw):
    base = dict(num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=128, num_tokens=5, num_keys=5, dtype=0,
                causal=1, split_tokens=0, q_stride=0, k_stride=0, v_stride=0)
    base.update(kw)
    return B.Prompt(*[base[n] for n, _ in B.Prompt._fields_])


def _attn(lib, p, q=FAKE, k=FAKE, v=FAKE, qs=FAKE, ks=FAKE, out=FAKE):
    return lib.pkv_prompt_attn(None if p is None else ctypes.byref(p), q, k, v, qs, ks, 0.1, out, None, 0, None)


@pytest.mark.parametrize("kw,code", [
    (dict(num_q_heads=6, num_kv_heads=4), -2), (dict(num_kv_heads=0), -2), (dict(num_seqs=-1), -2),
    (dict(num_tokens=-1), -2), (dict(num_keys=-1), -2), (dict(split_tokens=-1), -2),
    (dict(head_dim=80), -3), (dict(dtype=2), -3), (dict(num_q_heads=66), -3), (dict(num_keys=(1 << 30) + 1), -3),
    (dict(q_stride=1016), -2), (dict(k_stride=248), -2), (dict(v_stride=248), -2),
    (dict(q_stride=1028), -4), (dict(k_stride=260), -4), (dict(v_stride=260), -4),
    (dict(q_stride=1 << 39), -3), (dict(k_stride=1 << 39), -3),
])
def test_prompt_rejects_bad_sizes(lib, kw, code):
    assert _attn(lib, _prompt(**kw)) == code


def test_prompt_rejects_bad_arguments(lib):
    assert _attn(lib, None) == -1
    for name in ("q", "k", "v", "qs", "ks", "out"):
        assert _attn(lib, _prompt(), **{name: None}) == -1
        assert _attn(lib, _prompt(), **{name: FAKE + 2}) == -4
    assert _attn(lib, _prompt(num_seqs=0), q=None) == 0
    assert _attn(lib, _prompt(num_tokens=0), q=None) == 0
    n = ctypes.c_size_t(0)
    assert lib.pkv_prompt_workspace_bytes(None, ctypes.byref(n)) == -1
    assert lib.pkv_prompt_workspace_bytes(ctypes.byref(_prompt()), None) == -1
    assert lib.pkv_chunk_workspace_bytes(ctypes.byref(_shape(head_dim=48)), 5, ctypes.byref(n)) == -3
    assert lib.pkv_chunk_workspace_bytes(ctypes.byref(_shape()), -1, ctypes.byref(n)) == -2


def _axes_call(lib, axes, rope=None, fn="pkv_rope_append_axes"):
    rope = rope or B.Rope(128, 0, 64, 0, 0, 0)
    return getattr(lib, fn)(ctypes.byref(_shape()), ctypes.byref(rope), axes, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 5,
                            FAKE, FAKE, FAKE, None)


@pytest.mark.parametrize("fn", ["pkv_rope_append_axes", "pkv_kv4_append_axes"])
def test_axes_rejects_bad_sections(lib, fn):
    def axes(n, *sections):
        return ctypes.byref(B.RopeAxes(n, (ctypes.c_int32 * 4)(*sections)))
    assert _axes_call(lib, None, fn=fn) == -1
    assert _axes_call(lib, axes(0), fn=fn) == -2
    assert _axes_call(lib, axes(5, 16, 16, 16, 16), fn=fn) == -2
    assert _axes_call(lib, axes(3, 16, 24, 23), fn=fn) == -2
    assert _axes_call(lib, axes(3, 16, 24, 25), fn=fn) == -2
    assert _axes_call(lib, axes(3, -16, 56, 24), fn=fn) == -2
    assert _axes_call(lib, axes(2, 2 ** 31 - 1, 2 ** 31 - 1), fn=fn) == -2
    assert _axes_call(lib, axes(1, 0), B.Rope(0, 0, 64, 0, 0, 0), fn=fn) == -2


# ---------------------------------------------------------------- the binding
@pytest.fixture
def on_cpu(monkeypatch):
    """The checks that ask for CUDA tensors are lifted, so that the others are reached."""
    def dense(t, name, dtype=None):
        if not t.is_contiguous() or (dtype is not None and t.dtype != dtype):
            raise ValueError(name)
    monkeypatch.setattr(B, "_dense", dense)
    monkeypatch.setattr(B, "_one_device", lambda **kw: torch.device("cpu"))


def _chunk_args(**kw):
    f16, i32 = torch.float16, torch.int32
    a = dict(q=torch.zeros(5, 8, 64, dtype=f16), k_cache=torch.zeros(6, 2, 16, 64, dtype=f16),
             v_cache=torch.zeros(6, 2, 16, 64, dtype=f16), block_tables=torch.zeros(3, 2, dtype=i32),
             context_lens=torch.zeros(3, dtype=i32), query_starts=torch.zeros(4, dtype=i32), out=None, workspace=None)
    a.update(kw)
    return a


def test_chunk_binding_checks_extents(on_cpu):
    f16, i32 = torch.float16, torch.int32
    B._check_chunk(**_chunk_args())
    for kw in (dict(v_cache=torch.zeros(6, 2, 32, 64, dtype=f16)), dict(v_cache=torch.zeros(6, 2, 16, 64)),
               dict(q=torch.zeros(5, 8, 128, dtype=f16)), dict(q=torch.zeros(5, 512, dtype=f16)),
               dict(q=torch.zeros(5, 8, 64, dtype=torch.bfloat16)),
               dict(context_lens=torch.zeros(4, dtype=i32)), dict(block_tables=torch.zeros(4, 2, dtype=i32)),
               dict(query_starts=torch.zeros(3, dtype=i32)), dict(query_starts=torch.zeros(4, dtype=torch.int64)),
               dict(query_starts=torch.zeros(0, dtype=i32)), dict(query_starts=torch.zeros((4, 1), dtype=i32)),
               dict(out=torch.zeros(5, 8, 128, dtype=f16)), dict(out=torch.zeros(5, 8, 64)),
               dict(block_tables=torch.zeros(6, dtype=i32)),
               dict(k_cache=torch.zeros(6, 2, 16, 64), v_cache=torch.zeros(6, 2, 16, 64))):
        with pytest.raises(ValueError):
            B._check_chunk(**_chunk_args(**kw))


def test_prompt_binding_checks_extents(on_cpu):
    f16, i32 = torch.float16, torch.int32

    def args(**kw):
        a = dict(q=torch.zeros(5, 8, 64, dtype=f16), k=torch.zeros(7, 2, 64, dtype=f16),
                 v=torch.zeros(7, 2, 64, dtype=f16), query_starts=torch.zeros(4, dtype=i32),
                 key_starts=torch.zeros(4, dtype=i32), out=None, workspace=None)
        a.update(kw)
        return a
    B._check_prompt(**args())
    for kw in (dict(k=torch.zeros(7, 2, 128, dtype=f16)), dict(v=torch.zeros(6, 2, 64, dtype=f16)),
               dict(key_starts=torch.zeros(3, dtype=i32)), dict(query_starts=torch.zeros((2, 2), dtype=i32)),
               dict(q=torch.zeros(5, 512, dtype=f16)), dict(q=torch.zeros(5, 8, 64)),
               dict(out=torch.zeros(4, 8, 64, dtype=f16))):
        with pytest.raises(ValueError):
            B._check_prompt(**args(**kw))


def test_cpu_tensors_are_refused():
    a = _chunk_args()
    with pytest.raises(ValueError):
        B.paged_attn_chunk(a["q"], a["k_cache"], a["v_cache"], a["block_tables"], a["context_lens"],
                           a["query_starts"], 1.0)
    x, st = torch.zeros(5, 2, 64, dtype=torch.float16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        B.prompt_attn(x, x, x, st, 1.0)


def test_sizes_past_32_bits_are_refused():
    q = torch.empty((2 ** 31, 8, 64), dtype=torch.float16, device="meta")
    k = torch.empty((4, 8, 64), dtype=torch.float16, device="meta")
    with pytest.raises(ValueError):
        B._prompt(1, 8, 8, 64, q.shape[0], k.shape[0], 0, True, 0, 0, 0, 0)


# ---------------------------------------------------------------- how the work is cut
# The scheduler's arithmetic once more, in Python integers: items of a key head
# lie on a line, the lines one after the other are cut into equal lengths, one a
# CTA, and a cut is moved to a key tile that leaves no piece too short.
KEY, ITEM, TOKEN, KEY1, ITEM1 = 3, 3 * 320, 3, 2, 3 * 320


def _keys(n, L, per, t, causal):
    return L if not causal else max(0, L - n + min((t + 1) * per, n))


def _cost(n, L, per, half, t, causal):
    k = _keys(n, L, per, t, causal)
    if half < per and n - t * per <= half:
        return k * KEY1 + ITEM1 + causal * half * TOKEN
    return k * KEY + ITEM + causal * per * TOKEN


def _begin(n, L, per, t, causal):
    if not causal:
        keys = t * L
    else:
        d = L - n
        blind = (n - L) // per if d < 0 else 0
        keys = 0 if t <= blind else (t - blind) * d + per * ((t * (t + 1) - blind * (blind + 1)) // 2)
    return t * (ITEM + causal * per * TOKEN) + keys * KEY


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,L", [(1, 1), (1, 5000), (300, 300), (257, 4000), (1000, 30), (1000, 999), (64, 0), (511, 100)])
@pytest.mark.parametrize("G,tiles", [(1, 2), (4, 2), (7, 2), (32, 2), (1, 1), (12, 1)])
def test_items_lie_end_to_end(n, L, G, tiles, causal):
    half = 128 // G
    per = half * tiles
    at = 0
    for t in range(-(-n // per)):
        assert _begin(n, L, per, t, causal) == at
        at += _cost(n, L, per, half, t, causal)


def test_the_constants_are_the_kernels():
    import os
    import re
    text = open(os.path.join(build.CSRC, "pkv_prefill.h")).read()
    got = {k: eval(v) for k, v in re.findall(r"(kPrefill(?:Key|Item|Token)Cost1?) = ([0-9* ]+)[,;]", text)}
    assert got == dict(kPrefillKeyCost=KEY, kPrefillItemCost=ITEM, kPrefillTokenCost=TOKEN,
                       kPrefillKeyCost1=KEY1, kPrefillItemCost1=ITEM1)
