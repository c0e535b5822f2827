"""What is measured of the prompt side of the paged cache.

Three operators that bring a prompt into the cache and attend over it:
attention of a chunk of new tokens over the paged cache (``chunk``), attention
over whole prompts packed one after the other (``prompt``), and the rotation
append with positions of several axes (``axes``).  ``own`` chooses between the
plain forms below (elementary torch operations in 32 bits) and the package's
calls; ``exact`` holds the definitions once more in 64 bits.

Sequence i has the query rows starts[i] .. starts[i + 1].  Its j-th of n rows
stands at position L - n + j of its L keys and, where the mask is causal, sees
the keys up to that position; a row that sees no key is zero.
"""
import math
import random

import numpy as np
import torch

own = False

_DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _dev():
    return "cuda" if torch.cuda.is_available() else "cpu"


# ---------------------------------------------------------------- the cases
def _chunk(name, B, hq, hkv, D, bs, dt, new, ctx, lens_seed=1, fused=False):
    """``new``, ``ctx``: bounds of the new tokens and of the tokens cached before them."""
    return dict(name=name, op="chunk", B=B, hq=hq, hkv=hkv, D=D, bs=bs, dtype=dt, new_lo=new[0], new_hi=new[1],
                ctx_lo=ctx[0], ctx_hi=ctx[1], lens_seed=lens_seed, fused=fused, mixed=0)


def _prompt(name, B, hq, hkv, D, dt, new, ctx=(0, 0), lens_seed=1, fused=False, causal=True):
    return dict(name=name, op="prompt", B=B, hq=hq, hkv=hkv, D=D, dtype=dt, new_lo=new[0], new_hi=new[1],
                ctx_lo=ctx[0], ctx_hi=ctx[1], lens_seed=lens_seed, fused=fused, causal=causal)


def _axes(name, T, hq, hkv, D, bs, dt, sections, inter=False, fused=False, base=0, pad=0):
    """T tokens, text and images in turn from position ``base`` on; ``pad``: padding tokens (slot -1)."""
    return dict(name=name, op="axes", T=T, hq=hq, hkv=hkv, D=D, bs=bs, dtype=dt, s0=sections[0], s1=sections[1],
                s2=sections[2], inter=inter, fused=fused, base=base, pad=pad)


def listed():
    return [
        # a few drafted tokens of four short chats on a small model: the smallest call, latency counts
        _chunk("chunk 4 x 1-5", 4, 8, 8, 64, 16, "fp16", (1, 5), (0, 195)),
        # eight drafted tokens verified against long documents: few rows, bound by the cache's bytes
        _chunk("chunk 4 x 8 after 32760", 4, 64, 8, 128, 32, "bf16", (8, 8), (32760, 32760)),
        # the fifth chunk of one long prompt
        _chunk("chunk 2048 after 8192", 1, 32, 8, 128, 16, "bf16", (2048, 2048), (8192, 8192), fused=True),
        # a scheduler's step: 124 sequences in decode and four prompts' chunks of up to 600 tokens
        dict(_chunk("chunk mixed 128", 128, 32, 8, 128, 16, "fp16", (1, 1), (15, 4095)), mixed=4),
        # wide heads, odd sizes
        _chunk("chunk 2 x 1001 after 3001", 2, 8, 4, 256, 16, "bf16", (1001, 1001), (3001, 3001)),
        # three one-line prompts on a small model
        _prompt("prompt 3 x 5-40", 3, 8, 8, 64, "fp16", (5, 40)),
        # one long prompt, straight from a fused projection
        _prompt("prompt 8192", 1, 32, 8, 128, "bf16", (8192, 8192), fused=True),
        # a batch of prompts at every length, one query head a key head
        _prompt("prompt 32 x 1-2048", 32, 32, 32, 128, "fp16", (1, 2048)),
        # a prompt's chunk with its prefix read back from a 4-bit cache before it
        _prompt("prompt 1999 after 1025", 1, 32, 32, 128, "fp16", (1999, 1999), (1025, 1025)),
        # a decode step of 256 chats about images
        _axes("axes 256 tokens", 256, 32, 8, 128, 16, "fp16", (16, 24, 24), base=30000, pad=16),
        # a prompt of pages and text straight from a fused projection
        _axes("axes 8192 tokens", 8192, 32, 8, 128, 16, "bf16", (16, 24, 24), fused=True),
        # a short clip on a small model, neighbouring channels paired
        _axes("axes 1999 tokens", 1999, 8, 8, 64, 16, "fp16", (8, 12, 12), inter=True, base=77),
    ]


_MOST_FLOPS = 4 * 32 * 128 * 8192 * 8193 // 2


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng, most):
    hkv = rng.choice([1, 2, 3, 4, 8, 8, 16, 32])
    G = rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 8, 12, 16, 32])
    while hkv * G > most:
        G = max(1, G // 2)
    return hkv * G, hkv


def draw(rng):
    op = rng.choice(["chunk", "chunk", "prompt", "prompt", "axes"])
    D, bs, dt = rng.choice([64, 128, 128, 256]), rng.choice([16, 32]), rng.choice(["fp16", "bf16"])
    hq, hkv = _heads(rng, 64)
    if op == "axes":
        T = _log_uniform(rng, 1, 8192)
        while T * (hq + 2 * hkv) * D > 8192 * 48 * 128:
            T = max(1, T // 2)
        half = rng.choice([D // 2, D // 2, D // 4, 24])
        a = rng.randrange(1, half - 1)
        b = rng.randrange(1, half - a)
        c = _axes("", T, hq, hkv, D, bs, dt, (a, b, half - a - b), rng.random() < 0.4, rng.random() < 0.5,
                  rng.choice([0, 0, 30000]), rng.randrange(T) if rng.random() < 0.3 else 0)
        del c["name"]
        return c
    B, hi, back = _log_uniform(rng, 1, 128), _log_uniform(rng, 1, 8192), _log_uniform(rng, 1, 32768)
    if rng.random() < 0.4:
        hi = _log_uniform(rng, 1, 16)
    if op == "prompt" and rng.random() < 0.6:
        back = 0

    def cost():
        return 4 * hq * D * B * hi * (back + hi / 2), 4 * B * (back + hi) * hkv * D
    while cost()[0] > _MOST_FLOPS or cost()[1] > 4 * 4 * 32768 * 8 * 128 or B * hi * hq * D > 1 << 27:
        r = rng.random()
        if B > 1 and r < 0.4:
            B = max(1, B // 2)
        elif back > 1 and r < 0.7:
            back = back * 2 // 3
        else:
            hi = max(1, hi * 2 // 3)
    new = (rng.choice([1, hi, max(1, hi // 8)]), hi)
    ctx = (rng.choice([0, back, back // 8]), back)
    if op == "chunk":
        c = _chunk("", B, hq, hkv, D, bs, dt, new, ctx, rng.randrange(1 << 20), rng.random() < 0.5)
    else:
        c = _prompt("", B, hq, hkv, D, dt, new, ctx, rng.randrange(1 << 20), rng.random() < 0.5, rng.random() < 0.8)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs
def _lens(c):
    """New tokens and keys in all of every sequence."""
    r = np.random.RandomState(c["lens_seed"])
    new = r.randint(c["new_lo"], c["new_hi"] + 1, c["B"]).astype(np.int64)
    ctx = r.randint(c["ctx_lo"], c["ctx_hi"] + 1, c["B"]).astype(np.int64)
    if c.get("mixed"):
        at = r.permutation(c["B"])[:c["mixed"]]
        new[at] = r.randint(200, 601, c["mixed"])
    return new, new + ctx


def _keys(shape, g, dev):
    """Keys as models have them: a few channels of every head are larger, some have an offset."""
    h, d = shape[-2:]
    k = torch.randn(shape, generator=g, device=dev)
    k *= 1 + 3 * (torch.rand((h, d), generator=g, device=dev) < 0.06)
    return k.add_(2 * (torch.rand((h, d), generator=g, device=dev) < 0.03))


def _positions(c, r):
    """[3, T]: text counts on in all three axes; an image stands at one time, its patches at their row and column."""
    T, pos, at, now = c["T"], np.zeros((3, c["T"]), np.int32), 0, c["base"]
    while at < T:
        n = min(T - at, int(r.randint(1, 200)))
        pos[:, at:at + n] = now + np.arange(n)
        at, now = at + n, now + n
        h, w = int(r.randint(2, 32)), int(r.randint(2, 32))
        n = min(T - at, h * w)
        i = np.arange(n)
        pos[:, at:at + n] = now + np.stack([0 * i, i // w, i % w])
        at, now = at + n, now + max(h, w)
    return pos


def _rotation_table(n, rot, dev):
    """Positions 0 .. n - 1, worked out in 64 bits: far angles need them."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    a = torch.arange(n, dtype=torch.float64, device=dev)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _starts(n, dev):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).to(dev)


def _projected(T, hq, hkv, D, dt, fused, g, dev):
    """q, k, v of T tokens: slices of one projection's rows where ``fused``."""
    x = torch.randn((T, hq + 2 * hkv, D), generator=g, device=dev)
    x[:, hq:hq + hkv] = _keys((T, hkv, D), g, dev)
    q, k, v = x.to(dt).split([hq, hkv, hkv], 1)
    return (q, k, v) if fused else (q.contiguous(), k.contiguous(), v.contiguous())


def prepare(case, seed):
    dev = _dev()
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 13)
    r = np.random.RandomState((int(seed) * 31 + 7) % (1 << 32))
    c, dt, D, hq, hkv = case, _DT[case["dtype"]], case["D"], case["hq"], case["hkv"]
    s = dict(case=c, dtype=dt, scale=float(np.float32(1 / math.sqrt(D))))
    if c["op"] == "axes":
        T, bs = c["T"], c["bs"]
        q, k, v = _projected(T, hq, hkv, D, dt, c["fused"], g, dev)
        nb = T * 9 // 8 // bs + 2
        blocks = torch.from_numpy(r.permutation(nb)).to(dev)
        t = torch.arange(T, device=dev)
        slots = (blocks[t // bs] * bs + t % bs).int()
        if c["pad"]:
            slots[-c["pad"]:] = -1
        pos = torch.from_numpy(_positions(c, r)).to(dev)
        table = _rotation_table(c["base"] + T + 64, 2 * (c["s0"] + c["s1"] + c["s2"]), dev)
        caches = [torch.randn((nb, hkv, bs, D), generator=g, device=dev).to(dt) for _ in range(2)]
        s.update(q=q, k=k, v=v, slots=slots, positions=pos, table=table, k_cache=caches[0], v_cache=caches[1],
                 sections=(c["s0"], c["s1"], c["s2"]))
        return s
    new, lens = _lens(c)
    s.update(new=new.tolist(), lens=lens.tolist(), starts=_starts(new, dev))
    if c["op"] == "prompt":
        if (new == lens).all():
            q, k, v = _projected(int(new.sum()), hq, hkv, D, dt, c["fused"], g, dev)
            s.update(q=q, k=k, v=v, key_starts=s["starts"])
        else:
            S = int(lens.sum())
            q = _projected(int(new.sum()), hq, hkv, D, dt, c["fused"], g, dev)[0]
            s.update(q=q, k=_keys((S, hkv, D), g, dev).to(dt), key_starts=_starts(lens, dev),
                     v=torch.randn((S, hkv, D), generator=g, device=dev).to(dt))
        return s
    bs = c["bs"]
    q = _projected(int(new.sum()), hq, hkv, D, dt, c["fused"], g, dev)[0]
    nblk = -(-lens // bs)
    nb = int(nblk.sum() * 9 // 8) + 2
    perm, tables, at = r.permutation(nb), np.full((c["B"], int(nblk.max())), -1, np.int32), 0
    for i, n in enumerate(nblk):
        tables[i, :n] = perm[at:at + n]
        at += n
    kc, vc = _keys((nb, bs, hkv, D), g, dev).to(dt), torch.randn((nb, bs, hkv, D), generator=g, device=dev).to(dt)
    kc, vc = kc.transpose(1, 2).contiguous(), vc.transpose(1, 2).contiguous()
    free = torch.from_numpy(perm[at:]).to(dev)
    kc[free], vc[free] = math.nan, math.nan         # blocks that no sequence holds have never been written
    s.update(q=q, k_cache=kc, v_cache=vc, tables=torch.from_numpy(tables).to(dev),
             context_lens=torch.from_numpy(lens.astype(np.int32)).to(dev), max_len=int(lens.max()))
    return s


# ---------------------------------------------------------------- plain forms
def _attend(q, k, v, scale, causal):
    """softmax(q k^T scale) v of one sequence in 32 bits; q [n, hq, D], k and v [L, hkv, D]."""
    n, hq, D = q.shape
    L, hkv = k.shape[:2]
    G = hq // hkv
    k, v = k.float().permute(1, 2, 0), v.float().transpose(0, 1)                   # [hkv, D, L], [hkv, L, D]
    key = torch.arange(L, device=q.device)
    out, step = torch.zeros_like(q), max(1, (1 << 29) // max(1, hq * L))
    for at in range(0, n if L else 0, step):
        rows = q[at:at + step].float().transpose(0, 1)                             # [hq, m, D]
        m = rows.shape[1]
        a = (rows.reshape(hkv, G * m, D) @ k).view(hkv, G, m, L) * scale
        if causal:
            seen = key <= L - n + at + torch.arange(m, device=q.device)[:, None]
            a = torch.where(seen, a, -math.inf)
        top = a.amax(-1, keepdim=True)
        p = (a - torch.where(top > -math.inf, top, 0.0)).exp()
        total = p.sum(-1, keepdim=True)
        o = (p.view(hkv, G * m, L) @ v).view(hkv, G, m, D) / torch.where(total > 0, total, 1.0)
        out[at:at + m] = o.reshape(hq, m, D).transpose(0, 1).to(q.dtype)
    return out


def _plain_attention(s):
    c, outs, at, key = s["case"], [], 0, 0
    for i, (n, L) in enumerate(zip(s["new"], s["lens"])):
        if c["op"] == "chunk":
            nblk = -(-L // c["bs"])
            blocks = s["tables"][i, :nblk].long()
            k, v = (s[x][blocks].transpose(1, 2).flatten(0, 1)[:L] for x in ("k_cache", "v_cache"))
        else:
            k, v = s["k"][key:key + L], s["v"][key:key + L]
        outs.append(_attend(s["q"][at:at + n], k, v, s["scale"], c.get("causal", True)))
        at, key = at + n, key + L
    return torch.cat(outs)


def _rotate(x, cs, inter):
    """Rotated rows in 32 bits; channels past the table's width stay."""
    x, R = x.float(), cs.shape[-1]
    c, s = cs[:, None, :R // 2], cs[:, None, R // 2:]
    if inter:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([y, x[..., R:]], -1)


def _plain_axes(s):
    c, half = s["case"], sum(s["sections"])
    axis = torch.arange(3, device=s["q"].device).repeat_interleave(torch.tensor(s["sections"], device=s["q"].device))
    pos = s["positions"].long()[axis].T                                            # [T, half]: each pair's position
    pair = torch.arange(half, device=pos.device)
    cs = torch.cat([s["table"][pos, pair], s["table"][pos, half + pair]], 1)
    q, k = (_rotate(s[x], cs, c["inter"]).to(s["dtype"]) for x in ("q", "k"))
    keep = (s["slots"] >= 0).nonzero()[:, 0]
    slots = s["slots"][keep].long()
    s["k_cache"][slots // c["bs"], :, slots % c["bs"]] = k[keep]
    s["v_cache"][slots // c["bs"], :, slots % c["bs"]] = s["v"][keep]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def run(state):
    s, c = state, state["case"]
    if own:
        import paged_kv_cache_268_gb300 as pkv
        if c["op"] == "chunk":
            return pkv.paged_attn_chunk(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["context_lens"],
                                        s["starts"], s["scale"], max_context_len=s["max_len"])
        if c["op"] == "prompt":
            return pkv.prompt_attn(s["q"], s["k"], s["v"], s["starts"], s["scale"], key_starts=s["key_starts"],
                                   causal=c["causal"])
        q = pkv.rope_append(s["q"], s["k"], s["v"], s["positions"], s["table"], s["slots"], s["k_cache"],
                            s["v_cache"], interleaved=c["inter"], sections=s["sections"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return _plain_axes(s) if c["op"] == "axes" else _plain_attention(s)


# ---------------------------------------------------------------- work
def work(case):
    c = case
    hq, hkv = c["hq"] * c["D"], c["hkv"] * c["D"]
    if c["op"] == "axes":
        T, live, half = c["T"], c["T"] - c["pad"], c["s0"] + c["s1"] + c["s2"]
        return {"bytes": 4 * T * hq + 8 * live * hkv + T * (8 * half + 16),
                "flops": 6 * T * (c["hq"] + c["hkv"]) * half}
    new, lens = _lens(c)
    pairs = new * lens
    if c.get("causal", True):
        pairs = pairs - new * (new - 1) // 2
    b = 4 * int(new.sum()) * hq + 4 * int(lens.sum()) * hkv + 8 * c["B"]
    if c["op"] == "chunk":
        b += 4 * int((-(-lens // c["bs"])).sum())
    return {"bytes": b, "flops": 4 * hq * int(pairs.sum())}


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_heads(q, k, v, scale, causal):
    """One sequence, head by head: q [n, hq, D], k and v [L, hkv, D] in 64 bits."""
    (n, hq, D), (L, hkv) = q.shape, k.shape[:2]
    out = torch.zeros((n, hq, D), dtype=torch.float64, device=q.device)
    if L == 0:
        return out
    at = torch.arange(L - n, L, device=q.device)
    hidden = torch.arange(L, device=q.device)[None] > at[:, None] if causal else None
    for h in range(hq):
        a = torch.mm(q[:, h], k[:, h * hkv // hq].T).mul_(scale)
        if causal:
            a.masked_fill_(hidden, -math.inf)
        w = torch.softmax(a, -1)
        if causal:
            w[at < 0] = 0
        out[:, h] = torch.mm(w, v[:, h * hkv // hq])
    return out


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] != "axes":
        new, lens = _lens(c)
        q, outs = s["q"].double(), []
        for i in range(c["B"]):
            n0, L = int(new[:i].sum()), int(lens[i])
            if c["op"] == "chunk":
                t = torch.arange(L, device=q.device)
                block, row = s["tables"][i].long()[t // c["bs"]], t % c["bs"]
                k, v = (s[x][block, :, row].double() for x in ("k_cache", "v_cache"))
            else:
                k0 = int(lens[:i].sum())
                k, v = (s[x].narrow(0, k0, L).double() for x in ("k", "v"))
            outs.append(_exact_heads(q[n0:n0 + int(new[i])], k, v, s["scale"], c.get("causal", True)))
        return torch.cat(outs)
    table, pos = s["table"].double().cpu().numpy(), s["positions"].cpu().numpy()
    half = sum(s["sections"])
    w = np.zeros((c["T"], half), np.complex128)
    for i in range(half):
        axis = 0 if i < c["s0"] else (1 if i < c["s0"] + c["s1"] else 2)
        w[:, i] = table[pos[axis], i] + 1j * table[pos[axis], half + i]
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if c["inter"] else (slice(0, half), slice(half, 2 * half))
    got = {}
    for name in ("q", "k"):
        x = s[name].double().cpu().numpy().copy()
        y = (x[..., a] + 1j * x[..., b]) * w[:, None]
        x[..., a], x[..., b] = y.real, y.imag
        got[name] = x
    live = np.flatnonzero(s["slots"].cpu().numpy() >= 0)
    at = s["slots"].cpu().numpy()[live]
    out = {"q": torch.from_numpy(got["q"])}
    for name, x in (("k_cache", got["k"]), ("v_cache", s["v"].double().cpu().numpy())):
        cache = s[name].double().cpu().numpy()
        cache[at // c["bs"], :, at % c["bs"]] = x[live]
        out[name] = torch.from_numpy(cache)
    return out


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(i)) for i in range(6)]:
        print(c, work(c))
