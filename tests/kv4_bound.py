"""How far kv4_attn_decode may be off, element by element, for values of any
magnitude: every rounding that the kernel makes, with none of the bound's terms
larger than what the values themselves give (no absolute floor but the output
type's own)."""
from __future__ import annotations

import numpy as np

import kv4_ref as R


def attention_and_bound(b, eps: float, half_step: float):
    """Attention in 64 bits over the 4-bit caches of batch ``b``, and its bound.
    ``eps``: the output type's spacing relative to the value; ``half_step``: half of
    its smallest subnormal step.

    With w the softmax weights, v = s (n + z) the held values, W the sequence's
    largest weight and S the largest scale of the value's channel group among the
    tokens that share its stage (32 tokens; 31 to either side are counted):
     - the store: eps / 2 of the result, and ``half_step``;
     - each weight, rounded to binary16, and again after its scale: 2^-11 each; exp2
       2^-22; the sums in FP32, 2^-14 for 2^10 additions in a row, of the codes' and
       the zero points' parts, which may cancel: of sum w s (n + |z|);
     - the logits: as in kv4_ref.attention (FP32 sums and the queries' rounding), once
       in the weight and once in the normaliser;
     - weights below binary16's normal numbers: 2^-25 where the largest weight is
       at least 2^12: 2^-37 W for each token, times its |v|;
     - products of weight and scale below them: 2^-37 W for each token, times n + |z|,
       where the stage's largest scale S of the group is at least 2^-13; else the scales
       are multiplied by a power of two 2^k that brings S to at least 1/2, or k is at
       least 14: 2^(-37-k) W.  In all at most max(2^-24 S, 2^-51) W;
     - scales that this power of two makes subnormal (k negative, which S of at least 1
       gives): 2^-25 where S is at least 1/2: 2^-24 S w, times n + |z|;
       none of these three loses more than the whole term."""
    q, kc, vc, tables, lens, scale = (R.to_np(b["q"]), b["kc"], b["vc"], b["tables"], b["lens"], b["scale"])
    want, mag, _, smag = R.attention(q, kc, vc, tables, lens, scale)
    B, Hq, D = q.shape
    Hkv, bs = kc.shape[1:3]
    parts, low = np.zeros_like(want), np.zeros_like(want)
    for i, L in enumerate(lens):
        if L == 0:
            continue
        t = np.arange(L)
        slots = tables[i, t // bs].astype(np.int64) * bs + t % bs
        k, v = R.load(kc, slots, False), R.load(vc, slots, True)
        par = R._params(vc, slots, True)
        s, z = (np.repeat(par[..., j], 32, -1) for j in (0, 1))            # [L, Hkv, D]
        steps = np.abs(v / s - z) + np.abs(z)                              # n + |z|
        S = s.copy()
        for d in range(1, min(32, L)):
            S[d:] = np.maximum(S[d:], s[:-d])
            S[:-d] = np.maximum(S[:-d], s[d:])
        for h in range(Hq):
            g = h // (Hq // Hkv)
            a = scale * (k[:, g] @ q[i, h].astype(np.float64))
            w = np.exp(a - a.max())
            w /= w.sum()
            parts[i, h] = w @ (s[:, g] * steps[:, g])
            W, ws = w.max(), w[:, None] * s[:, g]
            low[i, h] = (np.minimum(w, 2.0 ** -37 * W)[:, None] * np.abs(v[:, g])
                         + np.minimum(ws, W * np.maximum(2.0 ** -24 * S[:, g], 2.0 ** -51)) * steps[:, g]
                         + np.minimum(ws, w[:, None] * (2.0 ** -24 * S[:, g] * (S[:, g] >= 1))) * steps[:, g]).sum(0)
    bound = (eps / 2 * np.abs(want) + half_step + (2 * 2.0 ** -11 + 2.0 ** -22 + 2 * smag[..., None]) * mag
             + 2.0 ** -14 * parts + low)
    return want, bound
