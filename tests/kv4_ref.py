"""Plain references of the rotation, the 4-bit cache format and the attention
over it, in numpy, from the definitions in include/pkv.h.  ``quantise`` and
``rotate`` follow the FP32 arithmetic that the header fixes step by step (every
step an IEEE operation, so the library must give the same bytes); everything
else is in 64 bits."""
from __future__ import annotations

import numpy as np
import torch

F32 = np.float32


def rotate(x: np.ndarray, cos_sin: np.ndarray, positions: np.ndarray, interleaved: bool,
           f=F32) -> np.ndarray:
    """x [T, H, D] rotated in the arithmetic of ``f`` (float32: each product
    and sum rounded on its own)."""
    y = x.astype(f).copy()
    R = cos_sin.shape[1]
    c = cos_sin[positions, : R // 2].astype(f)[:, None]
    s = cos_sin[positions, R // 2:].astype(f)[:, None]
    a, b = ((slice(0, R, 2), slice(1, R, 2)) if interleaved
            else (slice(0, R // 2), slice(R // 2, R)))
    p, q = x[..., a].astype(f), x[..., b].astype(f)
    y[..., a] = p * c - q * s
    y[..., b] = q * c + p * s
    return y


def quantise(x: np.ndarray):
    """Rows [..., D] float32 -> (codes [..., D/32, 32], s, z float16 [..., D/32])."""
    g = x.astype(F32).reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    with np.errstate(all="ignore"):
        bad = ~np.isfinite(g).all(-1)
        lo, hi = g.min(-1), g.max(-1)
        want = np.maximum(np.maximum((hi - lo) / F32(15),
                                     np.maximum(np.abs(lo), np.abs(hi)) * F32(2.0 ** -10)),
                          F32(2.0 ** -24))
        h = want.astype(np.float16)
        h = np.where(h.astype(F32) < want, np.nextafter(h, np.float16(np.inf)), h)
        h = np.minimum(h, np.float16(65504))
        s = h.astype(F32)
        z = np.clip(lo / s, F32(-65504), F32(65504)).astype(np.float16)
        n = np.clip(np.rint(g / s[..., None] - z.astype(F32)[..., None]), 0, 15)
    nan = np.float16(np.nan)
    n = np.where(bad[..., None], 0, n).astype(np.uint8)
    return n, np.where(bad, nan, h), np.where(bad, nan, z)


def row_offsets(bs: int, D: int, values: bool) -> np.ndarray:
    """[bs, 5D/8]: tile byte of every byte of a row kept as codes (channel
    order), then (s, z) of each group."""
    G = D // 32
    out = np.zeros((bs, D * 5 // 8), np.int64)
    for r in range(bs):
        for g in range(G):
            at = r * (D // 2) + 16 * (g ^ ((r * G // 8) % G))
            out[r, 16 * g:16 * g + 16] = at + np.arange(16)
            if values:
                p = bs * D // 2 + 8 * ((r // 2) * G + g) + 2 * (r % 2)
                q = p + 4
            else:
                p = bs * D // 2 + 4 * (r * G + g)
                q = p + 2
            out[r, D // 2 + 4 * g:D // 2 + 4 * g + 4] = [p, p + 1, q, q + 1]
    return out


def row_bytes(x: np.ndarray) -> np.ndarray:
    """Rows [..., D] float32 -> their bytes [..., 5D/8] in row order."""
    n, s, z = quantise(x)
    n = n.reshape(*x.shape)
    par = np.ascontiguousarray(np.stack([s, z], -1)).view(np.uint8).reshape(*x.shape[:-1], x.shape[-1] // 8)
    return np.concatenate([n[..., 0::2] | (n[..., 1::2] << 4), par], -1)


def store(cache: np.ndarray, x: np.ndarray, slots: np.ndarray, values: bool) -> None:
    """Write rows x [T, Hkv, D] float32 at their slots of cache [NB, Hkv, bs, 5D/8]."""
    NB, Hkv, bs, W = cache.shape
    off, rows = row_offsets(bs, W * 8 // 5, values), row_bytes(x)
    tiles = cache.reshape(NB, Hkv, bs * W)
    for t, s in enumerate(slots):
        if 0 <= s < NB * bs:
            tiles[s // bs][:, off[s % bs]] = rows[t]


def load(cache: np.ndarray, slots: np.ndarray, values: bool) -> np.ndarray:
    """The values [T, Hkv, D] in 64 bits at the slots."""
    NB, Hkv, bs, W = cache.shape
    D = W * 8 // 5
    off = row_offsets(bs, D, values)
    slots = np.asarray(slots, np.int64)
    tiles = cache.reshape(NB, Hkv, bs * W)
    rows = np.take_along_axis(tiles[slots // bs], off[slots % bs][:, None].repeat(Hkv, 1), -1)
    par = np.ascontiguousarray(rows[..., D // 2:]).view(np.float16).astype(np.float64)
    par = par.reshape(len(slots), Hkv, D // 32, 1, 2)
    n = np.stack([rows[..., :D // 2] & 15, rows[..., :D // 2] >> 4], -1).reshape(
        len(slots), Hkv, D // 32, 32).astype(np.float64)
    with np.errstate(all="ignore"):
        return (par[..., 0] * (n + par[..., 1])).reshape(len(slots), Hkv, D)


def to_np(t: torch.Tensor) -> np.ndarray:
    return t.detach().float().cpu().numpy()


def attention(q: np.ndarray, k_cache: np.ndarray, v_cache: np.ndarray, tables: np.ndarray,
              lens: np.ndarray, scale: float):
    """softmax(scale q . k) . v in 64 bits over the 4-bit caches; also what the
    error bound needs: per out element the weighted magnitude sum w |v| and the
    error of weights held in binary16's subnormals, per row the error of a logit
    (see attention_bound)."""
    B, Hq, D = q.shape
    Hkv, bs = k_cache.shape[1:3]
    G = Hq // Hkv
    out, mag, low = np.zeros((B, Hq, D)), np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    smag = np.zeros((B, Hq))
    for i, L in enumerate(lens):
        if L == 0:
            continue
        t = np.arange(L)
        slots = tables[i, t // bs].astype(np.int64) * bs + t % bs
        k, v = load(k_cache, slots, False), load(v_cache, slots, True)
        par = _magnitudes(k_cache, slots)
        top = _params(v_cache, slots, True)[..., 0].max((0, 2))     # largest value scale, per kv head
        for h in range(Hq):
            qh, g = q[i, h].astype(np.float64), h // G
            a = scale * (k[:, g] @ qh)
            w = np.exp(a - a.max())
            w /= w.sum()
            out[i, h], mag[i, h] = w @ v[:, g], w @ np.abs(v[:, g])
            E = max(0.0, np.floor(np.log2(top[g])))
            low[i, h] = w.max() * 2.0 ** (E - 37) * np.abs(v[:, g]).sum(0)
            # in units of the largest step count: D / 8 + 8 FP32 roundings of the
            # largest partial sum, and what q loses in binary16's subnormals
            steps, rest = (D / 8 + 8) * 2.0 ** -24, 2.0 ** -35 * np.abs(qh).max()
            smag[i, h] = abs(scale) * (steps * (par[:, g] @ np.abs(qh)).max()
                                       + rest * np.abs(k[:, g]).sum(-1).max())
    return out, mag, low, smag


def _params(cache, slots, values):
    """(s, z) of the rows at the slots, [T, Hkv, D/32, 2] in 64 bits."""
    NB, Hkv, bs, W = cache.shape
    D = W * 8 // 5
    off = row_offsets(bs, D, values)[:, D // 2:]
    tiles = cache.reshape(NB, Hkv, bs * W)
    rows = np.take_along_axis(tiles[slots // bs], off[slots % bs][:, None].repeat(Hkv, 1), -1)
    return np.ascontiguousarray(rows).view(np.float16).astype(np.float64).reshape(len(slots), Hkv, D // 32, 2)


def _magnitudes(k_cache, slots):
    """s (15 + |z|) of every channel: no partial sum of a key's products is larger."""
    par = _params(k_cache, slots, False)
    return (par[..., 0] * (15 + np.abs(par[..., 1])))[..., None].repeat(32, -1).reshape(*par.shape[:2], -1)


def attention_bound(out, mag, low, smag, eps: float) -> np.ndarray:
    """How far a correct result may be off, element by element:
     - the store: half a step, eps / 2 of the value (and half the smallest
       subnormal binary16, 2^-25);
     - each weight: rounded to binary16 and again after its scale, 2^-11 each
       at most, exp2 to 2^-22, the sums in FP32 (at most 2^-24 a term, pairwise
       within a warp: 2^-14 covers 2^10 terms in a row);
     - weights below binary16's smallest normal number are off by up to half
       its smallest step, 2^-25, where the largest weight is at least 2^(12-E)
       (E: the exponent of the largest value scale, at least 0): 2^(E-37) of
       the largest weight for each token, times its |v|;
     - each logit: FP32 products and sums of at most D / 8 + 8 steps, 2^-24 of
       the largest partial sum each, and the queries' rounding (half of
       binary16's smallest step, 2^-25, times 16, for a row of at least 2^14:
       2^-35 of the row's largest element) (smag; in the exponent, so it counts relative to
       the weight), once in the weight and once in the normaliser."""
    logits = 2 * smag[..., None]
    weights = 2 * 2.0 ** -11 + 2.0 ** -22 + 2.0 ** -14
    return eps / 2 * np.abs(out) + 2.0 ** -25 + (weights + logits) * mag + low
