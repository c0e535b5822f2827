"""Plain 64-bit attention of packed sequences, and how far 16-bit kernels may be off.

The bound, term by term.  With u half a step of the output's type (2^-11
binary16, 2^-8 bfloat16), w the softmax weights and A = sum w |v|:
  * the store rounds the result once:                        u |out|
  * a weight is rounded to 16 bits before its product:       u A
  * a logit is a sum of D products in FP32, added in D / 16 steps of which each
    may be off by two units in the last place of the largest partial sum, plus
    the rounding of its scaled difference from the maximum (logits of up to X):
    d = (D / 16 * 2^-22 + 2^-23) X with X = max_t scale sum |q k_t|, which moves
    a weight by a factor e^(+-d) and the sum of weights as well:  2 d A
    (e^d is not linear for large d, hence expm1)
  * 2^x of the hardware (2^-22), the FP32 sums of products, over L / 16 steps of
    two units each, and the division:                      2^-20 A + L 2^-26 A
  * a weight below binary16's normal range is off by up to 2^-25, where the
    largest is at least 2^-1 (at least 2^7 in fact):            L 2^-24 max|v|
"""
import torch

HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def attend(q, k, v, scale, causal=True):
    """(out, bound) [n, Hq, D] float64 of one sequence; q [n, Hq, D], k, v [L, Hkv, D]."""
    n, Hq, D = q.shape
    L, Hkv = k.shape[:2]
    u = HALF[q.dtype]
    out = torch.zeros((n, Hq, D), dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    if L == 0 or n == 0:
        return out, bound
    q, k, v = q.double(), k.double().repeat_interleave(Hq // Hkv, 1), v.double().repeat_interleave(Hq // Hkv, 1)
    a = torch.einsum("nhd,thd->hnt", q, k) * scale
    t = torch.arange(L, device=q.device)
    seen = (t <= L - n + torch.arange(n, device=q.device)[:, None]) if causal else torch.ones((n, L), dtype=torch.bool, device=q.device)
    a = a.masked_fill(~seen, float("-inf"))
    w = torch.softmax(a, -1).nan_to_num(0.0) if not a.isnan().any() else torch.softmax(a, -1)
    w = torch.where(seen, w, 0.0)
    w[:, ~seen.any(-1)] = 0
    out = torch.einsum("hnt,thd->nhd", w, torch.where(v.isfinite(), v, 0.0))
    A = torch.einsum("hnt,thd->nhd", w, torch.where(v.isfinite(), v.abs(), 0.0))
    X = torch.einsum("nhd,thd->hnt", q.abs(), torch.where(k.isfinite(), k.abs(), 0.0)) * abs(scale)
    d = (D / 16 * 2.0 ** -22 + 2.0 ** -23) * torch.where(seen, X, 0.0).amax(-1).T[..., None]
    bound = u * out.abs() + A * (u + torch.expm1(2 * d) + 2.0 ** -20 + L * 2.0 ** -26)
    bound = bound + L * 2.0 ** -24 * (u == 2.0 ** -11) * torch.where(v.isfinite(), v.abs(), 0.0).amax() + 2.0 ** -24
    # weights are positive: a value that is no number stays none in every row that sees it
    for i, h, c in (~v.isfinite()).nonzero().tolist():
        out[seen[:, i], h, c] += v[i, h, c]
    return out, bound


def packed(q, k, v, query_starts, key_starts, scale, causal=True):
    """attend() of every sequence, one after the other (lists of starts)."""
    parts = [attend(q[a:b], k[c:d], v[c:d], scale, causal)
             for a, b, c, d in zip(query_starts, query_starts[1:], key_starts, key_starts[1:])]
    return tuple(torch.cat(x) for x in zip(*parts))


def check(got, ref, bound):
    got = got.double()
    nan = ref.isnan()
    assert torch.equal(got.isnan(), nan), f"{int((got.isnan() != nan).sum())} of {nan.numel()} differ in being a number"
    inf = ref.isinf()
    assert torch.equal(got[inf], ref[inf])
    fine = ~(nan | inf)
    err = (got - ref).abs()[fine] - bound[fine]
    assert err.numel() == 0 or float(err.max()) <= 0, f"over the bound by {float(err.max()):.3e} ({int((err > 0).sum())} values)"


def starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def paged(k, v, lens, bs, g, fill=float("nan"), spare=2):
    """Caches [NB, Hkv, bs, D] and tables of packed k, v [S, Hkv, D]: blocks in a
    random order, everything that no token has written holds `fill`."""
    S, Hkv, D = k.shape
    nblk = [-(-n // bs) for n in lens]
    NB, MB = sum(nblk) + spare, max(max(nblk), 1)
    perm = torch.randperm(NB, generator=g)
    caches = [torch.full((NB, Hkv, bs, D), fill, dtype=k.dtype) for _ in range(2)]
    tables, at, row = torch.full((len(lens), MB), -1, dtype=torch.int32), 0, 0
    for i, n in enumerate(lens):
        blocks = perm[at:at + nblk[i]]
        tables[i, :nblk[i]] = blocks.int()
        t = torch.arange(n)
        for c, x in zip(caches, (k, v)):
            c[blocks[t // bs], :, t % bs] = x[row:row + n].cpu()
        at, row = at + nblk[i], row + n
    return caches[0], caches[1], tables
