"""Plain 64-bit forms of the attention operators, from their formulas
(include/attn_b200.h), and the helpers of their tests.  Test code only."""
import math

import torch

E4M3_MAX = 448.0


def prepared(qkv, hq, hkv, dim, qw, kw, eps, inv_freq, rot, layout, rope_scale, positions):
    """(q, k, v) [T, heads, dim] in 64 bits and, for each of q and k, the size
    (|a| + |b|) rope_scale a rotation worked with, for tolerances."""
    x = qkv.double().view(qkv.shape[0], hq + 2 * hkv, dim)
    out = []
    for rows, w in ((x[:, :hq], qw), (x[:, hq:hq + hkv], kw)):
        if w is not None:
            rows = rows / torch.sqrt((rows ** 2).mean(-1, keepdim=True) + eps) * w.double()
        y, size = rows.clone(), rows.abs()
        if rot:
            t = positions.double()[:, None, None] * inv_freq.double()
            c, s = torch.cos(t) * rope_scale, torch.sin(t) * rope_scale
            ia = torch.arange(rot // 2) if layout == 0 else torch.arange(0, rot, 2)
            ib = ia + (rot // 2 if layout == 0 else 1)
            a, b = rows[..., ia], rows[..., ib]
            y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
            size[..., ia] = size[..., ib] = (a.abs() + b.abs()) * abs(rope_scale)
        out.append((y, size))
    return out[0], out[1], x[:, hq + hkv:]


def attend(q, k, v, scale, limit):
    """One sequence: q [n, hq, d], k and v [m, hkv, d] in any type; query i
    sees keys 0 .. limit[i] - 1.  (o [n, hq, d], lse [n, hq], A = sum p |v|,
    the largest scaled sum of |q k| of each row), in 64 bits."""
    n, hq, d = q.shape
    g = hq // k.shape[1]
    q, k, v = q.double(), k.double().repeat_interleave(g, 1), v.double().repeat_interleave(g, 1)
    x = torch.einsum("ihd,jhd->hij", q, k) * scale
    big = (torch.einsum("ihd,jhd->hij", q.abs(), k.abs()) * abs(scale))
    hidden = torch.arange(k.shape[0])[None, :] >= torch.as_tensor(limit)[:, None]
    x = x.masked_fill(hidden[None], -math.inf)
    big = big.masked_fill(hidden[None], 0.0)
    lse = torch.logsumexp(x, -1) if k.shape[0] else torch.full((hq, n), -math.inf, dtype=torch.float64)
    p = torch.where(torch.isinf(lse)[..., None], torch.zeros_like(x), torch.exp(x - lse[..., None]))
    o = torch.einsum("hij,jhd->ihd", p, v)
    A = torch.einsum("hij,jhd->ihd", p, v.abs())
    return o, lse.T, A, (big.amax(-1) if k.shape[0] else torch.zeros_like(lse)).T


def check_attention(out, lse, ref):
    """Tolerances.  The kernels hold scores, maxima, sums and outputs in 32
    bits and round twice to bf16 (half a step: 2^-8 of the value): the
    probabilities before the second product, which moves o by at most 2^-8 A,
    and o itself, by 2^-8 |o|.  Scores: d / 16 <= 16 additions in the tensor
    core, each off by at most 2^-23 of the sum of magnitudes, 2^-19 big at
    most with the scale; a score's error e changes a probability by e, so o by
    2 e A.  exp2 and the sums of up to 2^17 terms kept in 32 bits: 2^-12 A."""
    o, z, A, big = ref
    assert torch.isfinite(out.double()).all()
    e = big * 2.0 ** -19 + 2.0 ** -21
    tol = 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2.0 ** -12 + 2 * e[..., None]) * A + 1e-30
    over = (out.double().cpu() - o).abs() - tol
    assert over.max() <= 0, "off by %.3e more than allowed" % over.max()
    if lse is not None:
        got = lse.double().cpu()
        assert torch.equal(torch.isinf(got), torch.isinf(z))
        fin = torch.isfinite(z)
        off = (got - z).abs()[fin] - (e + 2.0 ** -12 + 2.0 ** -22 * z.abs())[fin]
        assert off.numel() == 0 or off.max() <= 0, "lse off by %.3e more than allowed" % off.max()


def quantised(x):
    """(codes as float8_e4m3fn, fp32 scales) of fp32 rows along the last dimension."""
    top = x.abs().amax(-1)
    s = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
    return (x / s[..., None]).to(torch.float8_e4m3fn), s


def make_cache(gen, pages, hkv, page, dim, e4m3):
    """Random caches on the CPU: (k, v, k_scale, v_scale), scales None in 16 bits."""
    k, v = (torch.randn(pages, hkv, page, dim, generator=gen) for _ in range(2))
    if not e4m3:
        return k.bfloat16(), v.bfloat16(), None, None
    k, ks = quantised(k)
    v, vs = quantised(v * (0.1 + torch.rand(pages, hkv, page, 1, generator=gen) * 4))
    return k, v, ks, vs


def rows_of(cache, scale, table_row, n):
    """[n, hkv, dim] in 64 bits: the first n rows of a sequence."""
    page = cache.shape[2]
    ids = table_row[:(n + page - 1) // page].long()
    x = cache.float()[ids].double()
    if scale is not None:
        x = x * scale[ids].double()[..., None]
    return x.transpose(1, 2).reshape(-1, cache.shape[1], cache.shape[3])[:n]


def make_table(gen, lens, page, spare=2):
    """(page table [B, width] int32 in shuffled order, number of pages)."""
    need = [(n + page - 1) // page for n in lens]
    total = sum(need) + spare
    order = torch.randperm(total, generator=gen).int()
    table = torch.zeros(len(lens), max(1, max(need)), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def starts(lens):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32)
