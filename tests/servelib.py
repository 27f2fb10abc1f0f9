"""Float64 references of the serving operators (paged cache, attention over it,
beam selection and reordering) and the bounds the tests hold the kernels to.

Bounds are worst cases counted per element, as in ``layerlib``.
"""
import math

import torch

from layerlib import HALF

INF = float("inf")


def make_tables(lens, page, gen, spare=3, width=None):
    """Page table [n, width] (pages in no order, -1 where there is none) and the number of pages."""
    need = [-(-max(x, 0) // page) for x in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=gen).to(torch.int32)
    table = torch.full((len(lens), max(width or 0, max(need, default=0), 1)), -1, dtype=torch.int32)
    at = 0
    for s, m in enumerate(need):
        table[s, :m] = order[at:at + m]
        at += m
    return table, pages


def places(cu, lens, total):
    """(sequence, place) of every token, None for a token of no sequence."""
    if cu is None:
        return [(s, x - 1) for s, x in enumerate(lens)]
    out = [None] * total
    for s in range(len(lens)):
        a = min(max(cu[s], 0), total)
        b = min(max(cu[s + 1], a), total)
        for t in range(a, b):
            if out[t] is None:
                out[t] = (s, lens[s] - (b - t))
    return out


def row_of(table, pages, page, s, p):
    """(page, row in it) of a place, or None."""
    if p < 0 or p // page >= table.shape[1]:
        return None
    g = int(table[s, p // page])
    return (g, p % page) if 0 <= g < pages else None


def turned(x, pos, freq, sections, interleaved):
    """Rotated rows [N, heads, d] and, for the bound, the same over absolute values."""
    y, size = x.double().clone(), x.double().abs()
    if freq is None:
        return y, size * 0
    axis = torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections))
    angle = (pos.double()[:, axis] * freq)[:, None]
    c, s = torch.cos(angle), torch.sin(angle)
    P = len(axis)
    a, b = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if interleaved else (slice(0, P), slice(P, 2 * P))
    u, w = x.double()[..., a], x.double()[..., b]
    y[..., a], y[..., b] = u * c - w * s, w * c + u * s
    size[..., a] = size[..., b] = u.abs() + w.abs()
    return y, size


def turn_bound(want, size, dtype):
    """Cosine, sine and angle: 2^-21 together; products and sums: 2^-22."""
    return HALF[dtype] * want.abs() + 2.0 ** -20 * size


def attention(q, k_cache, v_cache, table, lens, scale, window=0):
    """o, lse, and for the bound sum p |v| and the largest sum |q| |k| of a row."""
    n, H, d = q.shape
    pages, page, Hk, _ = k_cache.shape
    o = torch.zeros(n, H, d, dtype=torch.float64)
    size, lse, dots = torch.zeros_like(o), torch.full((n, H), -INF, dtype=torch.float64), torch.zeros(n, H)
    for s in range(n):
        L = min(max(int(lens[s]), 0), table.shape[1] * page)
        first = max(L - window, 0) if window else 0
        at = [r for r in (row_of(table, pages, page, s, p) for p in range(first, L)) if r is not None]
        if not at:
            continue
        g, r = torch.tensor(at).T
        for h in range(H):
            K, V = k_cache[g, r, h // (H // Hk)].double(), v_cache[g, r, h // (H // Hk)].double()
            x = K @ q[s, h].double() * scale
            p = torch.softmax(x, 0)
            o[s, h], size[s, h] = p @ V, p @ V.abs()
            lse[s, h] = torch.logsumexp(x, 0)
            dots[s, h] = (K.abs() @ q[s, h].double().abs()).max() * abs(scale)
    return o, lse, size, dots


def score_error(dots, d):
    """Of a score: float32 products and sums of d terms (the tensor cores may cut, 2^-23 each), the scale's and
    the exponent's roundings."""
    return (d + 8) * 2.0 ** -23 * dots.double()


def attn_bound(want, size, dots, d, L, dtype):
    """A score off by e changes every weight by e and their sum by as much: 2 e of sum p |v|. The weights are held
    to 2^-15 at least (the exponential's 2^-21, two bfloat16 parts' 2^-16), sums of L terms to 2^-23 each, and the
    output is rounded once."""
    return HALF[dtype] * want.abs() + (2 * score_error(dots, d)[..., None] + 2.0 ** -15 + (L + 256) * 2.0 ** -23) * size + 1e-30


def lse_bound(want, dots, d, L):
    return score_error(dots, d) + 2.0 ** -15 + (L + 256) * 2.0 ** -23 + 2.0 ** -22 * want.abs()


# of a selection's scores: exp to 2^-22, the logit's distance from the row's maximum (about log V where it counts) to
# 2^-24 of itself, sums of 16 terms in pairs: 2^-20 of the sum and thus of its log, and the result's rounding
def select_bound(want):
    return 2.0 ** -24 * want.abs() + 2.0 ** -20


def candidates(logits, scores, done=None, eos=0):
    """c(w, v) in 64 bits, [B, W, V]; without a value: -infinity."""
    x = logits.double()
    c = scores.double()[..., None] + torch.log_softmax(x, -1)
    if done is not None:
        ended = torch.full_like(c, -INF)
        ended[..., eos] = scores.double()
        c = torch.where(done.bool()[..., None], ended, c)
    return torch.where(torch.isfinite(c), c, torch.full_like(c, -INF))


def selection(c, K):
    """The K best of each request, ties in the order of w*V + v: scores, parent, token."""
    V = c.shape[-1]
    best, at = torch.sort(-c.flatten(1), dim=1, stable=True)
    at = at[:, :K]
    return -best[:, :K], (at // V).int(), (at % V).int()


def nearest(c, K):
    """The smallest distance of two neighbours among the K + 1 best that are not of the same beam."""
    V = c.shape[-1]
    best, at = torch.sort(-c.flatten(1), dim=1, stable=True)
    best, at = best[:, :K + 1], at[:, :K + 1] // V
    gap = best[:, 1:] - best[:, :-1]
    other = (at[:, 1:] != at[:, :-1]) & torch.isfinite(best[:, 1:])
    return float(gap[other].min()) if bool(other.any()) else INF


def moved(rows, parent, W):
    """Row w of each request becomes what row parent[w] was (list of rows, None: no row)."""
    new = list(rows)
    for i, p in enumerate(parent.flatten().tolist()):
        j = i // W * W + p
        if 0 <= p < W and rows[i] is not None and rows[j] is not None:
            new[i] = rows[j]
    return new
