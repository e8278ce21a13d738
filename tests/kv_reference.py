"""Head norms with rotation, the paged cache and attention over it in 64 bits on the CPU, from their
formulas, with bounds on the library's difference, for the tests."""
from __future__ import annotations

import torch

import s8_reference as s8

TYPES = s8.TYPES
U32 = s8.U32
TOP = {2: 32600.0, 3: 8355000.0}   # what the largest of a row becomes in two and three digits
TILE = {torch.int8: 64, torch.float16: 32, torch.bfloat16: 32, torch.float32: 16}


def half_step(v, dtype):
    """A rounding of v to the type: half a step of it, or of its subnormals."""
    info = torch.finfo(dtype)
    return v.abs() * (info.eps / 2) + float(info.smallest_normal) * info.eps / 2


def norm_rope(x, w, eps, pos, freq, pairs):
    """(value, bound) of T x H x D heads: the library computes in 64 bits (a few dozen roundings of
    the pair's size, taken as 1e-14), rounds to fp32 and from there to the type."""
    v = x.double()
    if w is not None:
        v = v / torch.sqrt((v ** 2).mean(-1, keepdim=True) + eps) * w.double()
    y, size = v.clone(), v.abs()
    if freq is not None and len(freq):
        R = 2 * len(freq)
        angle = pos.double()[:, None] * freq.double()[None, :]
        c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
        ia, ib = (slice(0, R, 2), slice(1, R, 2)) if pairs else (slice(0, R // 2), slice(R // 2, R))
        a, b = v[..., ia], v[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        size = size.clone()
        size[..., ia] = size[..., ib] = a.abs() + b.abs()
    exact = 1e-14 * size
    return y, exact + U32 * (y.abs() + exact) + half_step(y.abs() * (1 + U32) + exact, x.dtype), exact


def codes_near(v, exact, code, scale):
    """Whether codes and scales (.., D and ..) are those of a row of fp32 values within ``exact`` of v: the scale
    within that and its two roundings, each code half a step from its value and what that moves."""
    top = v.abs().amax(-1)
    ds = exact.amax(-1) / 127 + 2.1 * U32 * top / 127
    ok = ((scale.double() - top / 127).abs() <= ds).all()
    err = (code.double() * scale.double()[..., None] - v).abs()
    return bool(ok) and bool((err <= scale.double()[..., None] * (0.5 + 1e-9) + exact + U32 * v.abs()).all())


def cache_rows(cache_k, scale, table_row, n, page_size, pages):
    """(rows Hk x n x D in 64 bits, which of the n tokens have a page)."""
    t = torch.arange(n)
    entry = table_row.long()[t // page_size] if n else t
    has = (entry >= 0) & (entry < pages)
    page, at = torch.where(has, entry, 0), t % page_size
    rows = cache_k[page, :, at].double()
    if scale is not None:
        rows = rows * scale[page, :, at].double()[..., None]
    return rows.permute(1, 0, 2), has


def attention(q, k, v, ks, vs, table, lengths, window, scale):
    """(o, lse, bound on o, bound on lse), all 64-bit, for q B x Hq x D.

    The bound counts, with A the largest sum of |q k| times the scale in a head's scores: the roundings of the
    scores and of their distance to the maximum, U32 of A each; with codes, half a step of the query's
    fixed-point row and half a rounding of its quotient; the exponential's own error, 2^-23, with every tile's
    rescaling; the weights' rounding (two numbers of the type, or half a step of a tile's largest); sums of n
    values in any order; and the output's rounding."""
    B, Hq, D = q.shape
    pages, Hk, ps, _ = k.shape
    G = Hq // Hk
    dtype, kind = q.dtype, k.dtype
    o = torch.zeros(B, Hq, D, dtype=torch.float64)
    lse = torch.full((B, Hq), float("-inf"), dtype=torch.float64)
    bo, bl = torch.zeros_like(o), torch.zeros_like(lse)
    digits = 3 if dtype == torch.float32 else 2
    for b in range(B):
        n = max(0, min(int(lengths[b]), table.shape[1] * ps))
        lo = max(0, n - window) if window else 0
        K, has = cache_rows(k, ks, table[b], n, ps, pages)
        V, _ = cache_rows(v, vs, table[b], n, ps, pages)
        t = torch.arange(n)
        t = t[has & (t >= lo)]
        if not len(t):
            continue
        K, V = K[:, t], V[:, t]
        qq = q[b].double().view(Hk, G, D)
        s = scale * (qq @ K.transpose(1, 2))
        A = abs(scale) * (qq.abs() @ K.abs().transpose(1, 2))
        a = A.amax(-1, keepdim=True)
        l = torch.logsumexp(s, -1, keepdim=True)
        w = torch.exp(s - l)
        out = w @ V
        tiles = t // TILE[kind]
        if kind == torch.int8:
            lsb = qq.abs().amax(-1) / TOP[3] * 1.01   # per value of q
            es = abs(scale) * lsb[..., None] * K.abs().sum(-1)[:, None, :].amax(-1, keepdim=True) + 16 * U32 * a
        else:
            es = (2 * D + 16) * U32 * a
        split = {torch.bfloat16: 2.0 ** -16, torch.float16: 2.0 ** -21}.get(kind, 0.0)
        delta = torch.expm1(es) + (len(tiles.unique()) + 12) * 2.0 ** -23 + split
        err = (2.02 * delta + 2 * (len(t) + 8) * U32) * (w @ V.abs())
        if kind == torch.float16:
            err = err + 2.0 ** -28 * V.abs().sum(1, keepdim=True)
        if kind == torch.int8:
            row = V.abs().amax(-1)[:, None, :] / 127         # a code's step, or less
            size = V.abs() / row[:, 0, :, None].clamp_min(1e-300)
            for m in torch.split(torch.arange(len(t)), tiles.unique_consecutive(return_counts=True)[1].tolist()):
                m = slice(int(m[0]), int(m[-1]) + 1)
                step = ((w[..., m] * row[..., m]).amax(-1, keepdim=True) * 1.02 + 2.0 ** -100) / TOP[digits]
                err = err + step * (1.01 if digits == 3 else 0.52) * size[:, m].sum(1)[:, None, :]
        o[b], lse[b] = out.reshape(Hq, D), l.reshape(Hq)
        bo[b] = (err + half_step(out.abs() + err, dtype)).reshape(Hq, D)
        bl[b] = (delta[..., 0] + (len(t) + 8) * U32 + 2.0 ** -21 + 8 * U32 * (l[..., 0].abs() + a[..., 0])).reshape(Hq)
    return o, lse, bo, bl
