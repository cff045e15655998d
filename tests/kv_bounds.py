"""Attention over the quantised key/value cache in 64 bits, with an error bound that counts every token by its own weight
and value scale, and the same sums with operands of 16 bits (what the bound has to tell apart)."""
import numpy as np
import torch

from kv_util import U32, half_step, least

# The operands of a row's sums lie at least 2^(6 - SPREAD) high where its largest p * vscale does, and fp16 rounds what is
# next to zero by 2^-25 at most.
SPREAD = {torch.float16: 8, torch.bfloat16: 14}


def terms(cache, batch, q, scale, window):
    """For every key/value head and row: (row, its query heads, scores, what was summed for them, tokens' value codes,
    scales and what is added to every dim of a token)."""
    D, group, mid = cache.D, q.shape[1] // cache.heads, 0 if cache.fmt == "i8" else 8
    for b, (n, length) in enumerate(zip(batch.n, batch.lens)):
        if length <= 0:
            continue
        pos = np.arange(length)
        page, t = batch.where(cache, b, pos)
        have = page >= 0
        page = np.maximum(page, 0)
        for h in range(cache.heads):
            held = []
            for i in range(2):
                x, low = cache.get(i, page, t, h)
                s = cache.meta(i, 0)[page, h, t].astype(np.float64)[:, None]
                held += [x - mid * s, (low + mid * s)[:, 0] if mid else 0 * s[:, 0], s[:, 0]]
            for i in range(n):
                row, at = int(batch.offsets[b]) + i, length - n + i
                seen = have & (pos <= at) & (pos > at - window if window else True)
                if seen.any():
                    heads = slice(h * group, (h + 1) * group)
                    yield (row, heads, q[row, heads]) + tuple(x[seen] for x in held)


def bounded(cache, batch, q, scale, window, dtype):
    """y and its error bound [rows][Hq][D] in float64; q: float64 [rows][Hq][D] as the type holds it.

    A score is scale * (sum q * kx + kmid * sum q), kx the code (4 bits: less 8) times its scale and kmid the minimum + 8
    scales (8 bits: none): D roundings of each sum's magnitudes and 8 of what is done with it; an exponent of base 2, less
    the row's, is rounded twice (of what the minima give and of itself).  bf16 queries go to fp16 after a power of two
    that keeps what is above 2^-31 of the row's largest.  exp2, the product with the value scale and the power of two: 2^-22.
    The operand p * vscale of the value's code: half a step of fp16, or 2^-22 where it is taken in two parts; next to zero
    2^-25, where the row's largest operand is 2^(6 - SPREAD) or more.  The sums over m tokens: m roundings; the joining of
    parts 2^-20; the second order of all of this 1 %."""
    rows, Hq, D = q.shape
    y, bound = np.zeros((batch.rows, Hq, D)), np.zeros((batch.rows, Hq, D))
    cast = 2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -22
    for row, heads, qq, kx, kmid, _, vx, vmid, vs in terms(cache, batch, q, scale, window):
        m, qa = len(kmid), np.abs(qq)
        low = kmid * qq.sum(1)[:, None] * scale
        s = qq @ kx.T * scale + low
        size = (qa @ np.abs(kx).T + np.abs(kmid) * qa.sum(1)[:, None]) * scale
        top = s.max(1, keepdims=True)
        p = np.exp(s - top)
        p /= p.sum(1, keepdims=True)
        ds = (D + 8) * U32 * size + 2 * U32 * (np.abs(s - top) + np.abs(top) + np.abs(low) + 2)
        if dtype == torch.bfloat16:
            ds += 2.0 ** -31 * D * qa.max(1)[:, None] * np.abs(kx).max(1) * scale
        eps = np.expm1(ds) + 2.0 ** -22
        out = p @ (vx + vmid[:, None])
        ax, amid = np.abs(vx), np.abs(vmid)[:, None]
        e = (p * (eps + cast + m * U32 + 2.0 ** -20)) @ ax + (p * (eps + m * U32 + 2.0 ** -20)) @ amid
        e += np.abs(out) * ((p * eps).sum(1, keepdims=True) + m * U32)
        codes = np.divide(ax, np.abs(vs)[:, None], out=np.zeros_like(ax), where=vs[:, None] != 0).sum(0)
        e += 2.0 ** (SPREAD[dtype] - 31) * (p * np.abs(vs)).max(1, keepdims=True) * codes
        e *= 1.01
        y[row, heads] = out
        bound[row, heads] = e + half_step(dtype) * (np.abs(out) + e) + least(dtype)
    return y, bound


def in_16_bits(cache, batch, q, scale, window, dtype, parts, by_row=True):
    """y in `dtype` where all is exact but the operand p * vscale, which goes to fp16 in `parts` parts, after a power of two
    that brings the row's largest (not by_row: the largest value scale of its sequence, at p = 1) to [2^6, 2^7)."""
    y = torch.zeros((batch.rows,) + q.shape[1:], dtype=torch.float64)
    largest = {int(batch.offsets[b]) + i: np.nanmax(np.abs(np.concatenate([cache.meta(1, 0)[x, :, :].ravel() for x in batch.table[b] if x >= 0])))
               for b, n in enumerate(batch.n) for i in range(n) if (batch.table[b] >= 0).any()}
    for row, heads, qq, kx, kmid, _, vx, vmid, vs in terms(cache, batch, q, scale, window):
        s = (qq @ kx.T + kmid * qq.sum(1)[:, None]) * scale
        p = np.exp(s - s.max(1, keepdims=True))
        w = p * vs
        unit = np.exp2(6 - np.floor(np.log2(np.abs(w).max(1, keepdims=True) if by_row else np.full((len(p), 1), largest[row]))))
        left, got = w * unit, 0
        for _ in range(parts):
            part = left.astype(np.float16).astype(np.float64)
            got, left = got + part, left - part
        codes = np.divide(vx, vs[:, None], out=np.zeros_like(vx), where=vs[:, None] != 0)
        y[row, heads] = torch.from_numpy((got / unit @ codes + (p @ vmid)[:, None]) / p.sum(1, keepdims=True))
    return y.to(dtype)


def far(got, y, bound):
    """The largest error, in bounds."""
    g = got.detach().cpu().to(torch.float64).numpy().reshape(y.shape)
    with np.errstate(invalid="ignore", divide="ignore"):
        r = np.abs(g - y) / bound
    return float(np.nanmax(np.where(np.abs(g - y) == 0, 0, r)))
