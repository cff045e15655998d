"""Caches whose value scales are far apart: what a row sees of them counts for much, for little or for nothing."""
import numpy as np
import torch

from kv_util import DT, Batch, Cache, rows


def filled(rng, fmt, pages, page, heads, D, dtype):
    cache = Cache(fmt, pages, page, heads, D)
    for i in range(2):
        x = rows(rng, pages * page, heads, D, dtype).float().numpy()
        at = np.arange(pages * page)
        for h in range(heads):
            cache.put(i, at // page, at % page, h, x[:, h])
    return cache


def positive(rng, n, Hq, D, dtype):
    """Queries whose product with a row of ones is far from zero."""
    return rows(rng, n, Hq, D, torch.float32).abs().clamp_(min=0.25).to(dtype)


def scaled(cache, i, where, f):
    """Keys or values of places (page, token) of all heads times f."""
    for which in range(cache.arrays // 2):
        cache.meta(i, which)[where[0], :, where[1]] *= np.float32(f)


KINDS = ("heavy", "behind", "sinks", "ladder")


def case(kind, fmt, D, dt, n, gap, long=False):
    """(cache, batch, q, scale) of one kind:

    heavy    one token's value scale is 2^gap times the others', its weight 2^-100 or so; the same in a second page
    behind   the values of a chunk's last tokens are 2^gap times the others': rows before them do not see them
    sinks    the first tokens take nearly all of the weight and their values are zeros; the others weigh some 2^-gap
    ladder   value scales of all sizes over 2^gap"""
    rng = np.random.default_rng(1000 * KINDS.index(kind) + D + gap)
    dtype, heads, group = DT[dt][1], 2, 2
    lens = [3000, 2500] if long else [200, 150]
    cache = filled(rng, fmt, 24 if long else 8, 256 if long else 64, heads, D, dtype)
    batch = Batch(cache, n, lens, rng)
    q = positive(rng, batch.rows, heads * group, D, dtype)
    scale = D ** -0.5 * 0.25
    ones = np.ones((1, D), np.float32)
    per = float(q.float().sum(-1).mean()) * scale                     # score of a row of ones
    for b, length in enumerate(lens):
        def place(p):
            page, t = batch.where(cache, b, np.atleast_1d(p))
            return page, t
        if kind == "heavy":
            for p in (3, 100):
                page, t = place(p)
                for h in range(heads):
                    cache.put(0, page, t, h, -ones * (70 / per))      # e^-70
                scaled(cache, 1, (page, t), 2.0 ** gap)
        elif kind == "behind":
            scaled(cache, 1, place(np.arange(length - (n[b] + 1) // 2, length)), 2.0 ** gap)
            if dt == "f16":                                           # results within the type's range
                scaled(cache, 1, place(np.arange(length)), 2.0 ** -max(gap - 10, 0))
        elif kind == "sinks":
            for p in (0, 1):
                page, t = place(p)
                for h in range(heads):
                    cache.put(0, page, t, h, ones * (gap * 0.6931 / per))
                    cache.put(1, page, t, h, 0 * ones)
            scaled(cache, 1, place(np.arange(length)), 2.0 ** (12 if dt == "f16" else 0))
        else:
            f = np.ldexp(1.0, -rng.integers(0, gap + 1, length)).astype(np.float32)
            page, t = place(np.arange(length))
            for which in range(cache.arrays // 2):
                cache.meta(1, which)[page, :, t] *= f[:, None]
    return cache, batch, q, float(np.float32(scale))


def largest(fmt, D, n, long, offset):
    """As above: bf16 values up to the type's largest (offset: all of one sign and close together), weights much alike."""
    rng = np.random.default_rng(D + 7 * long)
    lens = [3000, 2500] if long else [200, 150]
    cache = filled(rng, fmt, 24 if long else 8, 256 if long else 64, 1, D, torch.bfloat16)
    places = cache.pages * cache.page
    x = rng.uniform(0.75, 1.0, (places, D)) if offset else rng.uniform(-1, 1, (places, D))
    x = torch.from_numpy(np.ldexp(x, 127)).to(torch.bfloat16)
    at = np.arange(places)
    cache.put(1, at // cache.page, at % cache.page, 0, x.float().numpy())
    batch = Batch(cache, n, lens, rng)
    return cache, batch, rows(rng, batch.rows, 2, D, torch.bfloat16), float(np.float32(D ** -0.5 / 4))
