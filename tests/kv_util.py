"""The quantised key/value cache in numpy: rows quantised step by step in
binary32, pages laid out byte by byte from the formulas, attention in 64 bits
with the error bound of the library's steps."""
import numpy as np
import torch

import bit_weight_only_pack_amd as lb

FMT = {"i8": lb.LOWBIT_KV_I8, "u4": lb.LOWBIT_KV_U4}
DT = {"f16": (lb.LOWBIT_F16, torch.float16), "bf16": (lb.LOWBIT_BF16, torch.bfloat16)}
U32 = 2.0 ** -24                                   # half a step of binary32, relative
F32MAX = np.finfo(np.float32).max


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def least(dtype):
    """Half the spacing of subnormal values."""
    fi = torch.finfo(dtype)
    return fi.smallest_normal * fi.eps / 2


def quantise(fmt, x):
    """codes (uint8, biased by 128 for i8), scale, minimum (i8: None) of float32 rows [.., D]."""
    x = x.astype(np.float32)
    bad = ~np.isfinite(x).all(-1)
    x = np.where(bad[..., None], np.float32(0), x)
    with np.errstate(divide="ignore", over="ignore", invalid="ignore"):
        if fmt == "i8":
            amax = np.abs(x).max(-1)
            inv = np.minimum(np.float32(127) / amax, F32MAX)
            codes = np.rint(x * inv[..., None]) + 128
            scale = amax / np.float32(127)
            low = None
        else:
            lo, hi = x.min(-1), x.max(-1)
            h = np.float32(0.5) * hi - np.float32(0.5) * lo
            inv = np.minimum(np.float32(15) / h, F32MAX)
            codes = np.rint((np.float32(0.5) * x - np.float32(0.5) * lo[..., None]) * inv[..., None])
            scale = h / np.float32(7.5)
            low = np.where(bad, np.float32(0), lo).astype(np.float32)
    codes = np.where(bad[..., None], 128 if fmt == "i8" else 0, codes).astype(np.uint8)
    return codes, np.where(bad, np.float32(np.nan), scale).astype(np.float32), low


def places(fmt, page, D):
    """Byte (of a head's K or V codes) and shift of every (token, dim): K bytes, V bytes, K shift, V shift."""
    t, d = np.arange(page)[:, None], np.arange(D)[None, :]
    zero = np.zeros((page, D), np.int64)
    if fmt == "i8":
        return (((t // 16 * (D // 64) + d // 64) * 4 + d % 64 // 16) * 256 + t % 16 * 16 + d % 16,
                ((t // 64 * (D // 16) + d // 16) * 4 + t % 16 // 4) * 256 + d % 16 * 16 + t % 64 // 16 * 4 + t % 4,
                zero, zero)
    pair = {0: (0, 0), 2: (0, 4), 4: (1, 0), 6: (1, 4), 1: (2, 0), 3: (2, 4), 5: (3, 0), 7: (3, 4)}
    byte = np.array([pair[i][0] for i in range(8)])[d % 8]
    shift = np.array([pair[i][1] for i in range(8)])[d % 8]
    return (((t // 32 * (D // 64) + d // 64) * 4 + d % 64 // 16) * 256 + t % 16 * 16 + t % 32 // 16 * 8
            + d % 16 // 8 * 4 + byte,
            ((t // 64 * (D // 32) + d // 32) * 4 + t % 16 // 4) * 256 + d % 16 * 16 + t % 64 // 16 * 4 + t % 4,
            shift + zero, d % 32 // 16 * 4 + zero)


class Cache:
    """A cache as numpy bytes [pages][heads][part]."""

    def __init__(self, fmt, pages, page, heads, D, fill=0):
        self.fmt, self.pages, self.page, self.heads, self.D = fmt, pages, page, heads, D
        self.codes = page * D * (8 if fmt == "i8" else 4) // 8
        self.arrays = 2 if fmt == "i8" else 4
        self.part = 2 * self.codes + self.arrays * page * 4
        self.b = np.full((pages, heads, self.part), fill, np.uint8)
        self.place = places(fmt, page, D)

    def meta(self, i, which):
        """fp32 array of K (i = 0) or V: scale (which = 0) or minimum, as a view [pages][heads][page]."""
        at = 2 * self.codes + (i * self.arrays // 2 + which) * self.page * 4
        return self.b[:, :, at:at + self.page * 4].view(np.float32)

    def put(self, i, page, t, head, x):
        """Rows x [n][D] (float32) to places t [n] of pages page [n] of one head."""
        codes, scale, low = quantise(self.fmt, x)
        place, shift = self.place[i][t], self.place[2 + i][t]
        page = np.asarray(page)[:, None]
        at = i * self.codes + place
        if self.fmt == "i8":
            self.b[page, head, at] = codes
        else:
            for s in (0, 4):                        # the nibbles of a byte belong to one token: one after the other
                rows, cols = np.nonzero(shift == s)
                p, a = page[rows, 0], at[rows, cols]
                self.b[p, head, a] = (self.b[p, head, a] & (0xF0 >> s)) | (codes[rows, cols] << s)
            self.meta(i, 1)[page[:, 0], head, t] = low
        self.meta(i, 0)[page[:, 0], head, t] = scale

    def get(self, i, page, t, head):
        """code * scale and minimum, in float64, of places t of pages page."""
        place, shift = self.place[i][t], self.place[2 + i][t]
        c = self.b[np.asarray(page)[:, None], head, i * self.codes + place]
        scale = self.meta(i, 0)[page, head, t].astype(np.float64)[:, None]
        with np.errstate(invalid="ignore"):
            if self.fmt == "i8":
                return (c.astype(np.float64) - 128) * scale, np.zeros_like(scale)
            return ((c >> shift) & 15) * scale, self.meta(i, 1)[page, head, t].astype(np.float64)[:, None]

    def device(self):
        return torch.from_numpy(self.b).cuda()

    def handle(self, data):
        return lb.make_kv_cache(data, FMT[self.fmt], self.pages, self.page, self.heads, self.D)


class Batch:
    """Sequences: rows n[b] and lengths lens[b], with pages from `pages` (all different, shuffled) unless given."""

    def __init__(self, cache, n, lens, rng, width=None, extra_rows=0, max_rows=None):
        self.n, self.lens = list(n), list(lens)
        used = [-(-max(x, 0) // cache.page) for x in lens]
        self.width = max(used + [0]) if width is None else width
        ids = rng.permutation(cache.pages)
        assert sum(used) <= cache.pages
        self.table = np.full((len(n), self.width), -1, np.int32)
        at = 0
        for b, u in enumerate(used):
            u = min(u, self.width)
            self.table[b, :u] = ids[at:at + u]
            at += u
        self.offsets = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.rows = int(sum(n)) + extra_rows
        self.max_rows = max(self.n + [0]) if max_rows is None else max_rows

    def device(self):
        self.d = [torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda() for a in (self.table, self.lens, self.offsets)]
        return self.handle()

    def handle(self):
        t, lens, o = self.d
        return lb.make_kv_batch(t, self.width, lens, o, len(self.n), self.rows, self.max_rows)

    def where(self, cache, b, pos):
        """page (or -1) and place of positions pos of sequence b."""
        i = pos // cache.page
        ok = (pos >= 0) & (i < self.width)
        page = np.where(ok, self.table[b, np.clip(i, 0, max(self.width - 1, 0))] if self.width else -1, -1)
        return np.where((page >= 0) & (page < cache.pages), page, -1), pos % cache.page


def rows_of(batch):
    """(sequence, row, position) of every row of the batch."""
    for b, (n, length) in enumerate(zip(batch.n, batch.lens)):
        for i in range(n):
            yield b, int(batch.offsets[b]) + i, length - n + i


def write64(cache, batch, k, v):
    """lowbit_kv_write on the numpy cache; k, v: float32 [rows][heads][D]."""
    for b, row, pos in rows_of(batch):
        page, t = batch.where(cache, b, np.array([pos]))
        if page[0] < 0:
            continue
        for h in range(cache.heads):
            cache.put(0, page, t, h, k[row, h][None])
            cache.put(1, page, t, h, v[row, h][None])


def attention64(cache, batch, q, scale, window, dtype):
    """y and its error bound [rows][Hq][D] in float64; q: float64 [rows][Hq][D] as the type holds it.

    Steps, relative to sums of magnitudes: the score's D products and their scale (D + 6 roundings of binary32, each
    dim at most |q| (|code scale| + |minimum|)); the exponent's two roundings of |score|; p and its sum (a few roundings
    each, the sum over at most n tokens); p * vscale to fp16 (half a step 2^-11 for results of bf16; for those of fp16 the
    rest in a second part, and half a step of that: 2^-22; or half the spacing 2^-25 of what is near zero, in units of
    2^(E - 6), E the exponent of the largest value scale that some row of the call sees); the sum over tokens (n
    roundings); the joining of parts (a few roundings, one exp2 each, of 2^-22); the result's own."""
    rows, Hq, D = q.shape
    y, bound = np.zeros((batch.rows, Hq, D)), np.zeros((batch.rows, Hq, D))
    group = Hq // cache.heads
    for b, (n, length) in enumerate(zip(batch.n, batch.lens)):
        pos = np.arange(max(length, 0))
        page, t = batch.where(cache, b, pos)
        have = page >= 0
        page, t = np.maximum(page, 0), t
        for h in range(cache.heads):
            if len(pos):
                (kc, kl), (vc, vl) = cache.get(0, page, t, h), cache.get(1, page, t, h)
                vscale = np.abs(cache.meta(1, 0)[page, h, t].astype(np.float64))
            for i in range(n):
                row, at = int(batch.offsets[b]) + i, length - n + i
                seen = have & (pos <= at)
                if window:
                    seen &= pos > at - window
                seen = np.nonzero(seen)[0]
                if not len(seen):
                    continue
                qq = q[row, h * group:(h + 1) * group]
                s = (qq @ (kc[seen] + kl[seen]).T) * scale
                mag = (np.abs(qq) @ (np.abs(kc[seen]) + np.abs(kl[seen])).T) * scale
                with np.errstate(invalid="ignore"):
                    p = np.exp(s - s.max(1, keepdims=True))
                    p /= p.sum(1, keepdims=True)
                yy = p @ (vc[seen] + vl[seen])
                size = p @ (np.abs(vc[seen]) + np.abs(vl[seen]))
                ds = ((D + 8) * U32 * mag + 4 * U32 * np.abs(s)).max(1, keepdims=True)
                m = len(seen)
                rel = (2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -22) + 2 * np.expm1(ds) + (2 * m + 64) * U32 + 2.0 ** -20
                fine = vscale[have][np.isfinite(vscale[have])]
                tiny = m * 2.0 ** -25 * 2.0 ** -6 * (fine.max() if len(fine) else 0) * 128
                e = size * rel + tiny
                y[row, h * group:(h + 1) * group] = yy
                bound[row, h * group:(h + 1) * group] = e + half_step(dtype) * (np.abs(yy) + e) + least(dtype)
    return y, bound


def assert_within(got, y, bound, what=""):
    g = got.detach().cpu().to(torch.float64).numpy().reshape(y.shape)
    same_nan = np.isnan(g) & np.isnan(y)
    bad = ~((np.abs(g - y) <= bound) | same_nan)
    assert not bad.any(), "%s: %d of %d values off, worst %.3g of its bound at %s" % (
        what, bad.sum(), bad.size, np.nanmax(np.abs(g - y)[bad] / bound[bad]), np.argwhere(bad)[:3].tolist())


def rows(rng, n, heads, D, dtype, big=True):
    """Rows as a type holds them (torch, CPU): normal values of several sizes, some dims larger."""
    x = rng.standard_normal((n, heads, D)) * (0.5 + rng.random((n, heads, 1)))
    if big:
        x *= np.where(rng.random((1, heads, D)) < 0.03, 4.0, 1.0)
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


def attend(cache_handle, batch, q, q_stride, Hq, dt, scale, window, rows_out, D, fill=float("nan"), stream=None, nb=None):
    """lowbit_kv_attention into a prefilled y with a dirty workspace."""
    code, dtype = DT[dt]
    h = batch.handle()
    need = lb.lowbit_kv_attention_workspace_bytes(cache_handle, h, Hq)
    ws = torch.full((max(need, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    y = torch.full((rows_out, Hq, D), fill, dtype=dtype, device="cuda")
    lb.check(lb.lowbit_kv_attention(cache_handle, h, q, q_stride, Hq, code, scale, window, y, ws, need, stream))
    torch.cuda.synchronize()
    return y
