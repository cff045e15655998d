"""Cases that time the quantised key/value cache and attention over it, and say what they return.

Three operators over a cache whose pages hold 8-bit codes (fp32 scale per token and head) or 4-bit codes (fp32 scale and
minimum per token and head):
  write      new tokens' key and value rows quantised into the pages, and the same rows read back as the values held
  read       the last rows of every sequence read back from the pages
  attention  a chunk of new tokens of every sequence (one to thousands) over the sequence's pages, causal

Where ``own`` is false ``run`` computes them from elementary torch operations in binary32; where it is true it calls
the library.  Sizes are those of the decoder that the package's workloads use (32 query heads of 128 over 8 key/value
heads) and generic ones beside them.

A page holds ``page`` tokens of all heads; the part of one head is K codes, V codes, then fp32 arrays of ``page``
values: K scale, V scale (8 bits) or K scale, K minimum, V scale, V minimum (4 bits).
  8 bits: a byte holds code + 128.
    K of token t, dim d: byte ((t/16 * D/64 + d/64) * 4 + d%64/16) * 256 + t%16 * 16 + d%16
    V of token t, dim d: byte ((t/64 * D/16 + d/16) * 4 + t%16/4) * 256 + d%16 * 16 + t%64/16 * 4 + t%4
  4 bits: a byte holds two codes.
    K: bytes of 32 tokens x 64 dims lie in the order d%64/16, t%16, t%32/16, d%16/8, and 4 bytes of 8 dims whose nibbles,
       lowest first, hold dims 0 2 4 6 1 3 5 7
    V: as for 8 bits over 32 dims at a time, the low nibble for d%32 < 16 and the high one for d%32 >= 16
"""
import math

import torch

own = False

F16, BF16 = torch.float16, torch.bfloat16
DTYPES = {"f16": F16, "bf16": BF16}
LARGEST = 3.4028234663852886e38


def listed():
    return [
        # one token of one sequence over a short cache: latency counts
        {"name": "attention 1 token", "op": "attention", "fmt": "i8", "dtype": "f16", "B": 1, "rows": 1, "len": 777,
         "spread": "same", "Hq": 32, "Hkv": 8, "D": 128, "page": 64, "window": 0},
        # a decode batch of sequences of all lengths: the cache's stream counts
        {"name": "attention decode", "op": "attention", "fmt": "i8", "dtype": "bf16", "B": 64, "rows": 1, "len": 8192,
         "spread": "even", "Hq": 32, "Hkv": 8, "D": 128, "page": 128, "window": 0},
        # two long documents, one token each, 4 bits: few rows over a long axis
        {"name": "attention long 4 bit", "op": "attention", "fmt": "u4", "dtype": "f16", "B": 2, "rows": 1,
         "len": 131072, "spread": "even", "Hq": 32, "Hkv": 4, "D": 128, "page": 256, "window": 0},
        # a few drafted tokens a sequence, narrow heads, eight query heads to each
        {"name": "attention drafts", "op": "attention", "fmt": "i8", "dtype": "bf16", "B": 24, "rows": 5, "len": 4001,
         "spread": "even", "Hq": 16, "Hkv": 2, "D": 64, "page": 64, "window": 0},
        # a prefill chunk at the end of a long prompt: the matrix cores count
        {"name": "attention prefill", "op": "attention", "fmt": "i8", "dtype": "bf16", "B": 1, "rows": 2048,
         "len": 16384, "spread": "same", "Hq": 32, "Hkv": 8, "D": 128, "page": 128, "window": 0},
        # prompts of odd lengths under a window, five query heads to each head
        {"name": "attention ragged window", "op": "attention", "fmt": "u4", "dtype": "f16", "B": 6, "rows": 1499,
         "len": 5801, "spread": "even", "Hq": 20, "Hkv": 4, "D": 128, "page": 64, "window": 1000},
        # one prompt's chunk beside a decode batch, wide heads
        {"name": "attention mixed", "op": "attention", "fmt": "i8", "dtype": "bf16", "B": 32, "rows": 1024,
         "len": 4096, "spread": "mixed", "Hq": 8, "Hkv": 4, "D": 256, "page": 128, "window": 0},
        # a decode batch's new tokens: latency counts
        {"name": "write decode", "op": "write", "fmt": "i8", "dtype": "f16", "B": 32, "rows": 1, "len": 2048,
         "spread": "even", "Hq": 32, "Hkv": 8, "D": 128, "page": 64},
        # a long prompt
        {"name": "write prompt", "op": "write", "fmt": "i8", "dtype": "bf16", "B": 1, "rows": 16384, "len": 16384,
         "spread": "same", "Hq": 32, "Hkv": 8, "D": 128, "page": 128},
        # odd prompts whose blocks begin and end anywhere, 4 bits
        {"name": "write ragged 4 bit", "op": "write", "fmt": "u4", "dtype": "f16", "B": 7, "rows": 701, "len": 3333,
         "spread": "even", "Hq": 20, "Hkv": 4, "D": 128, "page": 64},
        # the end of one sequence, 4 bits
        {"name": "read one", "op": "read", "fmt": "u4", "dtype": "f16", "B": 1, "rows": 333, "len": 1001,
         "spread": "same", "Hq": 16, "Hkv": 2, "D": 64, "page": 64},
        # whole sequences taken out of the cache
        {"name": "read batch", "op": "read", "fmt": "i8", "dtype": "bf16", "B": 16, "rows": 8192, "len": 8192,
         "spread": "even", "Hq": 32, "Hkv": 8, "D": 128, "page": 128},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("attention", "attention", "attention", "write", "read"))
    while True:
        Hkv, group, D = rng.choice((1, 2, 3, 4, 8, 16)), rng.choice((1, 2, 3, 4, 5, 6, 7, 8, 16)), rng.choice((64, 128, 128, 256))
        B, length = _log(rng, 1, 128), _log(rng, 1, 131072)
        rows = min(length, 1 if op == "attention" and rng.random() < 0.5 else _log(rng, 1, 16384))
        case = {"op": op, "fmt": rng.choice(("i8", "u4")), "dtype": rng.choice(("f16", "bf16")), "B": B, "rows": rows,
                "len": length, "spread": rng.choice(("same", "even", "mixed")), "Hq": Hkv * group, "Hkv": Hkv, "D": D,
                "page": rng.choice((64, 128, 256))}
        # no more of the cache, and no more scores of the plain form, than the largest listed cases have
        if B * length * Hkv * D > 64 * 8192 * 8 * 128 or B * rows * Hkv * D > 16 * 8192 * 8 * 128:
            continue
        if op != "attention":
            return case
        if B * rows * Hkv * group * length <= 32 * 2048 * 16384 and B * rows * Hkv * group * length * D <= 32 * 2048 * 16384 * 128:
            return {**case, "window": 0 if rng.random() < 0.8 else _log(rng, 1, length)}


def _shape(case):
    """Rows and lengths of the sequences: all alike, of all sizes up to the case's, or one long chunk beside single rows."""
    B, rows, length = case["B"], case["rows"], case["len"]
    part = [1.0 if case["spread"] == "same" or b == 0 else ((b + 0.5) * 0.6180339887498949) % 1.0 for b in range(B)]
    lens = [max(1, int(length * p)) for p in part]
    n = [1 if case["spread"] == "mixed" and b else max(1, int(rows * part[B - 1 - b] if b else rows)) for b in range(B)]
    return [min(a, c) for a, c in zip(n, lens)], lens


def _bits(case):
    return 8 if case["fmt"] == "i8" else 4


def _generator(seed, part):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 64 + part)


def _rows(n, heads, D, seed, part):
    """Rows of n tokens: some dims larger than others in every token, as keys have them, and tokens of several sizes."""
    g = _generator(seed, part)
    x = torch.randn(n, heads, D, generator=g, device="cuda")
    x *= torch.where(torch.rand(1, heads, D, generator=g, device="cuda") < 0.03, 4.0, 1.0)
    x *= 0.5 + torch.rand(n, heads, 1, generator=g, device="cuda")
    return x


def _ratio(a, b):
    """a / b in one rounding: torch takes a number divided by a tensor, or the reverse, as a product with a reciprocal."""
    like = b if torch.is_tensor(b) else a
    return torch.as_tensor(a, dtype=like.dtype, device="cuda").expand_as(like) / torch.as_tensor(b, dtype=like.dtype, device="cuda").expand_as(like)


def _quantise(fmt, x):
    """Codes of rows in binary32 [.., D], and their scale and minimum (None for 8 bits)."""
    if fmt == "i8":
        amax = x.abs().amax(-1, keepdim=True)
        codes = torch.round(x * _ratio(127, amax).clamp_(max=LARGEST))
        return torch.where(amax > 0, codes, 0), _ratio(amax, 127)[..., 0], None
    lo = x.amin(-1, keepdim=True)
    h = 0.5 * x.amax(-1, keepdim=True) - 0.5 * lo
    codes = torch.round((0.5 * x - 0.5 * lo) * _ratio(15, h).clamp_(max=LARGEST))
    return torch.where(h > 0, codes, 0), _ratio(h, 7.5)[..., 0], lo[..., 0]


def _bytes(fmt, codes, values):
    """Bytes of rows of codes: for 8 bits and for the values' 4 bits as the rows lie, for the keys' 4 bits nibbles by 8 dims."""
    D = codes.shape[-1]
    if fmt == "i8":
        return (codes + 128).to(torch.uint8)
    c = codes.to(torch.uint8)
    c = c.view(*c.shape[:-1], D // 32, 2, 16) if values else c.view(*c.shape[:-1], D // 8, 4, 2).transpose(-1, -2).reshape(
        *c.shape[:-1], D // 8, 4, 2).transpose(-1, -2)
    return (c[..., 0, :] | c[..., 1, :] << 4).flatten(-2)


def _places(fmt, page, D):
    """Places [page][bytes of a row] of the bytes of a token's row among a head's codes: keys, values."""
    t = torch.arange(page, device="cuda")[:, None]
    b = torch.arange(D if fmt == "i8" else D // 2, device="cuda")
    # 4 bytes hold 4 tokens of a dim in the values' part, and the dims of a token in the keys'
    values = ((t // 64 * b.numel() // 16 + b // 16) * 4 + t % 16 // 4) * 256 + b % 16 * 16 + t % 64 // 16 * 4 + t % 4
    if fmt == "i8":
        return (t // 16 * (D // 64) * 4 + b // 16) * 256 + t % 16 * 16 + b % 16, values
    return (t // 32 * (D // 64) * 4 + b // 8) * 256 + t % 16 * 16 + t % 32 // 16 * 8 + b % 8, values


def _parts(fmt, page, D):
    """Bytes of a head's codes (of keys, or of values) in a page, and of its whole part of the page."""
    codes = page * D * (8 if fmt == "i8" else 4) // 8
    return codes, 2 * codes + page * (8 if fmt == "i8" else 16)


def prepare(case, seed):
    s = dict(case)
    fmt, B, Hq, Hkv, D, page = (case[k] for k in ("fmt", "B", "Hq", "Hkv", "D", "page"))
    n, lens = _shape(case)
    total, width = sum(n), -(-case["len"] // page)
    used = [-(-x // page) for x in lens]
    ids = torch.randperm(sum(used), generator=_generator(seed, 1), device="cuda").to(torch.int32)
    s["table"] = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    s["table"][torch.arange(width, device="cuda") < torch.tensor(used, device="cuda")[:, None]] = ids
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["offsets"] = torch.tensor([sum(n[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
    s["pages"], s["total"], s["most"] = sum(used), total, max(n)
    codes, part = _parts(fmt, page, D)
    s["cache"] = torch.zeros(s["pages"], Hkv, part, dtype=torch.uint8, device="cuda")
    s["place"] = _places(fmt, page, D)
    if case["op"] != "write":
        # pages as earlier steps left them, 64 Mi values at a time
        many = max(1, (1 << 26) // (Hkv * page * D))
        for at in range(0, s["pages"], many):
            piece = s["cache"][at:at + many]
            for i in range(2):
                x = _rows(piece.shape[0] * page, Hkv, D, seed, 16 + at // many * 2 + i).to(DTYPES[case["dtype"]]).float()
                q, scale, low = _quantise(fmt, x.view(-1, page, Hkv, D).transpose(1, 2))
                put = piece[..., i * codes:(i + 1) * codes]
                put[..., s["place"][i].flatten()] = _bytes(fmt, q, i == 1).flatten(-2)
                meta = piece[..., 2 * codes:].view(torch.float32)
                meta = meta.view(*meta.shape[:2], 2, -1, page)
                meta[:, :, i, 0] = scale
                if low is not None:
                    meta[:, :, i, 1] = low
    dtype = DTYPES[case["dtype"]]
    # query, key and value rows as the stacked projection leaves them, side by side
    s["qkv"] = torch.empty(total, (Hq + 2 * Hkv) * D, dtype=dtype, device="cuda")
    for i, (at, heads) in enumerate(((0, Hq), (Hq, Hkv), (Hq + Hkv, Hkv))):
        s["qkv"][:, at * D:(at + heads) * D] = _rows(total, heads, D, seed, 2 + i).flatten(1).to(dtype)
    if case["op"] == "attention":
        s["y"] = torch.zeros(total, Hq, D, dtype=dtype, device="cuda")
        # room for the partial results of any of these calls, as a program keeps it
        s["workspace"] = torch.empty(512 << 20, dtype=torch.uint8, device="cuda")
    else:
        s["k"] = torch.zeros(total, Hkv, D, dtype=dtype, device="cuda")
        s["v"] = torch.zeros(total, Hkv, D, dtype=dtype, device="cuda")
    return s


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import bit_weight_only_pack_amd as lb
    Hq, Hkv, D = s["Hq"], s["Hkv"], s["D"]
    dtype = lb.LOWBIT_BF16 if s["dtype"] == "bf16" else lb.LOWBIT_F16
    if "handle" not in s:
        fmt = lb.LOWBIT_KV_I8 if s["fmt"] == "i8" else lb.LOWBIT_KV_U4
        s["handle"] = (lb.make_kv_cache(s["cache"], fmt, s["pages"], s["page"], Hkv, D),
                       lb.make_kv_batch(s["table"], s["table"].shape[1], s["lens"], s["offsets"], s["B"], s["total"],
                                        s["most"]))
    cache, batch = s["handle"]
    stride = (Hq + 2 * Hkv) * D
    if s["op"] == "attention":
        lb.check(lb.lowbit_kv_attention(cache, batch, s["qkv"], stride, Hq, dtype, D ** -0.5, s["window"], s["y"],
                                        s["workspace"], s["workspace"].numel()))
        return s["y"]
    if s["op"] == "write":
        at = s["qkv"].data_ptr() + 2 * Hq * D
        lb.check(lb.lowbit_kv_write(cache, batch, at, stride, at + 2 * Hkv * D, stride, dtype))
    lb.check(lb.lowbit_kv_read(cache, batch, s["k"], Hkv * D, s["v"], Hkv * D, dtype))
    return {"k": s["k"], "v": s["v"]}


def _owners(s):
    """For every row: its sequence, and its position there."""
    offsets = s["offsets"].long()
    row = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(offsets[1:], row, right=True)
    return b, s["lens"].long()[b] - offsets[b + 1] + row


def _nibbles(fmt, rows, values):
    """Codes in binary32 of rows of bytes [.., bytes]."""
    if fmt == "i8":
        return rows.float() - 128
    if values:
        rows = rows.unflatten(-1, (-1, 16))
        return torch.stack((rows & 15, rows >> 4), -2).flatten(-3).float()
    rows = rows.unflatten(-1, (-1, 4))
    codes = torch.stack((rows & 15, rows >> 4), -1).flatten(-2)              # dims 0 2 4 6 1 3 5 7
    return codes.unflatten(-1, (2, 4)).transpose(-1, -2).flatten(-3).float()


def _values(s, pages, i):
    """Keys (i = 0) or values (1) that pages [.., Hkv, part] hold, in binary32: [.., Hkv, page, D]."""
    fmt, page, D = s["fmt"], s["page"], s["D"]
    codes, _ = _parts(fmt, page, D)
    c = pages[..., i * codes:(i + 1) * codes]
    if i:
        c = c.unflatten(-1, (page // 64, -1, 4, 16, 2, 2, 4))                # t/64, d/16, t%16/4, d%16, t%64/16, t%4
        c = c.movedim((-3, -2, -5, -1), (-6, -5, -4, -3))                    # t/64, t%64/16, t%16/4, t%4, d/16, d%16
    elif fmt == "i8":
        c = c.unflatten(-1, (page // 16, -1, 16, 16)).transpose(-3, -2)
        c = c.flatten(-2).flatten(-3, -2)
    else:
        c = c.unflatten(-1, (page // 32, -1, 16, 2, 8))                      # t/32, d/16, t%16, t%32/16, d%16
        c = c.movedim((-2, -3), (-4, -3))
    c = c.reshape(*pages.shape[:-1], page, D if fmt == "i8" else D // 2)
    meta = pages[..., 2 * codes:].view(torch.float32).unflatten(-1, (2, -1, page))[..., i, :, :]
    x = _nibbles(fmt, c, i == 1) * meta[..., 0, :, None]
    return x if fmt == "i8" else x + meta[..., 1, :, None]


def _plain(s):
    fmt, Hq, Hkv, D, page, dtype = s["fmt"], s["Hq"], s["Hkv"], s["D"], s["page"], DTYPES[s["dtype"]]
    if s["op"] == "attention":
        return _plain_attention(s)
    b, pos = _owners(s)
    at, t = s["table"].long()[b, pos // page], pos % page
    codes, _ = _parts(fmt, page, D)
    head = torch.arange(Hkv, device="cuda")[:, None]
    out = {}
    meta = s["cache"][..., 2 * codes:].view(torch.float32).unflatten(-1, (2, -1, page))

    def one(i):
        place = i * codes + s["place"][i][t]
        if s["op"] == "write":
            x = s["qkv"][:, (Hq + i * Hkv) * D:(Hq + (i + 1) * Hkv) * D].float().view(-1, Hkv, D)
            q, scale, low = _quantise(fmt, x)
            s["cache"][at[:, None, None], head, place[:, None]] = _bytes(fmt, q, i == 1)
            meta[at[:, None], head[:, 0], i, 0, t[:, None]] = scale
            if low is not None:
                meta[at[:, None], head[:, 0], i, 1, t[:, None]] = low
        x = _nibbles(fmt, s["cache"][at[:, None, None], head, place[:, None]], i == 1)
        x = x * meta[at[:, None], head[:, 0], i, 0, t[:, None]][..., None]
        if fmt == "u4":
            x = x + meta[at[:, None], head[:, 0], i, 1, t[:, None]][..., None]
        return x.to(dtype)

    out["k"] = one(0)
    out["v"] = one(1)
    return out


def _plain_attention(s):
    # every sequence padded to the most rows and the most tokens that one has
    B, Hq, Hkv, D, most, dtype = s["B"], s["Hq"], s["Hkv"], s["D"], s["most"], DTYPES[s["dtype"]]
    group, tokens = Hq // Hkv, s["table"].shape[1] * s["page"]
    pages = s["cache"][s["table"].long().clamp(min=0)]                       # [B, width, Hkv, part]
    k = _values(s, pages, 0).transpose(1, 2).reshape(B, Hkv, tokens, D)
    v = _values(s, pages, 1).transpose(1, 2).reshape(B, Hkv, tokens, D)
    offsets, lens = s["offsets"].long(), s["lens"].long()
    n = offsets[1:] - offsets[:-1]
    i = torch.arange(most, device="cuda")
    row = (offsets[:-1, None] + i).clamp(max=s["total"] - 1)
    q = s["qkv"][:, :Hq * D].float()[row].view(B, most, Hkv, group, D).transpose(1, 2).reshape(B, Hkv, most * group, D)
    scores = torch.matmul(q * D ** -0.5, k.transpose(-1, -2).contiguous())
    pos = (lens - n)[:, None] + i                                            # [B, most]
    token = torch.arange(tokens, device="cuda")
    seen = token <= pos[..., None]
    if s["window"]:
        seen &= token > pos[..., None] - s["window"]
    scores = scores.view(B, Hkv, most, group, tokens).masked_fill_(~seen[:, None, :, None], -math.inf)
    scores = torch.exp(scores - scores.amax(-1, keepdim=True).clamp_(min=-LARGEST))
    scores /= scores.sum(-1, keepdim=True).clamp_(min=1e-30)
    y = torch.matmul(scores.view(B, Hkv, most * group, tokens), v)
    y = y.view(B, Hkv, most, group, D).transpose(1, 2).reshape(B, most, Hq, D)
    return y[i < n[:, None]].to(dtype)


def work(case):
    n, lens = _shape(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    token = Hkv * (2 * D * _bits(case) // 8 + (8 if case["fmt"] == "i8" else 16))
    if case["op"] != "attention":
        values = sum(n) * 2 * Hkv * D * 2
        return {"bytes": sum(n) * token + values * (2 if case["op"] == "write" else 1), "flops": sum(n) * Hkv * D * 4}
    window = case["window"] or case["len"]
    read = sum(x - max(0, x - r + 1 - window) for r, x in zip(n, lens))
    # row i of a sequence sees min(len - rows + i + 1, window) tokens
    short = [max(0, min(r, window - (x - r))) for r, x in zip(n, lens)]
    seen = sum(c * (x - r) + c * (c + 1) // 2 + (r - c) * window for r, x, c in zip(n, lens, short))
    return {"bytes": read * token + sum(n) * Hq * D * 4, "flops": 4 * D * Hq * seen}


def _held(s, b, i):
    """Keys or values of sequence b in 64 bits [tokens, Hkv, D], byte by byte from where the layout says that they lie."""
    fmt, page, D, Hkv, length = s["fmt"], s["page"], s["D"], s["Hkv"], int(s["lens"][b])
    codes, _ = _parts(fmt, page, D)
    pages = s["cache"][s["table"][b, :-(-length // page)].long()]
    t = torch.arange(page, device="cuda")[:, None]
    d = torch.arange(D, device="cuda")
    if fmt == "i8":
        if i == 0:
            at = ((t // 16 * (D // 64) + d // 64) * 4 + d % 64 // 16) * 256 + t % 16 * 16 + d % 16
        else:
            at = ((t // 64 * (D // 16) + d // 16) * 4 + t % 16 // 4) * 256 + d % 16 * 16 + t % 64 // 16 * 4 + t % 4
        c = pages[:, :, (i * codes + at).flatten()].double() - 128
    else:
        if i == 0:
            at = (((t // 32 * (D // 64) + d // 64) * 4 + d % 64 // 16) * 16 + t % 16) * 16 + t % 32 // 16 * 8
            nibble = d % 2 * 4 + d % 8 // 2
            at, high = at + d % 16 // 8 * 4 + nibble // 2, nibble % 2
        else:
            at = ((t // 64 * (D // 32) + d // 32) * 4 + t % 16 // 4) * 256 + d % 16 * 16 + t % 64 // 16 * 4 + t % 4
            high = d % 32 // 16
        c = pages[:, :, (i * codes + at).flatten()].view(-1, Hkv, page, D)
        c = (c >> (4 * high).to(torch.uint8) & 15).double().flatten(2)
    arrays = pages[:, :, 2 * codes:].view(torch.float32).double().view(-1, Hkv, 2, 1 if fmt == "i8" else 2, page, 1)
    x = c.view(-1, Hkv, page, D) * arrays[:, :, i, 0]
    if fmt == "u4":
        x += arrays[:, :, i, 1]
    return x.transpose(1, 2).reshape(-1, Hkv, D)[:length]


def _held_after_write(s, i):
    """Values held of new rows: each step of the quantiser in 64 bits, rounded to binary32 where the definition rounds."""
    Hq, Hkv, D = s["Hq"], s["Hkv"], s["D"]
    x = s["qkv"].view(s["total"], Hq + 2 * Hkv, D)[:, Hq + i * Hkv:Hq + (i + 1) * Hkv].double()

    def f32(a):
        return a.float().double()

    def over(a, b):                                                          # one rounding, as above
        return f32(torch.div(torch.full_like(b, a) if isinstance(a, int) else a, b if torch.is_tensor(b) else torch.full_like(a, b)))

    if s["fmt"] == "i8":
        top = x.abs().max(2, keepdim=True).values
        return over(top, 127) * torch.round(f32(x * over(127, top)))
    least, half = x.min(2, keepdim=True).values, f32(x.max(2, keepdim=True).values / 2 - x.min(2, keepdim=True).values / 2)
    return least + over(half, 7.5) * torch.round(f32(f32(x / 2 - least / 2) * over(15, half)))


def exact(case, seed):
    s = prepare(case, seed)
    n, lens = _shape(case)
    if case["op"] == "write":
        return {"k": _held_after_write(s, 0), "v": _held_after_write(s, 1)}
    if case["op"] == "read":
        return {name: torch.cat([_held(s, b, i)[lens[b] - n[b]:] for b in range(case["B"])])
                for i, name in enumerate(("k", "v"))}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    group, out, first = Hq // Hkv, [], 0
    for b in range(case["B"]):
        k, v = _held(s, b, 0), _held(s, b, 1)
        q = s["qkv"][first:first + n[b], :Hq * D].double().view(n[b], Hq, D)
        first += n[b]
        ahead = torch.arange(lens[b], device="cuda") - torch.arange(lens[b] - n[b], lens[b], device="cuda")[:, None]
        hidden = ahead > 0
        if case["window"]:
            hidden |= ahead <= -case["window"]
        y = torch.empty(n[b], Hq, D, dtype=torch.float64, device="cuda")
        for h in range(Hq):
            a = torch.mm(q[:, h], k[:, h // group].t().contiguous()) / math.sqrt(D)
            y[:, h] = torch.mm(torch.softmax(a.masked_fill_(hidden, -math.inf), 1), v[:, h // group].contiguous())
        out.append(y)
    return torch.cat(out)
