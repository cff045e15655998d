"""Writing and reading the quantised key/value cache, against numpy: the bytes
that a write leaves (every one of the cache, so that no other token's are
touched) and the values that a read returns."""
import numpy as np
import pytest
import torch

import bit_weight_only_pack_amd as lb
from kv_util import DT, U32, Batch, Cache, half_step, least, rows, rows_of, write64

pytestmark = pytest.mark.gpu


def to_gpu_slice(x, extra, lead=8):
    """Rows in a wider matrix, as a stacked projection leaves them: (matrix, address of the rows, stride)."""
    flat = x.flatten(1)
    wide = torch.full((max(x.shape[0], 1), lead + flat.shape[1] + extra), float("nan"), dtype=x.dtype)
    wide[:x.shape[0], lead:lead + flat.shape[1]] = flat
    wide = wide.cuda()
    return wide, wide.data_ptr() + 2 * lead, wide.shape[1]


def write(cache, data, batch, k, v, dt, stream=None):
    wk, ak, sk = to_gpu_slice(k, 16)
    wv, av, sv = to_gpu_slice(v, 0)
    lb.check(lb.lowbit_kv_write(cache.handle(data), batch.device(), ak, sk, av, sv, DT[dt][0], stream))
    torch.cuda.synchronize()


def check_write(cache, batch, k, v, dt, what=""):
    data = cache.device()
    write(cache, data, batch, k, v, dt)
    write64(cache, batch, k.float().numpy(), v.float().numpy())
    got = data.cpu().numpy()
    bad = np.argwhere(got != cache.b)
    assert not len(bad), "%s: %d bytes differ, first at %s" % (what, len(bad), bad[:3].tolist())
    return data


def read(cache, data, batch, dt, fill=7.0):
    dtype = DT[dt][1]
    k = torch.full((batch.rows, cache.heads * cache.D + 8), fill, dtype=dtype, device="cuda")
    v = torch.full((batch.rows, cache.heads * cache.D), fill, dtype=dtype, device="cuda")
    lb.check(lb.lowbit_kv_read(cache.handle(data), batch.device(), k, k.shape[1], v, v.shape[1], DT[dt][0]))
    torch.cuda.synchronize()
    assert (k[:, -8:] == fill).all()
    shape = (batch.rows, cache.heads, cache.D)
    return k[:, :-8].reshape(shape).cpu(), v.reshape(shape).cpu()


def check_read(cache, data, batch, dt, fill=7.0):
    """One rounding of binary32 (of the product, or of the fused product and sum), then the type's own."""
    dtype = DT[dt][1]
    named = np.zeros(batch.rows, bool)
    for i, got in enumerate(read(cache, data, batch, dt, fill)):
        g = got.to(torch.float64).numpy()
        for b, row, pos in rows_of(batch):
            named[row] = True
            page, t = batch.where(cache, b, np.array([pos]))
            for h in range(cache.heads):
                if page[0] < 0:
                    assert (g[row, h] == 0).all()
                    continue
                c, low = cache.get(i, page, t, h)
                want = c[0] + low[0]
                if np.isnan(want).any():
                    assert np.isnan(g[row, h]).all()
                    continue
                e = U32 * np.abs(want)
                assert (np.abs(g[row, h] - want) <= e + half_step(dtype) * (np.abs(want) + e) + least(dtype)).all()
        assert (g[~named] == fill).all()


# heads, rows and lengths of the sequences: one token, block and page borders crossed, whole blocks, none
SHAPES = [
    (1, [1], [1]),
    (2, [1, 1, 0, 1], [64, 65, 10, 200]),
    (3, [5, 0, 63, 64, 65], [5, 0, 100, 128, 129]),
    (1, [130, 2, 200], [130, 66, 321]),
    (2, [66, 3], [130, 257]),
]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fmt", ["i8", "u4"])
def test_write_and_read(fmt, D, dt):
    for case, (heads, n, lens) in enumerate(SHAPES):
        page = (64, 128, 256)[case % 3]
        rng = np.random.default_rng(D + case)
        cache = Cache(fmt, 14, page, heads, D, fill=0x5A)
        batch = Batch(cache, n, lens, rng, extra_rows=3)
        k, v = rows(rng, batch.rows, heads, D, DT[dt][1]), rows(rng, batch.rows, heads, D, DT[dt][1])
        data = check_write(cache, batch, k, v, dt, "case %d" % case)
        check_read(cache, data, batch, dt)


@pytest.mark.parametrize("page", [64, 128, 256])
@pytest.mark.parametrize("fmt", ["i8", "u4"])
def test_every_start_in_a_block(fmt, page):
    """Chunks of 1 to 70 rows that begin at every place of a block."""
    rng = np.random.default_rng(page)
    n = [int(rng.integers(1, 71)) for _ in range(64)]
    lens = [i + c for i, c in enumerate(n)]
    cache = Cache(fmt, 64 * 3, page, 1, 64, fill=0xA5)
    batch = Batch(cache, n, lens, rng)
    k, v = (rows(rng, batch.rows, 1, 64, torch.float16) for _ in range(2))
    check_read(cache, check_write(cache, batch, k, v, "f16"), batch, "bf16")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("fmt", ["i8", "u4"])
def test_special_rows(fmt, dt):
    """Zeros, equal values, the type's largest and smallest, an infinity, a NaN, one value apart from the rest."""
    dtype = DT[dt][1]
    fi = torch.finfo(dtype)
    rng = np.random.default_rng(3)
    D = 64
    x = rows(rng, 12, 1, D, dtype)
    x[0] = 0
    x[1] = 3
    x[2] = torch.tensor([fi.max, -fi.max] * (D // 2))
    x[3] = fi.smallest_normal * fi.eps
    x[4] = torch.tensor([fi.smallest_normal * fi.eps, 0] * (D // 2))
    x[5, 0, 9] = float("inf")
    x[6, 0, 63] = float("nan")
    x[7] = 0
    x[7, 0, 5] = -fi.max
    x[8] = -1
    x[9] = -0.0
    x[10, 0, 0] = float("-inf")
    cache = Cache(fmt, 2, 64, 1, D, fill=0x11)
    batch = Batch(cache, [12], [70], rng)
    data = check_write(cache, batch, x, x.flip(0), dt)
    check_read(cache, data, batch, dt)


@pytest.mark.parametrize("fmt", ["i8", "u4"])
def test_damaged_tables(fmt):
    """Pages outside the cache, rows before token 0, tokens past the table, offsets past the rows, rows past max_rows."""
    rng = np.random.default_rng(5)
    cache = Cache(fmt, 9, 64, 2, 64, fill=0x33)
    batch = Batch(cache, [70, 10, 40, 3, 2], [150, 4, 100, 3, 0], rng, width=2)      # 150 tokens, room for 128
    batch.table[0, 1] = 9
    batch.table[2, 0] = -5
    batch.table[3, 0] = 2 ** 31 - 1
    k, v = (rows(rng, batch.rows, 2, 64, torch.bfloat16) for _ in range(2))
    check_read(cache, check_write(cache, batch, k, v, "bf16"), batch, "bf16")
    # offsets that end past the rows: cut; the last sequence then stands for fewer rows
    batch = Batch(cache, [4, 6], [40, 50], rng)
    batch.rows = 8
    batch.n = [4, 4]
    k, v = (rows(rng, 8, 2, 64, torch.bfloat16) for _ in range(2))
    data = cache.device()
    batch.offsets = np.array([0, 4, 99], np.int32)
    write(cache, data, batch, k, v, "bf16")
    batch.offsets = np.array([0, 4, 8], np.int32)
    write64(cache, batch, k.float().numpy(), v.float().numpy())
    assert np.array_equal(data.cpu().numpy(), cache.b)
    # descending offsets and negative lengths name no rows
    batch.offsets, batch.lens = np.array([8, 2, 1], np.int32), [-3, -2 ** 31]
    write(cache, data, batch, k, v, "bf16")
    assert np.array_equal(data.cpu().numpy(), cache.b)
    # rows of a sequence past max_rows are left out
    batch = Batch(cache, [5, 9], [40, 50], rng)
    k, v = (rows(rng, 14, 2, 64, torch.bfloat16) for _ in range(2))
    batch.max_rows = 5
    write(cache, data, batch, k, v, "bf16")
    few = Batch(cache, [5, 5], [40, 46], rng)
    few.table = batch.table
    write64(cache, few, k.float().numpy()[:10], v.float().numpy()[:10])
    assert np.array_equal(data.cpu().numpy(), cache.b)


def test_pages_past_4_gib():
    """Pages whose offsets pass 2^32 bytes."""
    rng = np.random.default_rng(8)
    heads, D = 16, 256
    part = lb.lowbit_kv_page_bytes(lb.LOWBIT_KV_I8, 256, 1, D)
    pages = (5 << 30) // (heads * part)
    data = torch.empty(pages * heads * part, dtype=torch.uint8, device="cuda")
    cache = Cache("i8", 4, 256, heads, D)
    batch = Batch(cache, [300, 2], [400, 258], rng)
    far = np.array([pages - 1, pages - 3, pages // 2, pages - 7], np.int32)
    small = batch.table.copy()
    batch.table = far[batch.table]
    k, v = (rows(rng, batch.rows, heads, D, torch.float16) for _ in range(2))
    view = data.view(pages, heads, part)
    view[torch.from_numpy(far).cuda().long()] = 0
    handle = lb.make_kv_cache(data, lb.LOWBIT_KV_I8, pages, 256, heads, D)
    lb.check(lb.lowbit_kv_write(handle, batch.device(), k.cuda(), heads * D, v.cuda(), heads * D, lb.LOWBIT_F16))
    torch.cuda.synchronize()
    batch.table = small
    write64(cache, batch, k.float().numpy(), v.float().numpy())
    assert np.array_equal(view[torch.from_numpy(far).cuda().long()].cpu().numpy(), cache.b)


@pytest.mark.parametrize("fmt", ["i8", "u4"])
def test_graph_replays_with_new_lengths(fmt):
    """One captured write and read; lengths, pages and rows change between the replays, with eager calls between."""
    rng = np.random.default_rng(9)
    cache = Cache(fmt, 12, 64, 2, 64, fill=1)
    data = cache.device()
    B, most = 3, 4
    batch = Batch(cache, [4, 1, 2], [100, 64, 2], rng, width=4)
    batch.max_rows, batch.rows = most, B * most
    handle = batch.device()
    k, v, ko, vo = (torch.zeros((B * most, 2, 64), dtype=torch.float16, device="cuda") for _ in range(4))
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()

    def call(st):
        lb.check(lb.lowbit_kv_write(cache.handle(data), handle, k, 128, v, 128, lb.LOWBIT_F16, st))
        lb.check(lb.lowbit_kv_read(cache.handle(data), handle, ko, 128, vo, 128, lb.LOWBIT_F16, st))

    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            call(stream.cuda_stream)
    for turn in range(4):
        n = [int(x) for x in rng.integers(0, most + 1, B)]
        new = Batch(cache, n, [int(c + rng.integers(0, 200)) for c in n], rng, width=4)
        for d, a in zip(batch.d, (new.table, new.lens, new.offsets)):
            d.copy_(torch.from_numpy(np.ascontiguousarray(a, np.int32)))
        kk, vv = (rows(rng, B * most, 2, 64, torch.float16) for _ in range(2))
        k.copy_(kk), v.copy_(vv), ko.fill_(5), vo.fill_(5)
        torch.cuda.synchronize()
        if turn % 2:
            call(None)
        else:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        new.rows = B * most
        write64(cache, new, kk.float().numpy(), vv.float().numpy())
        assert np.array_equal(data.cpu().numpy(), cache.b)
        total = sum(n)
        assert (ko[total:] == 5).all() and (vo[total:] == 5).all()
        for got, src in ((ko, kk), (vo, vv)):
            # a step of the codes at most: the row's largest over 254, or its span over 30
            x = src[:total].float()
            step = x.abs().amax(-1) / 254 if fmt == "i8" else (x.amax(-1) - x.amin(-1)) / 30
            off = (got[:total].cpu().float() - x).abs().amax(-1)
            assert (off <= step * 1.01 + 2.0 ** -10 * x.abs().amax(-1)).all()


@pytest.mark.parametrize("fmt", ["i8", "u4"])
def test_long_prompt_at_once_and_in_parts(fmt):
    """Rows of more than 32 MB in one call, and the same in calls of a few hundred: equal bytes, equal rows."""
    rng = np.random.default_rng(31)
    heads, D, page, total = 20, 128, 128, 3333
    assert total * heads * D * 4 > 32 << 20
    cache = Cache(fmt, 30, page, heads, D)
    k, v = (torch.randn((total, heads, D), device="cuda").to(torch.bfloat16) for _ in range(2))
    k[5, 3, 100] = float("inf")
    table = rng.permutation(30).astype(np.int32)
    stride, datas, outs = heads * D, [], []
    for step in (total, 700):
        data = torch.full(cache.b.shape, 0x55, dtype=torch.uint8, device="cuda")
        back = [torch.zeros((total, heads, D), dtype=torch.float16, device="cuda") for _ in range(2)]
        for call, x, y in ((lb.lowbit_kv_write, (k, v), lb.LOWBIT_BF16), (lb.lowbit_kv_read, back, lb.LOWBIT_F16)):
            for at in range(0, total, step):
                n = min(step, total - at)
                batch = Batch(cache, [n], [at + n], rng, width=27)
                batch.table[0] = table[:27]
                lb.check(call(cache.handle(data), batch.device(), x[0][at:].data_ptr(), stride, x[1][at:].data_ptr(),
                              stride, y))
        torch.cuda.synchronize()
        datas.append(data)
        outs.append(back)
    assert torch.equal(datas[0], datas[1])
    for a, b in zip(*outs):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    # 8 bits: half a step of amax / 127; 4: of the row's range / 15; the fp16 rounding is far below either's margin of 2 %
    step = (lambda x: x.amax(-1) - x.amin(-1)) if fmt == "u4" else (lambda x: x.abs().amax(-1))
    for x, y in ((k, outs[0][0]), (v, outs[0][1])):
        x = x.float()
        half = step(x) / (15 if fmt == "u4" else 127) / 2
        good = torch.isfinite(x).all(-1)
        assert ((x - y.float()).abs().amax(-1) <= half * 1.02 + 2.0 ** -9)[good].all()
        assert torch.isnan(y[~good]).all() and int((~good).sum()) == (1 if x.isinf().any() else 0)
