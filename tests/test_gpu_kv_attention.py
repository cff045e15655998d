"""Attention over the quantised key/value cache, against its definition in 64
bits on the bytes that the cache holds (laid out in numpy, not by the library).
Error bounds are derived step by step in kv_util.attention64."""
import numpy as np
import pytest
import torch

import bit_weight_only_pack_amd as lb
from kv_bounds import bounded
from kv_util import DT, Batch, Cache, assert_within, attend, attention64, rows

pytestmark = pytest.mark.gpu


def filled(rng, fmt, pages, page, heads, D, dtype=torch.float16):
    """A cache whose pages all hold quantised rows."""
    cache = Cache(fmt, pages, page, heads, D)
    for i in range(2):
        x = rows(rng, pages * page, heads, D, dtype).float().numpy()
        at = np.arange(pages * page)
        for h in range(heads):
            cache.put(i, at // page, at % page, h, x[:, h])
    return cache


def check(cache, batch, group, dt, rng, window=0, scale=None, data=None, strided=False, what="", q=None):
    Hq, D, dtype = cache.heads * group, cache.D, DT[dt][1]
    scale = D ** -0.5 if scale is None else scale
    if q is None:
        q = rows(rng, batch.rows, Hq, D, dtype)
    batch.device()
    stride = Hq * D + (24 if strided else 0)
    wide = torch.full((max(batch.rows, 1), stride), float("nan"), dtype=dtype)
    wide[:batch.rows, :Hq * D] = q.flatten(1)
    data = cache.device() if data is None else data
    y = attend(cache.handle(data), batch, wide.cuda(), stride, Hq, dt, scale, window, batch.rows, D, fill=7.0)
    want, bound = attention64(cache, batch, q.double().numpy(), float(np.float32(scale)), window, dtype)
    named = int(batch.offsets[-1])
    assert (y[named:] == 7).all()
    assert_within(y[:named], want[:named], bound[:named], what)
    return y


# group, rows, lengths: single tokens, drafts, chunks, whole prompts, sequences without rows, one row longer than all
SHAPES = [
    (1, [1], [1]),
    (4, [1, 1, 1], [63, 64, 65]),
    (3, [1, 0, 2, 5], [130, 7, 2, 300]),
    (5, [17, 1], [17, 129]),
    (8, [2, 40], [2, 193]),
    (16, [3, 1], [100, 500]),
    (17, [1, 2], [70, 2]),
    (2, [70, 1, 9], [70, 300, 200]),
    (1, [150], [400]),
]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fmt", ["i8", "u4"])
def test_attention(fmt, D, dt):
    for case, (group, n, lens) in enumerate(SHAPES):
        rng = np.random.default_rng(100 * D + case)
        page, heads = (64, 128, 256)[case % 3], 1 + case % 2
        cache = filled(rng, fmt, 14 if page == 64 else 8, page, heads, D, DT[dt][1])
        batch = Batch(cache, n, lens, rng, extra_rows=case % 3)
        check(cache, batch, group, dt, rng, strided=case % 2 == 1, what="case %d" % case)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fmt", ["i8", "u4"])
def test_attention_token_by_token(fmt, D, dt):
    """The same within bounds that count each token by its own weight: one part of p for two is told by them."""
    for case, (group, n, lens) in enumerate(SHAPES + [(2, [60, 20], [500, 100])]):
        rng = np.random.default_rng(200 * D + case)
        page, heads = (64, 128, 256)[case % 3], 1 + case % 2
        cache = filled(rng, fmt, 14 if page == 64 else 8, page, heads, D, DT[dt][1])
        batch = Batch(cache, n, lens, rng)
        batch.device()
        window = (0, 0, 90)[case % 3]
        q = rows(rng, batch.rows, heads * group, D, DT[dt][1])
        for scale in (0.04, 0.004):
            y = attend(cache.handle(cache.device()), batch, q.cuda(), heads * group * D, heads * group, dt, scale, window,
                       batch.rows, D)
            want, bound = bounded(cache, batch, q.double().numpy(), float(np.float32(scale)), window, DT[dt][1])
            assert_within(y, want, bound, "case %d" % case)


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 200, 2 ** 31 - 1])
@pytest.mark.parametrize("fmt", ["i8", "u4"])
def test_window(fmt, window):
    rng = np.random.default_rng(window % 1000)
    cache = filled(rng, fmt, 16, 64, 1, 64)
    for n in ([1, 1, 1], [4, 100, 20]):
        check(cache, Batch(cache, n, [150, 333, 400], rng), 3, "f16", rng, window=window, what=str(n))


@pytest.mark.parametrize("width", [None, 2048])
@pytest.mark.parametrize("fmt", ["i8", "u4"])
def test_long_cache_is_split_and_joined(fmt, width):
    """Few rows over many tokens, with tables for no more than that and for much more."""
    rng = np.random.default_rng(11)
    cache = filled(rng, fmt, 50, 256, 1, 64)
    batch = Batch(cache, [1, 3], [5000, 7001], rng, width=width)
    batch.device()
    assert lb.lowbit_kv_attention_workspace_bytes(cache.handle(256), batch.handle(), 4) > 0
    check(cache, batch, 4, "bf16", rng)
    # two lengths far apart in one call, the short one within one part
    check(cache, Batch(cache, [1, 1, 1], [7001, 3, 66], rng, width=width), 2, "f16", rng)


@pytest.mark.parametrize("fmt", ["i8", "u4"])
def test_results_are_the_same_each_time(fmt):
    rng = np.random.default_rng(12)
    cache = filled(rng, fmt, 40, 128, 2, 128)
    batch = Batch(cache, [1, 5, 90], [2500, 2000, 400], rng)
    q = rows(rng, batch.rows, 8, 128, torch.float16)
    first = check(cache, batch, 4, "f16", rng, q=q)
    for _ in range(3):
        assert torch.equal(first, check(cache, batch, 4, "f16", rng, q=q))


@pytest.mark.parametrize("n", [[1, 1, 1, 1, 3], [40, 1, 50, 33, 20]])
@pytest.mark.parametrize("fmt", ["i8", "u4"])
def test_rows_that_see_nothing(fmt, n):
    """Sequences without tokens, rows before token 0, missing pages everywhere or in the middle, tokens past the table."""
    rng = np.random.default_rng(13)
    cache = filled(rng, fmt, 14, 64, 2, 64)
    batch = Batch(cache, n, [0, 300, 200, 20, 2], rng, width=4)
    batch.table[1, 1] = -1
    batch.table[1, 3] = 14
    batch.table[2, :] = [2 ** 31 - 1, -7, -2 ** 31, 99]
    y = check(cache, batch, 3, "f16", rng)
    assert (y[:batch.offsets[1]] == 0).all() and (y[batch.offsets[2]:batch.offsets[3]] == 0).all()
    batch.lens = [-5, 2 ** 31 - 1, 256, 1, 1]
    for b in range(5):
        batch.table[b] = rng.permutation(14)[:4]
    # a length past the table: its tokens have no page, its rows stand after all that have one
    batch.device()
    q = rows(rng, batch.rows, 4, 64, torch.float16)
    y = attend(cache.handle(cache.device()), batch, q.cuda(), 256, 4, "f16", 0.125, 0, batch.rows, 64)
    batch.lens[0], batch.lens[1] = 0, 256 + n[1]
    want, bound = attention64(cache, batch, q.double().numpy(), 0.125, 0, torch.float16)
    assert_within(y, want, bound)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("fmt", ["i8", "u4"])
def test_what_is_not_seen_does_not_count(fmt, dt):
    """NaN and infinite scales and minima behind the last token, before the window and after a row's own token."""
    rng = np.random.default_rng(14)
    for n, window in (([1, 1], 0), ([1, 1], 70), ([6, 80], 0), ([6, 80], 50)):
        cache = filled(rng, fmt, 12, 64, 2, 64, DT[dt][1])
        batch = Batch(cache, n, [130, 200], rng)
        for b, length in enumerate(batch.lens):
            first = max(0, length - n[b] + 1 - window) if window else 0
            pos = np.array([p for p in range(-(-length // 64) * 64) if p >= length or p < first])
            page, t = batch.where(cache, b, pos)
            for i in range(2):
                for which in range(cache.arrays // 2):
                    cache.meta(i, which)[page, :, t] = np.where(pos % 2 == 0, np.nan, np.inf).astype(np.float32)[:, None]
        y = check(cache, batch, 4, dt, rng, window=window)
        assert torch.isfinite(y).all()
        # the last token's row is NaN: of a chunk, only the last row sees it
        page, t = batch.where(cache, 1, np.array([199]))
        for i in range(2):
            cache.meta(i, 0)[page, :, t] = np.nan
        y = check(cache, batch, 4, dt, rng, window=window)
        assert torch.isnan(y[-1]).all() and torch.isfinite(y[:-1]).all()


@pytest.mark.parametrize("fmt", ["i8", "u4"])
def test_scales_of_all_sizes(fmt):
    """Keys and values whose scales span many powers of two, queries of bf16's whole range."""
    rng = np.random.default_rng(15)
    cache = filled(rng, fmt, 8, 64, 1, 64)
    for n in ([1, 2], [70, 40]):
        batch = Batch(cache, n, [200, 150], rng)
        for i in range(2):
            f = np.ldexp(1.0, rng.integers(-12, 6, (8, 64))).astype(np.float32) if i else 1
            for which in range(cache.arrays // 2):
                cache.meta(i, which)[:, 0, :] *= f
        q = rows(rng, batch.rows, 4, 64, torch.float32).double().numpy()
        for e in (-100, -20, 0, 40, 100):
            x = torch.from_numpy(np.ldexp(q, e)).to(torch.bfloat16)
            check(cache, batch, 4, "bf16", rng, q=x, scale=float(np.ldexp(0.125, -e)), what="2^%d" % e)
        # rows that differ by up to 2^30, and by a little
        for spread in (30, 7):
            x = torch.from_numpy(q * np.ldexp(1.0, -rng.integers(0, spread + 1, (len(q), 1, 1)))).to(torch.bfloat16)
            check(cache, batch, 4, "bf16", rng, q=x, scale=8.0, what="spread %d" % spread)
        q = torch.from_numpy(q).to(torch.float16) * 1024
        check(cache, batch, 4, "f16", rng, q=q, scale=0.125 / 1024)
        q = rows(rng, batch.rows, 4, 64, torch.bfloat16)
        q[0] = 0                                           # every token alike
        q[1, 0, 3] = float("inf")
        wide = q.cuda()
        batch.device()
        y = attend(cache.handle(cache.device()), batch, wide, 256, 4, "bf16", 0.125, 0, batch.rows, 64)
        assert torch.isnan(y[1, 0]).all() and torch.isfinite(y[1, 1:]).all() and torch.isfinite(y[0]).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fmt", ["i8", "u4"])
def test_scales_of_either_sign(fmt, D):
    """A value is code * scale (+ minimum), also where a page that the caller made has a negative scale."""
    rng = np.random.default_rng(26)
    cache = filled(rng, fmt, 12, 64, 1, D)
    for i in range(2):
        cache.meta(i, 0)[:] *= rng.choice(np.array([-1, 1], np.float32), (12, 1, 64))
        cache.meta(i, 0)[3] = -np.abs(cache.meta(i, 0)[3])
    for n in ([1, 2, 0], [33, 90, 1]):
        batch = Batch(cache, n, [200, 230, 64], rng)
        batch.table[0, 1], batch.table[1, 2] = 3, 3                    # a block of negative scales alone
        check(cache, batch, 2, "f16", rng, what=str(n))


@pytest.mark.parametrize("fmt", ["i8", "u4"])
def test_one_token_far_above_the_rest(fmt):
    """A softmax of one token's weight, first, in the middle and last."""
    rng = np.random.default_rng(16)
    cache = filled(rng, fmt, 10, 64, 1, 64)
    batch = Batch(cache, [1, 1, 1], [150, 150, 150], rng)
    q = rows(rng, 3, 2, 64, torch.float16)
    for b, pos in enumerate((0, 70, 149)):
        page, t = batch.where(cache, b, np.array([pos]))
        cache.put(0, page, t, 0, 40 * q[b, 0].float().numpy()[None])
    check(cache, batch, 2, "f16", rng, q=q)


def test_pages_past_4_gib():
    rng = np.random.default_rng(17)
    heads, D = 16, 256
    small = filled(rng, "i8", 4, 256, heads, D)
    pages = (5 << 30) // (heads * small.part)
    data = torch.empty(pages * heads * small.part, dtype=torch.uint8, device="cuda").view(pages, heads, small.part)
    far = np.array([pages - 1, pages - 3, pages // 2, pages - 7], np.int32)
    data[torch.from_numpy(far).cuda().long()] = small.device()
    for n in ([1, 2], [80, 33]):
        batch = Batch(small, n, [500, 300], rng)
        q = rows(rng, batch.rows, heads, D, torch.float16)
        table = batch.table.copy()
        batch.table = np.where(table >= 0, far[table], -1)
        batch.device()
        y = attend(lb.make_kv_cache(data, lb.LOWBIT_KV_I8, pages, 256, heads, D), batch, q.cuda(), heads * D, heads,
                   "f16", 0.0625, 0, batch.rows, D)
        batch.table = table
        want, bound = attention64(small, batch, q.double().numpy(), 0.0625, 0, torch.float16)
        assert_within(y, want, bound)


@pytest.mark.parametrize("fmt", ["i8", "u4"])
def test_step_by_step_and_all_at_once(fmt):
    """A prompt written and attended in one call, in chunks, and token by token: write, attention and read together."""
    rng = np.random.default_rng(18)
    heads, group, D, total, dtype = 2, 4, 64, 150, torch.bfloat16
    Hq = heads * group
    width = (Hq + 2 * heads) * D
    qkv = rows(rng, total, Hq + 2 * heads, D, dtype).cuda()
    outs, caches = [], []
    for chunks in ([150], [64, 1, 1, 84], [100] + [1] * 50):
        cache = Cache(fmt, 4, 64, heads, D)
        data = torch.full(cache.b.shape, 0x77, dtype=torch.uint8, device="cuda")
        at, parts = 0, []
        table = rng.permutation(4)[:3].astype(np.int32)
        for n in chunks:
            batch = Batch(cache, [n], [at + n], rng, width=3)
            batch.table[0] = table
            h = batch.device()
            base = qkv[at:at + n].data_ptr()
            k, v = base + 2 * Hq * D, base + 2 * (Hq + heads) * D
            lb.check(lb.lowbit_kv_write(cache.handle(data), h, k, width, v, width, lb.LOWBIT_BF16))
            parts.append(attend(cache.handle(data), batch, base, width, Hq, "bf16", D ** -0.5, 0, n, D))
            at += n
        whole = Batch(cache, [total], [total], rng, width=3)
        whole.table[0] = table
        k, v = (torch.empty((total, heads, D), dtype=dtype, device="cuda") for _ in range(2))
        lb.check(lb.lowbit_kv_read(cache.handle(data), whole.device(), k, heads * D, v, heads * D, lb.LOWBIT_BF16))
        torch.cuda.synchronize()
        outs.append(torch.cat(parts))
        caches.append((k, v))
        cache.b = data.cpu().numpy()
        want, bound = attention64(cache, whole, qkv[:, :Hq].double().cpu().numpy(), float(np.float32(D ** -0.5)), 0,
                                  dtype)
        assert_within(outs[-1], want, bound)
    for k, v in caches[1:]:
        assert torch.equal(k, caches[0][0]) and torch.equal(v, caches[0][1])


@pytest.mark.parametrize("fmt", ["i8", "u4"])
def test_graph_replays_with_new_lengths(fmt):
    """A captured decode step (write, attention); lengths and pages change between replays, eager calls between."""
    rng = np.random.default_rng(19)
    heads, group, D, B, width = 2, 2, 128, 3, 40
    Hq = heads * group
    cache = filled(rng, fmt, 3 * width, 64, heads, D)
    data = cache.device()
    batch = Batch(cache, [1] * B, [1000, 70, 2000], rng, width=width)
    handle = batch.device()
    q, k, v = (torch.zeros((B, h, D), dtype=torch.float16, device="cuda") for h in (Hq, heads, heads))
    y = torch.zeros((B, Hq, D), dtype=torch.float16, device="cuda")
    need = lb.lowbit_kv_attention_workspace_bytes(cache.handle(data), handle, Hq)
    assert need > 0
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")

    def call(st):
        lb.check(lb.lowbit_kv_write(cache.handle(data), handle, k, heads * D, v, heads * D, lb.LOWBIT_F16, st))
        lb.check(lb.lowbit_kv_attention(cache.handle(data), handle, q, Hq * D, Hq, lb.LOWBIT_F16, 0.08, 0, y, ws, need,
                                        st))

    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            call(stream.cuda_stream)
    for turn in range(5):
        new = Batch(cache, [1] * B, [int(x) for x in rng.integers(1, 2400, B)], rng, width=width)
        for d, a in zip(batch.d, (new.table, new.lens, new.offsets)):
            d.copy_(torch.from_numpy(np.ascontiguousarray(a, np.int32)))
        q.copy_(rows(rng, B, Hq, D, torch.float16))
        k.copy_(rows(rng, B, heads, D, torch.float16))
        v.copy_(rows(rng, B, heads, D, torch.float16))
        y.fill_(float("nan"))
        torch.cuda.synchronize()
        if turn % 2:
            call(None)
        else:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        cache.b = data.cpu().numpy()
        want, bound = attention64(cache, new, q.double().cpu().numpy(), float(np.float32(0.08)), 0, torch.float16)
        assert_within(y, want, bound, "turn %d" % turn)


def test_calls_on_several_streams():
    """The same cache read by calls on four streams, each with its own workspace and output."""
    rng = np.random.default_rng(20)
    cache = filled(rng, "i8", 60, 64, 1, 128)
    data = cache.device()
    jobs = []
    for i in range(4):
        batch = Batch(cache, [1, 30 * i + 1], [1500, 1800], rng)
        q = rows(rng, batch.rows, 4, 128, torch.float16)
        jobs.append([batch, q, q.cuda(), batch.device(), torch.cuda.Stream()])
    for job in jobs:
        need = lb.lowbit_kv_attention_workspace_bytes(cache.handle(data), job[3], 4)
        job += [torch.zeros(max(need, 1), dtype=torch.uint8, device="cuda"),
                torch.zeros((job[0].rows, 4, 128), dtype=torch.float16, device="cuda"), need]
    torch.cuda.synchronize()
    for _ in range(5):
        for batch, q, qd, h, st, ws, y, need in jobs:
            lb.check(lb.lowbit_kv_attention(cache.handle(data), h, qd, 512, 4, lb.LOWBIT_F16, 0.09, 0, y, ws, need,
                                            st.cuda_stream))
    torch.cuda.synchronize()
    for batch, q, qd, h, st, ws, y, need in jobs:
        want, bound = attention64(cache, batch, q.double().numpy(), float(np.float32(0.09)), 0, torch.float16)
        assert_within(y, want, bound)


def test_pages_shared_between_sequences():
    """A prefix that several sequences read."""
    rng = np.random.default_rng(21)
    cache = filled(rng, "u4", 10, 64, 2, 64)
    batch = Batch(cache, [1, 3, 20], [100, 140, 200], rng)
    batch.table[1, :2] = batch.table[0, :2]
    batch.table[2, 0] = batch.table[0, 0]
    check(cache, batch, 4, "bf16", rng)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fmt", ["i8", "u4"])
def test_nan_of_no_weight(fmt, D):
    """A row that sees a token of NaN is NaN, whatever that token weighs and wherever it lies beside those that do."""
    rng = np.random.default_rng(27)
    cache = filled(rng, fmt, 50 if D == 64 else 12, 64, 1, D)
    q = torch.ones((200, 1, D), dtype=torch.float16)
    for length, n in ((300, 1), (300, 90)) + (((3000, 1), (3000, 90)) if D == 64 else ()):
        batch = Batch(cache, [n], [length], rng)
        for at, which in ((10, 0), (70, 0), (150, 0), (length - n, 0)) + (((130, 1),) if fmt == "u4" else ()):
            for heavy in (0, 100, 200):
                b = cache.b.copy()
                cache.put(0, *batch.where(cache, 0, np.array([heavy])), 0, np.full((1, D), 120 / D ** 0.5, np.float32))
                page, t = batch.where(cache, 0, np.array([at]))
                cache.put(0, page, t, 0, np.full((1, D), -120 / D ** 0.5, np.float32))
                cache.meta(1, which)[page, 0, t] = np.nan
                y = check(cache, batch, 1, "f16", rng, q=q[:n])
                assert torch.isnan(y).all(), (length, n, at, which, heavy)
                cache.b = b


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("fmt", ["i8", "u4"])
def test_queries_that_are_not_finite(fmt, dt):
    """A row whose query holds an infinity or a NaN is NaN, of whatever sign its scores are; other rows are not touched."""
    rng = np.random.default_rng(28)
    D, dtype = 64, DT[dt][1]
    for n, length in ((3, 100), (60, 200)):
        cache = filled(rng, fmt, 4, 64, 1, D)
        batch = Batch(cache, [n], [length], rng)
        page, t = batch.where(cache, 0, np.arange(length))
        cache.put(0, page, t, 0, rng.uniform(0.5, 1.5, (length, D)).astype(np.float32))     # keys above zero
        batch.device()
        data = cache.device()
        for value in (float("-inf"), float("inf"), float("nan")):
            q = rows(rng, n, 2, D, dtype).abs()
            q[n // 2, 1, 5] = value
            y = attend(cache.handle(data), batch, q.cuda(), 2 * D, 2, dt, 0.125, 0, n, D)
            bad = torch.zeros((n, 2), dtype=torch.bool)
            bad[n // 2, 1] = True
            assert torch.isnan(y[bad]).all() and torch.isfinite(y[~bad]).all(), (n, value)


@pytest.mark.parametrize("heads,group", [(1, 1), (1, 64), (5, 3), (7, 1), (16, 2), (32, 1)])
def test_head_layouts(heads, group):
    rng = np.random.default_rng(heads * 100 + group)
    cache = filled(rng, "i8", 5, 64, heads, 64)
    for n in ([1, 1], [40, 2]):
        check(cache, Batch(cache, n, [100, 130], rng), group, "f16", rng, what=str(n))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fmt", ["i8", "u4"])
def test_chunks_over_a_long_cache(fmt, D):
    """Tiles cut into a few pieces and into many, beside sequences of few rows that are cut as well."""
    rng = np.random.default_rng(22)
    cache = filled(rng, fmt, 32, 256, 1, D)
    check(cache, Batch(cache, [130], [1300], rng), 1, "f16", rng, what="few pieces")
    check(cache, Batch(cache, [130, 1, 3, 0, 9], [4000, 2000, 700, 50, 200], rng), 2, "bf16", rng, what="many pieces")
    check(cache, Batch(cache, [1, 40, 40], [1500, 2500, 3000], rng), 3, "f16", rng, window=1000, what="window")


def many(cache, rng, B, longest, width):
    """B sequences of few rows whose pages are any of the cache's."""
    batch = Batch(cache, [int(x) for x in rng.integers(0, 3, B)], [0] * B, rng, width=width)
    batch.lens = [int(x) for x in rng.integers(1, longest, B)]
    batch.table = rng.integers(0, cache.pages, (B, width)).astype(np.int32)
    return batch


@pytest.mark.parametrize("B", [63, 64, 65, 511, 513])
def test_many_sequences(B):
    rng = np.random.default_rng(23)
    cache = filled(rng, "i8", 20, 64, 1, 64)
    check(cache, many(cache, rng, B, 1500 if B < 100 else 300, 24), 2, "bf16", rng)


def test_offsets_that_go_back():
    """Sequences that name the same rows again and again: nothing past the workspace or the rows is written."""
    rng = np.random.default_rng(24)
    cache = filled(rng, "i8", 20, 64, 1, 128)
    B, rows_, Hq, D = 100, 150, 2, 128
    batch = many(cache, rng, B, 1500, 24)
    batch.rows, batch.max_rows = rows_, rows_
    batch.offsets = np.where(np.arange(B + 1) % 2 == 0, 0, rows_).astype(np.int32)
    handle = batch.device()
    q = rows(rng, rows_, Hq, D, torch.bfloat16).cuda()
    ch = cache.handle(cache.device())
    need = lb.lowbit_kv_attention_workspace_bytes(ch, handle, Hq)
    ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    y = torch.full((rows_ + 8, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lb.check(lb.lowbit_kv_attention(ch, handle, q, Hq * D, Hq, lb.LOWBIT_BF16, 0.1, 0, y, ws, need))
    torch.cuda.synchronize()
    assert (ws[need:] == 0x5A).all() and (y[rows_:] == 7).all()


@pytest.mark.parametrize("B", [13, 14, 16, 31])
def test_one_long_sequence_among_tiles(B):
    """A tile over many tokens is cut, whatever the number of short ones beside it."""
    rng = np.random.default_rng(29)
    heads, D, n, dtype = 32, 256, 20, torch.bfloat16                  # 8 workgroups a head are resident
    cache = filled(rng, "i8", 3, 256, heads, D)
    batch = Batch(cache, [n] * B, [0] * B, rng, width=16)
    batch.lens = [4096] + [130] * (B - 1)
    batch.table = rng.integers(0, cache.pages, (B, 16)).astype(np.int32)
    handle, ch = batch.device(), cache.handle(cache.device())
    q = rows(rng, batch.rows, heads, D, dtype)
    need = lb.lowbit_kv_attention_workspace_bytes(ch, handle, heads)
    ws = torch.full((need,), 0x5A, dtype=torch.uint8, device="cuda")
    y = torch.zeros((batch.rows, heads, D), dtype=dtype, device="cuda")
    lb.check(lb.lowbit_kv_attention(ch, handle, q.cuda(), heads * D, heads, lb.LOWBIT_BF16, 0.1, 0, y, ws, need))
    torch.cuda.synchronize()
    # results of at least two pieces of 20 rows of every head
    assert (ws != 0x5A).sum().item() > 2 * heads * n * D * 4 * 0.9
    first = Batch(cache, [n] * 2, [0] * 2, rng, width=16)            # the long one and one of the others
    first.lens, first.table = batch.lens[:2], batch.table[:2]
    want, bound = attention64(cache, first, q[:2 * n].double().numpy(), float(np.float32(0.1)), 0, dtype)
    assert_within(y[:2 * n], want, bound)


@pytest.mark.parametrize("n", [[1], [40], [130], [1, 3, 70], [130, 20, 40]])
@pytest.mark.parametrize("D", [64, 256])
def test_nothing_behind_the_workspace_is_written(D, n):
    """Workspaces of tables that are short enough to limit the pieces, filled as far as they are asked for."""
    rng = np.random.default_rng(30)
    cache = filled(rng, "i8", 12, 64, 2, D)
    for blocks in (17, 20, 24, 33, 70):
        batch = Batch(cache, n, [0] * len(n), rng, width=blocks)
        batch.lens = [64 * blocks - 7 * b for b in range(len(n))]
        batch.table = rng.integers(0, cache.pages, (len(n), blocks)).astype(np.int32)
        handle, ch, q = batch.device(), cache.handle(cache.device()), rows(rng, batch.rows, 4, D, torch.float16)
        need = lb.lowbit_kv_attention_workspace_bytes(ch, handle, 4)
        assert need > 0
        ws = torch.full((need + 65536,), 0x5A, dtype=torch.uint8, device="cuda")
        y = torch.zeros((batch.rows, 4, D), dtype=torch.float16, device="cuda")
        lb.check(lb.lowbit_kv_attention(ch, handle, q.cuda(), 4 * D, 4, lb.LOWBIT_F16, 0.06, 0, y, ws, need))
        torch.cuda.synchronize()
        assert (ws[need:] == 0x5A).all(), blocks
        want, bound = attention64(cache, batch, q.double().numpy(), float(np.float32(0.06)), 0, torch.float16)
        assert_within(y, want, bound, "%d blocks" % blocks)


def test_graphs_that_share_a_workspace():
    """A chunk's graph and a decode step's, captured without a call before them, replayed in turn on one workspace."""
    rng = np.random.default_rng(25)
    heads, group, D = 2, 2, 256
    Hq = heads * group
    cache = filled(rng, "u4", 30, 128, heads, D)
    data = cache.device()
    stream, jobs = torch.cuda.Stream(), []
    for n, lens in (([90, 1], [1500, 1100]), ([1, 1], [1200, 2000])):
        batch = Batch(cache, n, lens, rng)
        q = rows(rng, batch.rows, Hq, D, torch.float16)
        jobs.append((batch, q, q.cuda(), batch.device(), torch.cuda.CUDAGraph(),
                     torch.zeros((batch.rows, Hq, D), dtype=torch.float16, device="cuda")))
    need = max(lb.lowbit_kv_attention_workspace_bytes(cache.handle(data), job[3], Hq) for job in jobs)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for batch, q, qd, h, graph, y in jobs:
            with torch.cuda.graph(graph, stream=stream):
                lb.check(lb.lowbit_kv_attention(cache.handle(data), h, qd, Hq * D, Hq, lb.LOWBIT_F16, 0.06, 0, y, ws, need,
                                                stream.cuda_stream))
        for turn in range(3):
            for job in jobs:
                job[5].fill_(float("nan"))
            for job in jobs:
                job[4].replay()
            torch.cuda.synchronize()
            for batch, q, qd, h, graph, y in jobs:
                want, bound = attention64(cache, batch, q.double().numpy(), float(np.float32(0.06)), 0, torch.float16)
                assert_within(y, want, bound, "turn %d" % turn)
                eager = attend(cache.handle(data), batch, qd, Hq * D, Hq, "f16", 0.06, 0, batch.rows, D)
                assert torch.equal(eager, y)
