"""Host-side checks (CPU only) of the key/value cache's entry points: every
refusal comes back as a status code before anything is enqueued, and empty
calls return OK without touching memory."""
import math

import pytest

import bit_weight_only_pack_amd as lb

OK, ARG, UNS, WS = lb.LOWBIT_OK, lb.LOWBIT_E_INVALID_ARG, lb.LOWBIT_E_UNSUPPORTED, lb.LOWBIT_E_WORKSPACE
FAKE = 1 << 20  # a non-null address that must never be dereferenced on these paths
I8, U4 = lb.LOWBIT_KV_I8, lb.LOWBIT_KV_U4


def cache(data=FAKE, fmt=I8, pages=8, page_size=64, heads=4, dim=128):
    return lb.make_kv_cache(data, fmt, pages, page_size, heads, dim)


def batch(table=FAKE, width=4, lens=FAKE, offs=FAKE, count=2, rows=6, most=3):
    return lb.make_kv_batch(table, width, lens, offs, count, rows, most)


def write(c=None, b=None, k=FAKE, ks=512, v=FAKE, vs=512, dt=0, call=None, **kw):
    bk = {n: kw.pop(n) for n in ("table", "width", "lens", "offs", "count", "rows", "most") if n in kw}
    return (call or lb.lowbit_kv_write)(c or cache(**kw), b or batch(**bk), k, ks, v, vs, dt)


def attention(c=None, b=None, q=FAKE, qs=1024, Hq=8, dt=0, scale=0.1, window=0, y=FAKE, ws=FAKE, nb=1 << 40, **kw):
    bk = {n: kw.pop(n) for n in ("table", "width", "lens", "offs", "count", "rows", "most") if n in kw}
    return lb.lowbit_kv_attention(c or cache(**kw), b or batch(**bk), q, qs, Hq, dt, scale, window, y, ws, nb)


def test_page_bytes():
    for page in (64, 128, 256):
        for dim in (64, 128, 256):
            assert lb.lowbit_kv_page_bytes(I8, page, 3, dim) == 3 * page * (2 * dim + 8)
            assert lb.lowbit_kv_page_bytes(U4, page, 3, dim) == 3 * page * (dim + 16)
    for bad in ((2, 64, 1, 64), (-1, 64, 1, 64), (I8, 32, 1, 64), (I8, 96, 1, 64), (I8, 64, 0, 64), (I8, 64, -1, 64),
                (I8, 64, 1, 32), (I8, 64, 1, 96), (I8, 64, 1 << 15, 64)):
        assert lb.lowbit_kv_page_bytes(*bad) == 0


@pytest.mark.parametrize("call", [write, lambda **kw: write(call=lb.lowbit_kv_read, **kw), attention])
def test_shared_refusals(call):
    assert call(pages=-1) == ARG and call(heads=0) == ARG and call(width=-1) == ARG
    assert call(count=-1) == ARG and call(rows=-1) == ARG and call(most=-1) == ARG
    assert call(fmt=2) == UNS and call(page_size=32) == UNS and call(page_size=0) == UNS and call(dim=96) == UNS
    assert call(width=1 << 25) == UNS                              # positions past 2^30
    assert call(count=1 << 24) == UNS and call(heads=1 << 15) in (UNS, ARG)
    for name in ("table", "lens", "offs", "data"):
        assert call(**{name: None}) == ARG, name
        assert call(**{name: FAKE + 2}) == ARG, name
    assert call(data=FAKE + 128) == ARG                            # 256-byte aligned
    assert call(dt=2) == UNS and call(dt=-1) == UNS
    assert call(count=1 << 20, rows=1 << 30, most=1 << 20) == UNS  # more workgroups than a grid takes


def test_null_structs():
    c, b = cache(), batch()
    for x, y in ((None, b), (c, None)):
        assert lb.lowbit_kv_write(x, y, FAKE, 512, FAKE, 512, 0) == ARG
        assert lb.lowbit_kv_read(x, y, FAKE, 512, FAKE, 512, 0) == ARG
        assert lb.lowbit_kv_attention(x, y, FAKE, 1024, 8, 0, 0.1, 0, FAKE) == ARG
        assert lb.lowbit_kv_attention_workspace_bytes(x, y, 8) == 0


@pytest.mark.parametrize("call", [lb.lowbit_kv_write, lb.lowbit_kv_read])
def test_row_refusals(call):
    for kw in (dict(k=None), dict(v=None), dict(k=FAKE + 8), dict(v=FAKE + 2), dict(ks=504), dict(vs=511), dict(ks=516),
               dict(ks=-512), dict(ks=0)):
        assert write(call=call, **kw) == ARG, kw
    for kw in (dict(count=0), dict(rows=0), dict(most=0)):
        assert write(call=call, k=None, v=None, table=None, lens=None, offs=None, data=None, **kw) == OK, kw


def test_attention_refusals():
    for kw in (dict(q=None), dict(y=None), dict(q=FAKE + 8), dict(y=FAKE + 8), dict(qs=1016), dict(qs=1028), dict(Hq=0),
               dict(Hq=-4), dict(Hq=6), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan),
               dict(window=-1)):
        assert attention(**kw) == ARG, kw
    assert attention(Hq=1 << 15, qs=1 << 22) == UNS
    for kw in (dict(count=0), dict(rows=0), dict(most=0)):
        assert attention(q=None, y=None, table=None, lens=None, offs=None, data=None, ws=None, nb=0, **kw) == OK, kw


def test_attention_workspace_is_checked():
    seen = 0
    for count, most, width, dim in ((1, 1, 64, 128), (1, 5, 2048, 64), (4, 1, 512, 256), (2, 300, 512, 128)):
        b, c = batch(count=count, rows=count * most, most=most, width=width), cache(dim=dim)
        nb = lb.lowbit_kv_attention_workspace_bytes(c, b, 8)
        assert nb <= 1 << 28
        if nb:
            seen += 1
            args = dict(c=c, b=b, qs=8 * dim)
            assert attention(**args, ws=None, nb=0) == WS and attention(**args, nb=nb - 1) == WS
            assert attention(**args, ws=FAKE + 128, nb=nb) == ARG
    assert seen
    for kw in (dict(dim=96), dict(page_size=16), dict(heads=0)):
        assert lb.lowbit_kv_attention_workspace_bytes(cache(**kw), batch(), 8) == 0
    for Hq in (0, -8, 6, 1 << 15):
        assert lb.lowbit_kv_attention_workspace_bytes(cache(), batch(), Hq) == 0
    for kw in (dict(count=0), dict(rows=0), dict(most=0), dict(count=-1), dict(width=1 << 25)):
        assert lb.lowbit_kv_attention_workspace_bytes(cache(), batch(**kw), 8) == 0


def test_attention_workspace_is_known_before_the_buffers():
    """The query takes the sizes alone: any pointer may be missing, or not be one yet."""
    seen = 0
    for count, most, width, dim in ((1, 1, 64, 128), (1, 5, 2048, 64), (4, 1, 512, 256), (2, 300, 512, 128), (3, 2, 1, 64)):
        sizes = dict(count=count, rows=count * most, most=most, width=width)
        nb = lb.lowbit_kv_attention_workspace_bytes(cache(dim=dim), batch(**sizes), 8)
        seen += nb > 0
        none = dict(table=None, lens=None, offs=None)
        assert lb.lowbit_kv_attention_workspace_bytes(cache(data=None, dim=dim), batch(**sizes, **none), 8) == nb
        assert lb.lowbit_kv_attention_workspace_bytes(cache(data=FAKE + 8, dim=dim), batch(**sizes), 8) == nb
        for name in none:
            assert lb.lowbit_kv_attention_workspace_bytes(cache(dim=dim), batch(**sizes, **{name: None}), 8) == nb
    assert seen >= 3


def test_attention_workspace_is_for_pieces_that_there_can_be():
    """A piece is 4 blocks of 64 tokens or more: a short table makes few of them, whatever the compute units could take."""
    for dim, rows, group in ((128, 40, 1), (64, 70, 2), (256, 20, 1), (64, 3, 4), (128, 5, 2)):
        for heads in (1, 8, 512):
            for count in (1, 3):
                for blocks in (17, 18, 40, 1000, 5000):
                    b = batch(count=count, rows=rows * count, most=rows, width=blocks)
                    nb = lb.lowbit_kv_attention_workspace_bytes(cache(dim=dim, heads=heads), b, heads * group)
                    items = count * -(-rows * group // 16)               # of the narrowest kind
                    one = heads * (128 if rows * group > 64 else 64) * (dim * 4 + 8)
                    assert 0 < nb <= 2 * (items * -(-blocks // 4) * one + 1025 * 16), (dim, heads, count, blocks, nb)
