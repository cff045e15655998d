"""GPU parity of the sorting of tokens by expert and back, through the C ABI:
the index exactly by its definition, permuted rows byte for byte, sums and
gradients against 64-bit evaluations (bounds: the rounding to the output type
plus one binary32 rounding per term) and against differences, which are exact
on inputs of small whole numbers."""
import numpy as np
import pytest
import torch

import bit_weight_only_pack_amd as lb
from gpu_util import dev
from w8a8_util import DT, U32, assert_rounded, gpu_sort, routing, sort64

pytestmark = pytest.mark.gpu


def _map(rng, E, El):
    m = np.full(E, -1, np.int32)
    m[rng.permutation(E)[:El]] = rng.permutation(El)
    return m


# ---------------------------------------------------------------- index
@pytest.mark.parametrize("T,top_k,E,El", [
    (1, 1, 1, 1), (1, 8, 128, 128), (3, 2, 5, 5), (37, 8, 128, 128), (64, 1, 2, 2), (129, 6, 1024, 1024),
    (1000, 8, 60, 17), (1024, 8, 128, 128), (1025, 8, 128, 128),      # the last size of one workgroup, and one more
    (5000, 7, 1000, 333), (16384, 8, 128, 128), (70001, 9, 3, 2), (9000, 1, 1024, 1024),
    (200, 5, 900, 801), (150000, 8, 40, 40),                          # past the slots that stay in registers
])
def test_sort_bitexact(T, top_k, E, El):
    rng = np.random.default_rng(T + E)
    ids = routing(rng, T, E, top_k) if E >= top_k else rng.integers(0, E, (T, top_k)).astype(np.int32)
    emap = _map(rng, E, El) if El < E else None
    got = gpu_sort(ids, E, emap, El)
    for g, want, what in zip(got, sort64(ids, E, emap, El), ("row_slot", "slot_row", "offsets")):
        assert np.array_equal(g.cpu().numpy(), want), what


@pytest.mark.parametrize("T", [50, 6000])
def test_sort_odd_ids(T):
    """The same expert twice for a token, ids outside the range, maps that point outside, everything dropped."""
    rng = np.random.default_rng(T)
    E, El, top_k = 20, 9, 4
    ids = rng.integers(-3, E + 3, (T, top_k)).astype(np.int32)
    ids[::5] = 7
    ids[1::50] = np.array([2 ** 31 - 1, -2 ** 31, E, -1], np.int32)
    emap = rng.integers(-4, El + 4, E).astype(np.int32)
    for m, el in ((emap, El), (None, El), (np.full(E, -1, np.int32), El), (None, E)):
        for g, want in zip(gpu_sort(ids, E, m, el), sort64(ids, E, m, el)):
            assert np.array_equal(g.cpu().numpy(), want)
    same = np.full((T, top_k), 3, np.int32)
    for g, want in zip(gpu_sort(same, E, None, E), sort64(same, E, None, E)):
        assert np.array_equal(g.cpu().numpy(), want)


@pytest.mark.parametrize("T,top_k", [(0, 4), (5, 0)])
def test_sort_without_slots_writes_offsets(T, top_k):
    _, _, offs = gpu_sort(np.zeros((T, top_k), np.int32), 6, None, 6)
    assert offs.cpu().tolist() == [0] * 7


# ---------------------------------------------------------------- permute
def _case(T, top_k, E, El, seed=0):
    rng = np.random.default_rng(seed + T)
    ids = routing(rng, T, E, top_k)
    emap = _map(rng, E, El) if El < E else None
    rs, sr, of = sort64(ids, E, emap, El)
    return rng, rs, sr, int(of[-1])


@pytest.mark.parametrize("T,top_k,E,El", [(1, 1, 1, 1), (1, 8, 16, 16), (33, 3, 8, 3), (700, 2, 8, 8), (40, 17, 40, 33)])
@pytest.mark.parametrize("row_bytes", [0, 8, 16, 24, 264, 2048, 4096, 6160, 40960])
def test_permute_bytes(T, top_k, E, El, row_bytes):
    rng, rs, sr, n = _case(T, top_k, E, El, row_bytes)
    x = rng.integers(0, 256, (T, row_bytes)).astype(np.uint8)
    scale = rng.random(T).astype(np.float32)
    S = T * top_k
    for scaled in (True, False):
        xp = torch.full((S + 1, row_bytes), 0x5A, dtype=torch.uint8, device="cuda")
        ps = torch.full((S + 1,), -3.0, device="cuda")
        lb.check(lb.lowbit_moe_permute(dev(x), dev(scale) if scaled else None, T, top_k, row_bytes, dev(sr), xp,
                                       ps if scaled else None))
        torch.cuda.synchronize()
        assert np.array_equal(xp[:n].cpu().numpy(), x[rs[:n] // top_k])
        assert bool((xp[n:] == 0x5A).all())
        if scaled:
            assert np.array_equal(ps[:n].cpu().numpy(), scale[rs[:n] // top_k])
        assert bool((ps[n if scaled else 0:] == -3).all())


# ---------------------------------------------------------------- unpermute
def unpermute64(yp, w, sr, T, top_k):
    y, mag = np.zeros((T, yp.shape[1])), np.zeros((T, yp.shape[1]))
    for j in range(top_k):
        r = sr.reshape(T, top_k)[:, j]
        has = r >= 0
        term = (1.0 if w is None else w[has, j].astype(np.float64)[:, None]) * yp[r[has]]
        y[has] += term
        mag[has] += np.abs(term)
    return y, (top_k + 1) * U32 * mag


def _rows(rng, n, H, dtype):
    return torch.from_numpy(rng.standard_normal((n, H))).to(dtype)


@pytest.mark.parametrize("T,top_k,E,El,H", [
    (1, 1, 1, 1, 8), (1, 8, 16, 16, 2048), (5, 3, 8, 2, 24), (33, 8, 128, 96, 264), (200, 2, 8, 8, 4096),
    (64, 10, 16, 16, 1032), (17, 17, 40, 33, 8200),
])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("weighted", [True, False])
def test_unpermute_parity(T, top_k, E, El, H, dt, weighted):
    code, dtype = DT[dt]
    rng, rs, sr, n = _case(T, top_k, E, El, H)
    yp = _rows(rng, T * top_k, H, dtype)
    yp[n:] = float("nan")                            # no slot names these
    w = rng.standard_normal((T, top_k)).astype(np.float32) if weighted else None
    y64, step = unpermute64(np.nan_to_num(yp.to(torch.float64).numpy()), w, sr, T, top_k)
    if weighted:
        w[sr.reshape(T, top_k) < 0] = np.nan         # and no row has these
    whole = torch.full((T * H + 64,), 3.0, dtype=dtype, device="cuda")
    y = whole[:T * H].view(T, H)
    lb.check(lb.lowbit_moe_unpermute(yp.cuda(), code, None if w is None else dev(w), T, top_k, H, dev(sr), y))
    torch.cuda.synchronize()
    assert_rounded(y, y64, step, dtype)
    assert bool((whole[T * H:] == 3).all())


def test_unpermute_without_rows_gives_zeros():
    T, top_k, H = 9, 2, 64
    y = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    yp = torch.full((T * top_k, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    none = torch.full((T * top_k,), -1, dtype=torch.int32, device="cuda")
    lb.check(lb.lowbit_moe_unpermute(yp, lb.LOWBIT_BF16, None, T, top_k, H, none, y))
    torch.cuda.synchronize()
    assert bool((y == 0).all())
    y.fill_(float("nan"))
    lb.check(lb.lowbit_moe_unpermute(None, lb.LOWBIT_BF16, None, T, 0, H, None, y))
    torch.cuda.synchronize()
    assert bool((y == 0).all())


def test_infinities_stay_in_their_token():
    T, top_k, H = 6, 2, 16
    rng, rs, sr, n = _case(T, top_k, 4, 4)
    yp = _rows(rng, T * top_k, H, torch.float16)
    r = sr.reshape(T, top_k)
    yp[r[2, 0], 3], yp[r[4, 1], 5] = float("inf"), float("nan")
    y = torch.zeros((T, H), dtype=torch.float16, device="cuda")
    lb.check(lb.lowbit_moe_unpermute(yp.cuda(), lb.LOWBIT_F16, None, T, top_k, H, dev(sr), y))
    torch.cuda.synchronize()
    bad = ~torch.isfinite(y.cpu())
    assert bad.nonzero().tolist() == [[2, 3], [4, 5]]


# ---------------------------------------------------------------- gradient
def run_backward(dy, yp, code, w, T, top_k, H, sr, dyp):
    dw = torch.full((T, top_k), float("nan"), device="cuda")
    lb.check(lb.lowbit_moe_unpermute_backward(dy, yp, code, dev(w), T, top_k, H, dev(sr), dyp, dw))
    torch.cuda.synchronize()
    return dw


@pytest.mark.parametrize("T,top_k,E,El,H", [
    (1, 1, 1, 1, 8), (1, 8, 16, 16, 2048), (5, 3, 8, 2, 24), (33, 8, 128, 96, 264), (200, 2, 8, 8, 4096),
    (64, 10, 16, 16, 1032), (17, 17, 40, 33, 8200), (900, 1, 4, 4, 512),
])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_unpermute_backward_parity(T, top_k, E, El, H, dt):
    code, dtype = DT[dt]
    rng, rs, sr, n = _case(T, top_k, E, El, H + 1)
    S = T * top_k
    yp, dy = _rows(rng, S, H, dtype), _rows(rng, T, H, dtype)
    w = rng.standard_normal((T, top_k)).astype(np.float32)
    dyp = torch.full((S, H), 3.0, dtype=dtype, device="cuda")
    dw = run_backward(dy.cuda(), yp.cuda(), code, w, T, top_k, H, sr, dyp)
    g64, y64 = dy.to(torch.float64).numpy(), yp.to(torch.float64).numpy()
    r = rs[:n]
    want = w.reshape(-1)[r].astype(np.float64)[:, None] * g64[r // top_k]
    assert_rounded(dyp[:n], want, U32 * np.abs(want), dtype, "rows")
    assert bool((dyp[n:] == 3).all())
    prod = g64[r // top_k] * y64[:n]
    dots, bound = np.zeros(S), np.zeros(S)
    dots[r], bound[r] = prod.sum(1), (H + 1) * U32 * np.abs(prod).sum(1)      # one rounding per term, any order
    assert np.all(np.abs(dw.cpu().to(torch.float64).numpy().reshape(-1) - dots) <= bound)
    # in place: the rows' gradient over the rows
    over = yp.cuda()
    again = run_backward(dy.cuda(), over, code, w, T, top_k, H, sr, over)
    assert torch.equal(over[:n].view(torch.int16), dyp[:n].view(torch.int16)) and torch.equal(again, dw)


def test_gradients_equal_differences():
    """Whole numbers small enough that every product and sum is exact: (L(p + d) - L(p - d)) / 2d is the gradient
    itself, for L = sum(g * unpermute(yp, w)) in w and yp and for L = sum(g * permute(x)) in x."""
    T, top_k, E, El, H = 7, 3, 6, 4, 24
    rng, rs, sr, n = _case(T, top_k, E, El)
    S = T * top_k
    yp = rng.integers(-3, 4, (S, H)).astype(np.float16)
    w = (rng.integers(-8, 9, (T, top_k)) / 4).astype(np.float32)
    g = rng.integers(-3, 4, (T, H)).astype(np.float16)

    def loss(yp_, w_):
        y = torch.zeros((T, H), dtype=torch.float16, device="cuda")
        lb.check(lb.lowbit_moe_unpermute(dev(yp_), lb.LOWBIT_F16, dev(w_), T, top_k, H, dev(sr), y))
        torch.cuda.synchronize()
        return float((y.cpu().double() * torch.from_numpy(g).double()).sum())

    dyp = torch.zeros((S, H), dtype=torch.float16, device="cuda")
    dw = run_backward(dev(g), dev(yp), lb.LOWBIT_F16, w, T, top_k, H, sr, dyp).cpu().numpy()
    for t in range(T):
        for j in range(top_k):
            up, dn = w.copy(), w.copy()
            up[t, j] += 0.25
            dn[t, j] -= 0.25
            assert (loss(yp, up) - loss(yp, dn)) / 0.5 == dw[t, j]
    for _ in range(40):
        r, h = rng.integers(0, S), rng.integers(0, H)
        up, dn = yp.copy(), yp.copy()
        up[r, h] += 1
        dn[r, h] -= 1
        assert (loss(up, w) - loss(dn, w)) / 2 == float(dyp[r, h])

    x = rng.integers(-3, 4, (T, H)).astype(np.float16)
    gp = rng.integers(-3, 4, (S, H)).astype(np.float16)

    def loss_x(x_):
        xp = torch.zeros((S, H), dtype=torch.float16, device="cuda")
        lb.check(lb.lowbit_moe_permute(dev(x_), None, T, top_k, 2 * H, dev(sr), xp, None))
        torch.cuda.synchronize()
        return float((xp.cpu().double() * torch.from_numpy(gp).double()).sum())

    dx = torch.zeros((T, H), dtype=torch.float16, device="cuda")
    lb.check(lb.lowbit_moe_unpermute(dev(gp), lb.LOWBIT_F16, None, T, top_k, H, dev(sr), dx))
    torch.cuda.synchronize()
    for _ in range(60):
        t, h = rng.integers(0, T), rng.integers(0, H)
        up, dn = x.copy(), x.copy()
        up[t, h] += 1
        dn[t, h] -= 1
        assert (loss_x(up) - loss_x(dn)) / 2 == float(dx[t, h])


def test_rows_past_2_31_bytes():
    """T * top_k * H * 2 bytes past 2^31: the last slots' rows."""
    T, top_k, H = 140000, 8, 1024
    S = T * top_k
    sr = torch.arange(S - 1, -1, -1, dtype=torch.int32, device="cuda")        # slot s in row S - 1 - s
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    xp = torch.zeros((S, H), dtype=torch.bfloat16, device="cuda")
    lb.check(lb.lowbit_moe_permute(x, None, T, top_k, 2 * H, sr, xp, None))
    y = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    lb.check(lb.lowbit_moe_unpermute(xp, lb.LOWBIT_BF16, None, T, top_k, H, sr, y))
    torch.cuda.synchronize()
    assert torch.equal(xp.view(T, top_k, H)[:, 0].flip(0), x) and torch.equal(xp.view(T, top_k, H)[:, 7].flip(0), x)
    assert torch.equal(y, (x.float() * 8).to(torch.bfloat16))
    w = torch.full((T, top_k), 0.5, device="cuda")
    dw = torch.zeros((T, top_k), device="cuda")
    dyp = torch.zeros_like(xp)
    lb.check(lb.lowbit_moe_unpermute_backward(y, xp, lb.LOWBIT_BF16, w, T, top_k, H, sr, dyp, dw))
    torch.cuda.synchronize()
    assert torch.equal(dyp.view(T, top_k, H)[:, 3].flip(0), (y.float() * 0.5).to(torch.bfloat16))
    for t in (0, T - 1):
        want = float((y[t].double() * x[t].double()).sum())
        assert abs(float(dw[t, 0]) - want) <= (H + 1) * U32 * abs(want)      # all terms positive: y is 8 x


# ---------------------------------------------------------------- graphs
def test_most_tokens():
    """2^24 - 1 tokens, the most there may be: the index against torch's stable sort, rows and sums exact."""
    T, H, E = (1 << 24) - 1, 8, 3
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(0, E, (T, 1), dtype=torch.int32, device="cuda", generator=g)
    nb = lb.lowbit_moe_sort_workspace_bytes(T, 1, E)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    rs, sr = (torch.full((T,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    of = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    lb.check(lb.lowbit_moe_sort(ids, T, 1, E, None, E, rs, sr, of, ws, nb))
    order = torch.sort(ids.view(-1), stable=True).indices
    assert torch.equal(rs.long(), order)
    assert torch.equal(sr[order].long(), torch.arange(T, device="cuda"))
    assert of.tolist() == [0] + torch.cumsum(torch.bincount(ids.view(-1).long(), minlength=E), 0).tolist()
    x = torch.randint(-8, 9, (T, H), device="cuda", generator=g).half()
    w = torch.randint(-4, 5, (T, 1), device="cuda", generator=g).float()
    xp, y, dyp = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    dw = torch.zeros((T, 1), device="cuda")
    lb.check(lb.lowbit_moe_permute(x, None, T, 1, 2 * H, sr, xp, None))
    assert torch.equal(xp, x[order])
    lb.check(lb.lowbit_moe_unpermute(xp, lb.LOWBIT_F16, w, T, 1, H, sr, y))
    assert torch.equal(y, (w * x.float()).half())
    lb.check(lb.lowbit_moe_unpermute_backward(x, xp, lb.LOWBIT_F16, w, T, 1, H, sr, dyp, dw))
    assert torch.equal(dyp, (w * x.float()).half()[order])
    assert torch.equal(dw.view(-1), (x.float() * x.float()).sum(1))


@pytest.mark.parametrize("T", [40, 3000])
def test_sort_and_rows_graph_replays(T):
    """Sort, permute, unpermute and its gradient captured once and replayed on new routings."""
    top_k, E, H = 4, 16, 264
    S = T * top_k
    rng = np.random.default_rng(T)
    ids = dev(routing(rng, T, E, top_k))
    x = _rows(rng, T, H, torch.bfloat16).cuda()
    w = dev(rng.random((T, top_k)).astype(np.float32))
    out = dict(rs=torch.empty(S, dtype=torch.int32, device="cuda"), sr=torch.empty(S, dtype=torch.int32, device="cuda"),
               of=torch.empty(E + 1, dtype=torch.int32, device="cuda"),
               xp=torch.empty((S, H), dtype=torch.bfloat16, device="cuda"),
               y=torch.empty((T, H), dtype=torch.bfloat16, device="cuda"),
               dyp=torch.empty((S, H), dtype=torch.bfloat16, device="cuda"),
               dw=torch.empty((T, top_k), device="cuda"))
    nb = lb.lowbit_moe_sort_workspace_bytes(T, top_k, E)
    ws = torch.empty(max(nb, 1), dtype=torch.uint8, device="cuda")

    def calls(st):
        lb.check(lb.lowbit_moe_sort(ids, T, top_k, E, None, E, out["rs"], out["sr"], out["of"], ws, nb, st))
        lb.check(lb.lowbit_moe_permute(x, None, T, top_k, 2 * H, out["sr"], out["xp"], None, st))
        lb.check(lb.lowbit_moe_unpermute(out["xp"], lb.LOWBIT_BF16, w, T, top_k, H, out["sr"], out["y"], st))
        lb.check(lb.lowbit_moe_unpermute_backward(x, out["xp"], lb.LOWBIT_BF16, w, T, top_k, H, out["sr"], out["dyp"],
                                                  out["dw"], st))

    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            calls(stream.cuda_stream)
    for rep in range(3):
        ids.copy_(torch.from_numpy(routing(rng, T, E, top_k)))
        torch.cuda.synchronize()
        calls(None)
        torch.cuda.synchronize()
        eager = {k: v.clone() for k, v in out.items()}
        for v in out.values():
            v.fill_(-1)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.synchronize()
        for k, v in out.items():
            assert torch.equal(v, eager[k]), k
