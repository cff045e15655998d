"""GPU parity of the W8A8 products (int8 codes x int8 codes, a scale per token
and per channel) with a 64-bit evaluation of their definition, through the C
ABI: dense and for rows sorted by expert.  The bound of every value is its own
rounding to the output type plus the four binary32 steps of the epilogue; the
integer sums are exact, so nothing else may differ.  Outputs start as NaN and
lie between guard values that have to survive."""
import numpy as np
import pytest
import torch

import bit_weight_only_pack_amd as lb
import oracle
from bit_weight_only_pack_amd import synth
from gpu_util import dev
from w8a8_util import DT, U32, assert_rounded, codes, gpu_sort, product64, routing, sort64

pytestmark = pytest.mark.gpu

GUARD = 64          # elements before and after an output


def guarded(rows, N, dtype):
    """(whole buffer, the [rows][N] view inside it): guards 3.0, the view NaN."""
    whole = torch.full((rows * N + 2 * GUARD,), 3.0, dtype=dtype, device="cuda")
    view = whole[GUARD:GUARD + rows * N].view(rows, N)
    view.fill_(float("nan"))
    return whole, view


def guards_ok(whole):
    return bool((whole[:GUARD] == 3).all()) and bool((whole[-GUARD:] == 3).all())


def gemm(xq, xs, wq, ws, bias, dt, y=None, stream=None):
    code, dtype = DT[dt]
    (M, K), N = xq.shape, wq.shape[0]
    whole = None
    if y is None:
        whole, y = guarded(M, N, dtype)
    nb = lb.lowbit_gemm_w8a8_workspace_bytes(M, N, K)
    work = torch.full((max(nb, 1),), 0x5A, dtype=torch.uint8, device="cuda")
    lb.check(lb.lowbit_gemm_w8a8(M, N, K, xq, xs, wq, ws, bias, y, code, work, nb, stream))
    torch.cuda.synchronize()
    if whole is not None:
        assert guards_ok(whole), "values beside the output were written"
    return y


SHAPES = [
    # decode: one token, few tokens, ragged channels, K with and without a tail below 16 and 64
    (1, 1, 8), (1, 16, 64), (1, 300, 1056), (2, 33, 24), (3, 64, 136), (5, 1000, 4104), (8, 48, 14336), (15, 17, 72),
    (16, 4096, 1024), (1, 4096, 4096), (2, 20, 3000), (11, 35, 4200), (16, 24, 4224), (7, 18, 9000),
    # few rows and many channels
    (4, 12288, 4096), (9, 13001, 2200), (16, 12300, 4216), (5, 12295, 4224),
    # K shared between workgroups
    (17, 64, 9000), (40, 200, 14336), (64, 1000, 4104), (100, 131, 6664),
    # around the row counts where a tile ends
    (17, 40, 264), (31, 129, 512), (32, 128, 128), (33, 257, 200), (63, 64, 2048), (64, 64, 64), (65, 130, 1032),
    (100, 1023, 520), (127, 255, 8), (128, 256, 128), (129, 257, 136), (200, 96, 7176),
    # prefill
    (255, 511, 1024), (256, 256, 4096), (257, 513, 2056), (300, 1000, 384), (512, 6144, 256), (1030, 770, 1288),
    (2048, 2056, 520), (4097, 40, 144),
    # weights streamed: every width of channels and rows, K below one unit of a wave, rings that are not full and full
    (8, 4096, 1000), (9, 4097, 1160), (16, 4095, 7176), (17, 4090, 136), (32, 4000, 4104), (33, 4095, 2184),
    (48, 4096, 64), (64, 4081, 6152), (1, 4100, 4104), (8, 8190, 264), (16, 8192, 2312), (18, 4120, 4088),
    (32, 8177, 1032), (33, 4111, 72), (64, 8192, 520), (50, 5003, 4104), (3, 8193, 1096), (16, 8200, 520),
    # K shared between workgroups, tiles of 64 with few and with many of them
    (17, 8200, 136), (64, 8193, 1032), (40, 9000, 4104), (65, 64, 9000), (70, 200, 14336), (96, 1000, 4104),
]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dt,bias", [("f16", False), ("bf16", True)])
def test_gemm_parity(M, N, K, dt, bias):
    rng = np.random.default_rng(M * 1000003 + N * 1009 + K)
    (xq, xs), (wq, ws) = codes(rng, M, K), codes(rng, N, K)
    b = rng.standard_normal(N).astype(np.float32) if bias else None
    y64, step = product64(xq, xs, wq, ws, b)
    if dt == "f16":
        xs /= np.float32(max(1.0, np.abs(y64).max() / 30000))     # inside binary16's range
        y64, step = product64(xq, xs, wq, ws, b)
    y = gemm(dev(xq), dev(xs), dev(wq), dev(ws), None if b is None else dev(b), dt)
    assert_rounded(y, y64, step, DT[dt][1], "M=%d N=%d K=%d" % (M, N, K))


@pytest.mark.parametrize("M,N,K", [
    (4090, 4095, 8200), (4096, 4096, 4096), (700, 9000, 520),
    # tiles of 64 (more than one a CU), 128, 256; K shared by workgroups
    (150, 6001, 200), (70, 9001, 208), (1500, 1502, 200), (3000, 4097, 2056), (24, 20567, 20384), (1500, 1501, 8200),
    (70, 9001, 4104), (70, 9002, 14328), (1001, 4097, 8200), (150, 9001, 14328),
    # 128 x 256 unsplit and by 2 and 4; 128 by 4; 256 by 2 and 4
    (1001, 4097, 200), (333, 6003, 8200), (150, 6001, 8200), (2100, 777, 14328), (131, 16463, 16184), (8193, 133, 18136),
])
def test_gemm_large(M, N, K):
    """Sizes of the wider tiles, ragged and not; the 64-bit product on the GPU, all values."""
    g = torch.Generator(device="cuda").manual_seed(M + K)
    xq = torch.randint(-128, 128, (M, K), dtype=torch.int8, device="cuda", generator=g)
    wq = torch.randint(-128, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    xs = torch.rand(M, device="cuda", generator=g) * 0.01
    ws = torch.rand(N, device="cuda", generator=g) * 0.01
    bias = torch.randn(N, device="cuda", generator=g)
    y = gemm(xq, xs, wq, ws, bias, "bf16").double()
    p64 = torch.mm(xq.double(), wq.double().t()) * xs.double()[:, None] * ws.double()[None, :]
    y64 = p64 + bias.double()
    step = 4.01 * U32 * (p64.abs() + bias.double().abs())
    bound = 2.0 ** -8 * (y64.abs() + step) + step + 2.0 ** -134
    assert bool(((y - y64).abs() <= bound).all())


@pytest.mark.parametrize("M", [1, 40, 300])
def test_gemm_largest_sums_are_exact(M):
    """Codes of -128 and 127 at the largest K: sums next to 2^31, each its own exact value."""
    K, N = 131064, 70
    wq = np.full((N, K), -128, np.int8)
    wq[1] = 127
    xq = np.full((M, K), -128, np.int8)
    xq[-1] = 127
    one_m, one_n = np.full(M, 2.0 ** -20, np.float32), np.ones(N, np.float32)
    y64, step = product64(xq, one_m, wq, one_n)
    assert np.abs(y64).max() * 2 ** 20 > 2 ** 31 - 2 ** 25
    y = gemm(dev(xq), dev(one_m), dev(wq), dev(one_n), None, "bf16")
    assert_rounded(y, y64, step, torch.bfloat16)


@pytest.mark.parametrize("M,N", [((1 << 24) - 1, 3), (2, (1 << 24) - 1), (70, (1 << 24) - 1)])
def test_gemm_most_rows_and_channels(M, N):
    """2^24 - 1 rows or channels, the most there may be; sums of small codes, exact in the output type."""
    K = 8
    g = torch.Generator(device="cuda").manual_seed(M % 1000)
    xq = torch.randint(-3, 4, (M, K), dtype=torch.int8, device="cuda", generator=g)
    wq = torch.randint(-3, 4, (N, K), dtype=torch.int8, device="cuda", generator=g)
    y = gemm(xq, torch.ones(M, device="cuda"), wq, torch.ones(N, device="cuda"), None, "f16")
    step = 1 << 20
    for lo in range(0, max(M, N), step):
        a, b = (xq[lo:lo + step], wq) if M > N else (xq, wq[lo:lo + step])
        want = a.float() @ b.float().t()
        assert torch.equal((y[lo:lo + step] if M > N else y[:, lo:lo + step]).float(), want)


def test_gemm_one_hot_is_exact():
    """One code 1 per token and scales of 1 return the weights' codes themselves."""
    rng = np.random.default_rng(11)
    for M, N, K in ((7, 90, 1000), (150, 260, 392)):
        wq, _ = codes(rng, N, K)
        xq = np.zeros((M, K), np.int8)
        at = rng.integers(0, K, M)
        xq[np.arange(M), at] = 1
        y = gemm(dev(xq), dev(np.ones(M, np.float32)), dev(wq), dev(np.ones(N, np.float32)), None, "f16")
        assert np.array_equal(y.cpu().numpy(), wq[:, at].T.astype(np.float16))


@pytest.mark.parametrize("M", [1, 9, 130])
def test_gemm_k_zero_and_empty(M):
    bias = np.linspace(-2, 2, 37).astype(np.float32)
    y = gemm(torch.empty((M, 0), dtype=torch.int8, device="cuda"), dev(np.ones(M, np.float32)),
             torch.empty((37, 0), dtype=torch.int8, device="cuda"), dev(np.ones(37, np.float32)), dev(bias), "f16")
    assert np.array_equal(y.cpu().numpy(), np.broadcast_to(bias.astype(np.float16), (M, 37)))
    y = gemm(torch.empty((M, 0), dtype=torch.int8, device="cuda"), dev(np.ones(M, np.float32)),
             torch.empty((37, 0), dtype=torch.int8, device="cuda"), dev(np.ones(37, np.float32)), None, "f16")
    assert bool((y == 0).all())


@pytest.mark.parametrize("M", [3, 70, 300])
def test_gemm_scales_that_are_not_finite_stay_in_their_row_and_column(M):
    rng = np.random.default_rng(M)
    N, K = 200, 328
    (xq, xs), (wq, ws) = codes(rng, M, K), codes(rng, N, K)
    xs[M // 2], ws[N // 3] = np.inf, np.nan
    xq[M // 2, 0] |= 1
    y64, step = product64(xq, np.where(np.isfinite(xs), xs, 1), wq, np.where(np.isfinite(ws), ws, 1))
    y = gemm(dev(xq), dev(xs), dev(wq), dev(ws), None, "bf16")
    g = y.cpu().to(torch.float64).numpy()
    assert np.isnan(g[:, N // 3]).all()
    others = np.delete(np.arange(N), N // 3)
    s = xq[M // 2].astype(np.int64) @ wq.astype(np.int64).T
    want = np.where(s[others] == 0, np.nan, np.sign(s[others]) * np.inf)
    assert np.array_equal(g[M // 2, others], want, equal_nan=True)
    rows = np.delete(np.arange(M), M // 2)
    assert_rounded(y[rows][:, others], y64[np.ix_(rows, others)], step[np.ix_(rows, others)], torch.bfloat16)


def test_gemm_reads_the_codes_of_the_quantizer():
    """lowbit_quant_act_i8's codes and scales go straight in; a zero row gives zeros."""
    M, N, K = 21, 130, 4096
    x = synth.activations_f16(M, K, outlier_frac=0.01, workload_id=810)
    x[4] = 0
    xq = torch.empty((M, K), dtype=torch.int8, device="cuda")
    xs = torch.empty((M,), dtype=torch.float32, device="cuda")
    lb.check(lb.lowbit_quant_act_i8(M, K, dev(x), xq, xs))
    rng = np.random.default_rng(3)
    wq, ws = codes(rng, N, K)
    y = gemm(xq, xs, dev(wq), dev(ws), None, "bf16")
    rq, rs = oracle.quant_act_i8(x)
    assert_rounded(y, *product64(rq, rs, wq, ws), torch.bfloat16)
    assert bool((y[4] == 0).all())


@pytest.mark.parametrize("M,offset", [(3, 1), (90, 1), (300, 1), (300, 2)])
def test_gemm_output_at_any_element(M, offset):
    """y may start at any element: stores wider than one element need more than that."""
    rng = np.random.default_rng(M + offset)
    N, K = 264, 256
    (xq, xs), (wq, ws) = codes(rng, M, K), codes(rng, N, K)
    whole = torch.full((M * N + 16,), 3.0, dtype=torch.bfloat16, device="cuda")
    y = whole[offset:offset + M * N].view(M, N)
    gemm(dev(xq), dev(xs), dev(wq), dev(ws), None, "bf16", y=y)
    assert_rounded(y, *product64(xq, xs, wq, ws), torch.bfloat16)
    assert bool((whole[:offset] == 3).all()) and bool((whole[offset + M * N:] == 3).all())


@pytest.mark.parametrize("which", ["weights", "tokens", "output"])
def test_gemm_past_2_31(which):
    """Weights, tokens and outputs whose offsets pass 2^31 (bytes, or elements of y): the last rows and columns."""
    K = {"weights": 8200, "tokens": 8200, "output": 16}[which]
    M, N = {"weights": (3, 262160), "tokens": (262160, 16), "output": (66000, 33000)}[which]
    g = torch.Generator(device="cuda").manual_seed(5)
    xq = torch.randint(-128, 128, (M, K), dtype=torch.int8, device="cuda", generator=g)
    wq = torch.randint(-128, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    xs = torch.rand(M, device="cuda", generator=g) * 0.01
    ws = torch.rand(N, device="cuda", generator=g) * 0.01
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    gemm(xq, xs, wq, ws, None, "bf16", y=y)
    rng = np.random.default_rng(1)
    rows = np.unique(np.concatenate([[0, M - 1], rng.integers(0, M, 6)]))
    cols = np.unique(np.concatenate([np.arange(min(N, 20)), np.arange(max(0, N - 20), N), rng.integers(0, N, 40)]))
    tr, tc = torch.from_numpy(rows).cuda(), torch.from_numpy(cols).cuda()
    want = product64(xq[tr].cpu().numpy(), xs[tr].cpu().numpy(), wq[tc].cpu().numpy(), ws[tc].cpu().numpy())
    assert_rounded(y[tr][:, tc], *want, torch.bfloat16, which)
    for lo in range(0, M, 1 << 14):
        assert not bool(torch.isnan(y[lo:lo + (1 << 14)]).any())


# ---------------------------------------------------------------- by expert
def experts64(xq, xs, wq, ws, src, offs):
    """Rows of the grouped product and their binary32 bound; rows outside the ranges stay NaN."""
    rows = len(src)
    y, step = np.full((rows, wq.shape[1]), np.nan), np.zeros((rows, wq.shape[1]))
    for e in range(wq.shape[0]):
        lo, hi = offs[e], offs[e + 1]
        a = src[lo:hi]
        y[lo:hi], step[lo:hi] = product64(xq[a], xs[a], wq[e], ws[e])
    return y, step


def run_experts(xq, xs, wq, ws, row_slot, row_div, offs, rows, dt, stream=None):
    code, dtype = DT[dt]
    E, N, K = wq.shape
    whole, y = guarded(rows, N, dtype)
    lb.check(lb.lowbit_moe_gemm_w8a8(E, N, K, wq, ws, xq, xs, xq.shape[0], row_slot, row_div, offs, rows, y, code,
                                     stream))
    torch.cuda.synchronize()
    assert guards_ok(whole)
    return y


@pytest.mark.parametrize("T,top_k,E,N,K,skew", [
    (1, 1, 1, 8, 8, 0.7), (1, 8, 128, 96, 256, 0.7), (3, 2, 4, 40, 72, 0.7), (16, 8, 128, 64, 264, 0.7),
    (40, 3, 4, 130, 512, 0.7), (37, 2, 300, 24, 136, 0.7),
    (300, 2, 8, 260, 520, 0.7), (300, 4, 16, 100, 1032, 3.0),      # ragged experts; most rows with a few experts
    (700, 2, 5, 513, 136, 0.7), (1500, 1, 3, 300, 264, 2.0),
    (5, 4, 1000, 16, 64, 0.7),                                     # most experts empty
    (400, 2, 2, 300, 4104, 0.0), (90, 2, 6, 70, 4232, 0.7), (3, 3, 3, 50, 9000, 0.7),      # long K
])
@pytest.mark.parametrize("gather,dt", [(True, "bf16"), (False, "f16")])
def test_experts_parity(T, top_k, E, N, K, skew, gather, dt):
    rng = np.random.default_rng(T * 31 + E * 7 + K)
    ids = routing(rng, T, E, top_k, skew)
    S = T * top_k
    row_slot, _, offs = sort64(ids, E, None, E)
    xq, xs = codes(rng, T if gather else S, K)
    wq, ws = codes(rng, E * N, K)
    ws = ws.reshape(E, N) * np.float32(0.01)
    wq = wq.reshape(E, N, K)
    src = row_slot // top_k if gather else np.arange(S)
    y64, step = experts64(xq, xs, wq, ws, src, offs)
    y = run_experts(dev(xq), dev(xs), dev(wq), dev(ws), dev(row_slot) if gather else None, top_k, dev(offs), S, dt)
    assert_rounded(y, y64, step, DT[dt][1], "T=%d E=%d" % (T, E))


@pytest.mark.parametrize("E,counts,N,K", [
    (100, {5: 700}, 70, 264), (100, {3: 16, 5: 17, 63: 33, 64: 300, 70: 1, 99: 48}, 40, 1608),   # the runs of 16 rows
    (70, {0: 8, 1: 9, 65: 400, 69: 31}, 33, 1536), (64, {63: 768}, 64, 2048), (1000, {1: 40, 998: 2000, 999: 50}, 9, 72),
    (3, {1: 36}, 100, 3000), (2, {0: 24}, 50, 64),
])
@pytest.mark.parametrize("gather", [True, False])
def test_experts_uneven(E, counts, N, K, gather):
    """Few rows an expert on average, but many with one or some of them."""
    rng = np.random.default_rng(E + K)
    S = sum(counts.values())
    offs = np.concatenate([[0], np.cumsum([counts.get(e, 0) for e in range(E)])]).astype(np.int32)
    (xq, xs), (wq, ws) = codes(rng, S, K), codes(rng, E * N, K)
    wq, ws = wq.reshape(E, N, K), ws.reshape(E, N) * np.float32(0.01)
    src = rng.permutation(S).astype(np.int32) if gather else np.arange(S)
    y64, step = experts64(xq, xs, wq, ws, src, offs)
    y = run_experts(dev(xq), dev(xs), dev(wq), dev(ws), dev(src) if gather else None, 1, dev(offs), S, "bf16")
    assert_rounded(y, y64, step, torch.bfloat16)


@pytest.mark.parametrize("counts,E,N,K", [
    ({0: 256, 3: 257, 90: 64, 91: 65, 92: 128, 93: 129, 94: 192, 99: 209}, 100, 777, 136),     # tiles of 128
    ({0: 1000, 5: 2064, 14: 1896, 15: 40}, 16, 333, 136),
    ({0: 2300, 1: 1412, 2: 1288}, 3, 3001, 2056), ({0: 128, 1: 2432, 2: 2440}, 3, 3001, 2064),  # of 256
    ({e: 20 + e for e in range(0, 40)}, 40, 333, 136),                                         # of 64
    ({0: 128, 2: 129, 3: 640, 9: 65, 12: 64, 13: 192, 14: 500, 15: 282}, 16, 1500, 136),       # of 128 x 256
    ({0: 300, 4: 1000, 15: 700}, 16, 2001, 2088),
    # one to sixteen experts a lane of the tile search, some of them empty
    ({e: e % 29 + 1 for e in range(0, 256, 1)}, 256, 40, 72), ({e: e % 31 for e in range(1, 257)}, 257, 70, 64),
    ({e: e % 27 + 2 for e in range(0, 1024)}, 1024, 33, 72), ({1: 1, 700: 13000, 1023: 70}, 1024, 64, 128),
])
@pytest.mark.parametrize("gather,dt", [(True, "bf16"), (False, "f16")])
def test_experts_large(counts, E, N, K, gather, dt):
    """Rows in tiles of every width whose last one is whole, more than half full and less; 64 bits on the GPU."""
    S = sum(counts.values())
    g = torch.Generator(device="cuda").manual_seed(S + K)
    offs = np.concatenate([[0], np.cumsum([counts.get(e, 0) for e in range(E)])]).astype(np.int32)
    xq = torch.randint(-128, 128, (S, K), dtype=torch.int8, device="cuda", generator=g)
    wq = torch.randint(-128, 128, (E, N, K), dtype=torch.int8, device="cuda", generator=g)
    xs = torch.rand(S, device="cuda", generator=g) * 0.001
    ws = torch.rand(E, N, device="cuda", generator=g) * 0.01
    src = torch.randperm(S, device="cuda", generator=g)
    if not gather:
        src = torch.arange(S, device="cuda")
    y = run_experts(xq, xs, wq, ws, (2 * src + 1).int() if gather else None, 2, dev(offs), S, dt)
    dtype = DT[dt][1]
    eps, tiny = torch.finfo(dtype).eps / 2, torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2
    for e in counts:
        at = slice(int(offs[e]), int(offs[e + 1]))
        a = src[at]
        y64 = torch.mm(xq[a].double(), wq[e].double().t()) * xs[a].double()[:, None] * ws[e].double()[None, :]
        step = 4.01 * U32 * y64.abs()
        assert bool(((y[at].double() - y64).abs() <= eps * (y64.abs() + step) + step + tiny).all()), e


@pytest.mark.parametrize("T", [20, 400])
def test_experts_rows_outside_stay(T):
    """Slots without a local expert: rows behind the last one keep what they held, and so does a table cut to `rows`."""
    rng = np.random.default_rng(T)
    top_k, E, El, N, K = 3, 16, 5, 70, 200
    ids = routing(rng, T, E, top_k)
    emap = np.full(E, -1, np.int32)
    emap[rng.permutation(E)[:El]] = rng.permutation(El)
    row_slot, slot_row, offs = gpu_sort(ids, E, emap, El)
    S, last = T * top_k, int(offs[-1])
    assert 0 < last < S
    (xq, xs), (wq, ws) = codes(rng, T, K), codes(rng, El * N, K)
    wq, ws = wq.reshape(El, N, K), ws.reshape(El, N)
    y = run_experts(dev(xq), dev(xs), dev(wq), dev(ws), row_slot, top_k, offs, S, "bf16")
    src = np.minimum(row_slot.cpu().numpy() // top_k, T - 1)
    y64, step = experts64(xq, xs, wq, ws, src, offs.cpu().numpy())
    assert_rounded(y[:last], y64[:last], step[:last], torch.bfloat16)
    assert bool(torch.isnan(y[last:]).all())
    cut = last - 7                                   # fewer rows than the table names
    y = run_experts(dev(xq), dev(xs), dev(wq), dev(ws), row_slot, top_k, offs, cut, "bf16")
    assert_rounded(y, y64[:cut], step[:cut], torch.bfloat16)


@pytest.mark.parametrize("x_rows", [262160, 524300])
@pytest.mark.parametrize("rows", [10, 100, 600])
def test_experts_gather_past_2_31(x_rows, rows):
    """Gathered rows whose offsets pass 2^31 and 2^32 bytes, among them the first and the last ones."""
    E, N, K = 4, 40, 8200
    g = torch.Generator(device="cuda").manual_seed(7)
    xq = torch.empty((x_rows, K), dtype=torch.int8, device="cuda")
    for lo in range(0, x_rows, 1 << 16):
        xq[lo:lo + (1 << 16)].random_(-128, 128, generator=g)
    wq = torch.randint(-128, 128, (E, N, K), dtype=torch.int8, device="cuda", generator=g)
    xs = torch.rand(x_rows, device="cuda", generator=g) * 0.01
    ws = torch.rand(E, N, device="cuda", generator=g) * 0.01
    rng = np.random.default_rng(rows)
    src = rng.integers(0, x_rows, rows)
    src[:2], src[-2:] = [0, x_rows - 1], [x_rows - 1, x_rows - 2]
    offs = np.array([0, rows // 3, rows // 3, rows - 5, rows], np.int32)
    y = run_experts(xq, xs, wq, ws, dev((3 * src + 1).astype(np.int32)), 3, dev(offs), rows, "bf16")
    t = torch.from_numpy(src).cuda()
    xc, xsc = xq[t].cpu().numpy(), xs[t].cpu().numpy()
    y64, step = experts64(xc, xsc, wq.cpu().numpy(), ws.cpu().numpy(), np.arange(rows), offs)
    assert_rounded(y, y64, step, torch.bfloat16)


@pytest.mark.parametrize("rows", [6, 90])
def test_experts_k_zero(rows):
    y = run_experts(torch.empty((rows, 0), dtype=torch.int8, device="cuda"), dev(np.ones(rows, np.float32)),
                    torch.empty((3, 20, 0), dtype=torch.int8, device="cuda"),
                    dev(np.ones((3, 20), np.float32)), None, 1, dev(np.array([0, 2, 2, rows], np.int32)), rows, "f16")
    assert bool((y == 0).all())


def test_experts_damaged_tables_stay_inside():
    """Slots and offsets outside their ranges read and write inside the matrices (what they compute is undefined)."""
    rng = np.random.default_rng(2)
    E, N, K, rows = 3, 40, 64, 50
    (xq, xs), (wq, ws) = codes(rng, 10, K), codes(rng, E * N, K)
    wq, ws = wq.reshape(E, N, K), ws.reshape(E, N)
    slots = np.full(rows, 1 << 30, np.int32)
    slots[::3] = -5
    offs = np.array([-4, 20, 900, 10 ** 9], np.int32)
    run_experts(dev(xq), dev(xs), dev(wq), dev(ws), dev(slots), 2, dev(offs), rows, "f16")


def test_experts_one_expert_equals_the_dense_product():
    rng = np.random.default_rng(8)
    for M, N, K in ((4, 100, 520), (260, 300, 1032)):
        (xq, xs), (wq, ws) = codes(rng, M, K), codes(rng, N, K)
        a = gemm(dev(xq), dev(xs), dev(wq), dev(ws), None, "bf16")
        b = run_experts(dev(xq), dev(xs), dev(wq[None]), dev(ws[None]), None, 1, dev(np.array([0, M], np.int32)), M,
                        "bf16")
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


# ---------------------------------------------------------------- streams and graphs
@pytest.mark.parametrize("M,N,K", [(1, 512, 2048), (60, 200, 4096), (100, 200, 8192), (300, 520, 1024)])
def test_gemm_graph_replays(M, N, K):
    """Captured once, replayed with new inputs and eager work between: every replay equals the eager bits."""
    rng = np.random.default_rng(M)
    (xq, xs), (wq, ws) = codes(rng, M, K), codes(rng, N, K)
    dx, dxs, dw, dws = dev(xq), dev(xs), dev(wq), dev(ws)
    y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    nb = lb.lowbit_gemm_w8a8_workspace_bytes(M, N, K)
    work = torch.empty(max(nb, 1), dtype=torch.uint8, device="cuda")
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            lb.check(lb.lowbit_gemm_w8a8(M, N, K, dx, dxs, dw, dws, None, y, lb.LOWBIT_BF16, work, nb,
                                         stream.cuda_stream))
    for rep in range(3):
        new = rng.integers(-128, 128, (M, K)).astype(np.int8)
        dx.copy_(torch.from_numpy(new))
        eager = gemm(dx, dxs, dw, dws, None, "bf16")
        y.fill_(float("nan"))
        work.fill_(rep)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.int16), eager.view(torch.int16))


def test_gemm_two_streams_at_once():
    """Two calls in flight with a workspace each give what they give alone."""
    rng = np.random.default_rng(4)
    sets = []
    for M, N, K in ((48, 512, 8192), (64, 300, 8200), (100, 512, 8192), (90, 300, 8200)):
        (xq, xs), (wq, ws) = codes(rng, M, K), codes(rng, N, K)
        d = (dev(xq), dev(xs), dev(wq), dev(ws))
        nb = lb.lowbit_gemm_w8a8_workspace_bytes(M, N, K)
        sets.append((M, N, K, d, torch.empty(max(nb, 1), dtype=torch.uint8, device="cuda"), nb,
                     torch.empty((M, N), dtype=torch.bfloat16, device="cuda"), gemm(*d, None, "bf16"),
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for M, N, K, d, work, nb, y, _, st in sets:
            lb.check(lb.lowbit_gemm_w8a8(M, N, K, *d, None, y, lb.LOWBIT_BF16, work, nb, st))
    torch.cuda.synchronize()
    for s in sets:
        assert torch.equal(s[6].view(torch.int16), s[7].view(torch.int16))


@pytest.mark.parametrize("T", [6, 300])
def test_experts_graph_replays(T):
    """Captured with the sorting before it, replayed on new routings: every replay equals the eager bits."""
    E, N, K, top_k = 12, 200, 520, 3
    rng = np.random.default_rng(T)
    (xq, xs), (wq, ws) = codes(rng, T, K), codes(rng, E * N, K)
    dx, dxs, dw, dws = dev(xq), dev(xs), dev(wq.reshape(E, N, K)), dev(ws.reshape(E, N))
    S = T * top_k
    ids, (rs, sr, of) = dev(routing(rng, T, E, top_k)), [torch.empty(n, dtype=torch.int32, device="cuda")
                                                         for n in (S, S, E + 1)]
    y = torch.empty((S, N), dtype=torch.float16, device="cuda")
    assert lb.lowbit_moe_sort_workspace_bytes(T, top_k, E) == 0

    def calls(st):
        lb.check(lb.lowbit_moe_sort(ids, T, top_k, E, None, E, rs, sr, of, None, 0, st))
        lb.check(lb.lowbit_moe_gemm_w8a8(E, N, K, dw, dws, dx, dxs, T, rs, top_k, of, S, y, lb.LOWBIT_F16, st))

    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            calls(stream.cuda_stream)
    for rep in range(3):
        ids.copy_(torch.from_numpy(routing(rng, T, E, top_k, 2.0 * rep)))
        torch.cuda.synchronize()
        calls(None)
        torch.cuda.synchronize()
        eager = y.clone()
        y.fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.int16), eager.view(torch.int16))


# ---------------------------------------------------------------- the operators together
@pytest.mark.parametrize("T,E,El,top_k,H,I", [(1, 8, 8, 2, 256, 128), (24, 16, 16, 4, 512, 264), (200, 8, 6, 2, 264, 136)])
def test_quantized_moe_layer_from_the_operators(T, E, El, top_k, H, I):
    """quantize -> sort -> gate/up by expert -> SiLU(gate) * up -> quantize -> down by expert -> back in token order,
    each step against 64 bits from what the step before left on the GPU; the rows gathered inside the product give the
    same bits as rows that were permuted before it."""
    rng = np.random.default_rng(T)
    ids = routing(rng, T, E, top_k)
    emap = None
    if El < E:
        emap = np.full(E, -1, np.int32)
        emap[np.sort(rng.permutation(E)[:El])] = np.arange(El)
    weights = rng.random((T, top_k)).astype(np.float32)
    x = synth.activations_f16(T, H, outlier_frac=0.01, workload_id=811, part=T)
    w1, s1 = codes(rng, El * 2 * I, H)
    w2, s2 = codes(rng, El * H, I)
    w1, w2 = w1.reshape(El, 2 * I, H), w2.reshape(El, H, I)
    s1, s2 = (s1.reshape(El, 2 * I) * 0.02).astype(np.float32), (s2.reshape(El, H) * 0.02).astype(np.float32)
    S = T * top_k

    xq = torch.empty((T, H), dtype=torch.int8, device="cuda")
    xs = torch.empty((T,), dtype=torch.float32, device="cuda")
    lb.check(lb.lowbit_quant_act_i8(T, H, dev(x), xq, xs))
    row_slot, slot_row, offs = gpu_sort(ids, E, emap, El)
    rs, sr, of = sort64(ids, E, emap, El)
    assert np.array_equal(row_slot.cpu().numpy(), rs) and np.array_equal(offs.cpu().numpy(), of)
    n = of[-1]
    gu = run_experts(xq, xs, dev(w1), dev(s1), row_slot, top_k, offs, S, "f16")
    y64, step = experts64(xq.cpu().numpy(), xs.cpu().numpy(), w1, s1, np.minimum(rs // top_k, T - 1), of)
    assert_rounded(gu[:n], y64[:n], step[:n], torch.float16, "gate/up")

    xp = torch.zeros((S, H), dtype=torch.int8, device="cuda")
    xps = torch.zeros((S,), dtype=torch.float32, device="cuda")
    lb.check(lb.lowbit_moe_permute(xq, xs, T, top_k, H, slot_row, xp, xps))
    again = run_experts(xp, xps, dev(w1), dev(s1), None, 1, offs, S, "f16")
    assert torch.equal(again[:n].view(torch.int16), gu[:n].view(torch.int16))

    act = torch.zeros((S, I), dtype=torch.float16, device="cuda")
    act[:n] = (torch.nn.functional.silu(gu[:n, :I].float()) * gu[:n, I:].float()).clamp(-60000, 60000).half()
    aq = torch.empty((S, I), dtype=torch.int8, device="cuda")
    as_ = torch.empty((S,), dtype=torch.float32, device="cuda")
    lb.check(lb.lowbit_quant_act_i8(S, I, act, aq, as_))
    down = run_experts(aq, as_, dev(w2), dev(s2), None, 1, offs, S, "bf16")
    y64, step = experts64(aq.cpu().numpy(), as_.cpu().numpy(), w2, s2, np.arange(S), of)
    assert_rounded(down[:n], y64[:n], step[:n], torch.bfloat16, "down")

    y = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    lb.check(lb.lowbit_moe_unpermute(down, lb.LOWBIT_BF16, dev(weights), T, top_k, H, slot_row, y))
    torch.cuda.synchronize()
    d64 = down[:n].cpu().to(torch.float64).numpy()
    y64, mag = np.zeros((T, H)), np.zeros((T, H))
    for s in range(S):
        if sr[s] >= 0:
            term = np.float64(weights.reshape(-1)[s]) * d64[sr[s]]
            y64[s // top_k] += term
            mag[s // top_k] += np.abs(term)
    assert_rounded(y, y64, (top_k + 1) * U32 * mag, torch.bfloat16, "layer")
