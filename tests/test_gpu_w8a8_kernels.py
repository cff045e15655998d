"""GPU parity of every kernel of the W8A8 products with K long enough that its
loop runs: stages are refilled, rings wrap, waits are partial.  Each case
asserts the kernel it is for before it runs it.  All values against the 64-bit
product, bounds as in w8a8_util."""
import numpy as np
import pytest
import torch

import bit_weight_only_pack_amd as lb
from gpu_util import dev
from w8a8_cases import DENSE, EXPERTS, choice
from w8a8_util import DT, U32, half_step, least

pytestmark = pytest.mark.gpu

GUARD = 64          # elements before and after an output


def codes(gen, *shape):
    return torch.randint(-128, 128, shape, dtype=torch.int8, device="cuda", generator=gen)


def scales(gen, *shape):
    return torch.rand(*shape, device="cuda", generator=gen) * 0.01


def check_rounded(y, p64, dtype, what, bias=None):
    """y is the product p64 (+ bias) within its own rounding and the four binary32 steps before it."""
    y64, mag = p64, p64.abs()
    if bias is not None:
        y64, mag = p64 + bias.double(), mag + bias.double().abs()
    step = 4.01 * U32 * mag
    bound = half_step(dtype) * (y64.abs() + step) + step + least(dtype)
    bad = ~((y.double() - y64).abs() <= bound)
    assert not bool(bad.any()), "%s: %d of %d values off, first at %s" % (
        what, int(bad.sum()), bad.numel(), bad.nonzero()[:3].tolist())


def guarded(rows, N, dtype):
    whole = torch.full((rows * N + 2 * GUARD,), 3.0, dtype=dtype, device="cuda")
    view = whole[GUARD:GUARD + rows * N].view(rows, N)
    view.fill_(float("nan"))
    return whole, view


def guards_ok(whole):
    return bool((whole[:GUARD] == 3).all()) and bool((whole[-GUARD:] == 3).all())


@pytest.mark.parametrize("kernel,sizes", DENSE, ids=lambda v: "x".join(map(str, v)))
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_dense(kernel, sizes, dt):
    M, N, K = sizes
    assert choice(M, N, K) == kernel
    code, dtype = DT[dt]
    g = torch.Generator(device="cuda").manual_seed(M * 7 + K)
    xq, wq, xs, ws = codes(g, M, K), codes(g, N, K), scales(g, M), scales(g, N)
    bias = torch.randn(N, device="cuda", generator=g) if dt == "bf16" else None
    whole, y = guarded(M, N, dtype)
    nb = lb.lowbit_gemm_w8a8_workspace_bytes(M, N, K)
    assert (nb > 0) == (kernel.splits > 1)
    work = torch.full((max(nb, 1),), 0x5A, dtype=torch.uint8, device="cuda")
    lb.check(lb.lowbit_gemm_w8a8(M, N, K, xq, xs, wq, ws, bias, y, code, work, nb))
    torch.cuda.synchronize()
    assert guards_ok(whole)
    p64 = torch.mm(xq.double(), wq.double().t()) * xs.double()[:, None] * ws.double()
    check_rounded(y, p64, dtype, "%s %s" % (kernel, sizes), bias)


@pytest.mark.parametrize("kernel,counts,sizes", EXPERTS, ids=lambda v: "x".join(map(str, v)) if len(v) < 6 else "")
@pytest.mark.parametrize("gather,dt", [(True, "bf16"), (False, "f16")])
def test_experts(kernel, counts, sizes, gather, dt):
    E, N, K = sizes
    S = sum(counts.values())
    assert choice(S, N, K, E, S if gather else 0) == kernel
    code, dtype = DT[dt]
    g = torch.Generator(device="cuda").manual_seed(S + K)
    offs = np.concatenate([[0], np.cumsum([counts.get(e, 0) for e in range(E)])]).astype(np.int32)
    xq, wq, xs, ws = codes(g, S, K), codes(g, E, N, K), scales(g, S), scales(g, E, N)
    src = torch.randperm(S, device="cuda", generator=g) if gather else torch.arange(S, device="cuda")
    whole, y = guarded(S, N, dtype)
    lb.check(lb.lowbit_moe_gemm_w8a8(E, N, K, wq, ws, xq, xs, S, (3 * src + 1).int() if gather else None, 3, dev(offs),
                                     S, y, code))
    torch.cuda.synchronize()
    assert guards_ok(whole)
    for e in counts:
        a = src[int(offs[e]):int(offs[e + 1])]
        p64 = torch.mm(xq[a].double(), wq[e].double().t()) * xs[a].double()[:, None] * ws[e].double()
        check_rounded(y[int(offs[e]):int(offs[e + 1])], p64, dtype, "%s expert %d" % (kernel, e))


def test_split_products_on_two_streams():
    """Products that each share K between workgroups, in flight together with a workspace each."""
    cases = [c for k, c in DENSE if k.splits > 1 and c[0] * c[1] * c[2] < 4e9]
    assert len(cases) >= 8
    sets = []
    for i, (M, N, K) in enumerate(cases):
        g = torch.Generator(device="cuda").manual_seed(i)
        d = (codes(g, M, K), scales(g, M), codes(g, N, K), scales(g, N))
        nb = lb.lowbit_gemm_w8a8_workspace_bytes(M, N, K)
        assert nb > 0
        work = torch.full((nb,), 0x5A, dtype=torch.uint8, device="cuda")
        alone, y = (torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        lb.check(lb.lowbit_gemm_w8a8(M, N, K, *d, None, alone, lb.LOWBIT_BF16, work, nb))
        sets.append((M, N, K, d, y, work, nb, alone))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for i, (M, N, K, d, y, work, nb, _) in enumerate(sets):
            lb.check(lb.lowbit_gemm_w8a8(M, N, K, *d, None, y, lb.LOWBIT_BF16, work, nb, streams[i % 2]))
    torch.cuda.synchronize()
    for M, N, K, _, y, _, _, alone in sets:
        assert torch.equal(y.view(torch.int16), alone.view(torch.int16)), (M, N, K)


@pytest.mark.parametrize("kernel,counts,sizes", EXPERTS, ids=lambda v: "x".join(map(str, v)) if len(v) < 6 else "")
def test_experts_with_offsets_that_do_not_ascend(kernel, counts, sizes):
    """Offsets that jump between both ends, whose row ranges overlap: what is computed is undefined, but every launch
    ends and nothing beside the output is written."""
    E, N, K = sizes
    S = sum(counts.values())
    assert choice(S, N, K, E) == kernel
    g = torch.Generator(device="cuda").manual_seed(S)
    xq, wq, xs, ws = codes(g, S, K), codes(g, E, N, K), scales(g, S), scales(g, E, N)
    up_down = np.where(np.arange(E + 1) % 2 == 0, 0, S)
    for offs in (up_down, S - up_down, np.linspace(S, 0, E + 1).astype(int),
                 np.where(np.arange(E + 1) % 2 == 0, -2 ** 31, 2 ** 31 - 1)):
        whole, y = guarded(S, N, torch.bfloat16)
        lb.check(lb.lowbit_moe_gemm_w8a8(E, N, K, wq, ws, xq, xs, S, None, 1, dev(offs.astype(np.int32)), S, y,
                                         lb.LOWBIT_BF16))
        torch.cuda.synchronize()
        assert guards_ok(whole)


def epilogue(total, xs, ws, bias, dtype):
    """fl(fl(fl(S) x_scale) w_scale + bias) rounded to `dtype`, all of it exact but the roundings: the product of two
    binary32 values is exact in binary64, and the sum goes there with its last bit odd if anything is left, so that the
    rounding to binary32 (29 bits shorter) is that of the exact sum."""
    p = total.float() * xs[:, None]
    t, b = p.double() * ws.double(), torch.zeros((), dtype=torch.float64, device="cuda") if bias is None else bias.double()
    s = t + b
    back = s - t
    left = (t - (s - back)) + (b - back)             # what the rounding of t + b dropped
    bits = s.view(torch.int64)
    toward = torch.where((left > 0) == (s > 0), 1, -1)
    odd = torch.where((left != 0) & (bits % 2 == 0), bits + toward, bits)
    return odd.view(torch.float64).float().to(dtype)


BITS = 6506, 10448, (5, 16, 20, 30, 50, 70, 130, 300, 400, 600, 800, 1500)      # N, K, numbers of rows


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("with_bias", [True, False])
def test_equal_inputs_give_equal_bits(dt, with_bias):
    """The same rows, alone and among others, through every kind of kernel: the bits of the documented steps."""
    N, K, counts = BITS
    kernels = {choice(M, N, K) for M in counts}
    assert len(kernels) == len(counts)
    assert {k.rows for k in kernels if k.stream} == {8, 16, 32, 64} and {k.splits for k in kernels} == {1, 2, 4}
    assert {(k.rows, k.channels) for k in kernels if not k.stream} == {(64, 64), (128, 128), (128, 256), (256, 256)}
    code, dtype = DT[dt]
    g = torch.Generator(device="cuda").manual_seed(3)
    xq, wq, xs, ws = codes(g, max(counts), K), codes(g, N, K), scales(g, max(counts)), scales(g, N)
    bias = torch.randn(N, device="cuda", generator=g) if with_bias else None
    total = torch.mm(xq.double(), wq.double().t())   # whole numbers below 2^53: exact
    want = epilogue(total, xs, ws, bias, dtype)
    if with_bias:                                    # a product rounded before the sum would show
        two = ((total.float() * xs[:, None]) * ws + bias).to(dtype)
        assert bool((two.view(torch.int16) != want.view(torch.int16)).any())
    for M in counts:
        nb = lb.lowbit_gemm_w8a8_workspace_bytes(M, N, K)
        work = torch.empty(max(nb, 1), dtype=torch.uint8, device="cuda")
        y = torch.full((M, N), float("nan"), dtype=dtype, device="cuda")
        lb.check(lb.lowbit_gemm_w8a8(M, N, K, xq, xs, wq, ws, bias, y, code, work, nb))
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.int16), want[:M].view(torch.int16)), (M, choice(M, N, K))
        if not with_bias:                            # by expert: one expert has all rows
            y.fill_(float("nan"))
            offs = torch.tensor([0, M], dtype=torch.int32, device="cuda")
            lb.check(lb.lowbit_moe_gemm_w8a8(1, N, K, wq, ws, xq, xs, M, None, 1, offs, M, y, code))
            torch.cuda.synchronize()
            assert torch.equal(y.view(torch.int16), want[:M].view(torch.int16)), (M, choice(M, N, K, 1))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_product_and_bias_have_one_rounding(dt):
    """A bias that is minus the first row's rounded product leaves what that rounding dropped, and not zero."""
    N, K, counts = BITS
    code, dtype = DT[dt]
    g = torch.Generator(device="cuda").manual_seed(4)
    xq, wq, xs, ws = codes(g, max(counts), K), codes(g, N, K), scales(g, max(counts)), scales(g, N)
    total = torch.mm(xq.double(), wq.double().t())
    bias = -((total[0].float() * xs[0]) * ws)
    want = epilogue(total, xs, ws, bias, dtype)
    assert bool((want[0] != 0).float().mean() > 0.5)
    for M in counts:
        nb = lb.lowbit_gemm_w8a8_workspace_bytes(M, N, K)
        work = torch.empty(max(nb, 1), dtype=torch.uint8, device="cuda")
        y = torch.full((M, N), float("nan"), dtype=dtype, device="cuda")
        lb.check(lb.lowbit_gemm_w8a8(M, N, K, xq, xs, wq, ws, bias, y, code, work, nb))
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.int16), want[:M].view(torch.int16)), (M, choice(M, N, K))
