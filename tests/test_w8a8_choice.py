"""Host-side checks (CPU only) of which kernel a W8A8 product takes: the sizes
that the GPU tests run every kernel with still take it, all of them are
there, and a product with K split asks for its workspace."""
import bit_weight_only_pack_amd as lb
from w8a8_cases import DENSE, EXPERTS, Kernel, choice


def test_cases_take_the_kernels_they_are_for():
    for kernel, (M, N, K) in DENSE:
        assert choice(M, N, K) == kernel, (M, N, K)
    for kernel, counts, (E, N, K) in EXPERTS:
        rows = sum(counts.values())
        assert choice(rows, N, K, E) == kernel and choice(rows, N, K, E, rows) == kernel, (E, rows, N, K)


def test_every_kernel_has_cases():
    """Every kernel with a remainder of K behind its whole steps and without one."""
    dense = {(k, c[2] % 128 != 0) for k, c in DENSE}
    for tail in (False, True):
        have = {k for k, t in dense if t == tail}
        for rows in (8, 16, 32, 64):
            for channels in (16, 32, 64) if rows <= 16 else (16, 32):
                assert any(k.stream and (k.rows, k.channels) == (rows, channels) for k in have)
        for rows, channels, waves in ((64, 64, 8), (64, 64, 4), (128, 128, 4), (128, 256, 8), (256, 256, 4)):
            for splits in (1, 2, 4):
                assert Kernel(0, rows, channels, waves, splits) in have
    grouped = {(k, c[2] % 128 != 0) for k, _, c in EXPERTS}
    for k in (Kernel(1, 16, 32, 2, 1), Kernel(1, 16, 32, 4, 1), Kernel(0, 64, 64, 8, 1), Kernel(0, 64, 64, 4, 1),
              Kernel(0, 128, 128, 4, 1), Kernel(0, 128, 256, 8, 1), Kernel(0, 256, 256, 4, 1)):
        assert (k, False) in grouped and (k, True) in grouped, k


def test_k_has_more_steps_than_stages():
    """K is walked further than its first stages reach: twice round the ring, or by a split's share of it once."""
    for k, (M, N, K) in DENSE:
        if k.stream:
            stages = 3 if k.channels == 16 and k.rows < 64 else 2
            assert K // 128 // k.waves > stages, (M, N, K)
        else:
            step, stages = (256 if k.rows == 64 and k.waves == 8 else 128), {64: 4, 128: 3, 256: 2}[k.rows]
            assert K // step // k.splits > 2 * stages - (k.splits > 1) * stages, (M, N, K)
    for k, counts, (E, N, K) in EXPERTS:
        if k.stream:
            assert K // 128 // k.waves > (3 if k.waves == 4 else 2), (E, N, K)
        else:
            step, stages = (256 if k.rows == 64 and k.waves == 8 else 128), {64: 4, 128: 3, 256: 2}[k.rows]
            assert K // step > 2 * stages, (E, N, K)


def test_split_products_ask_for_a_workspace():
    split = [(k, c) for k, c in DENSE if k.splits > 1]
    assert len(split) >= 20
    at = 1 << 20                                     # a non-null address that is not read on these paths
    for k, (M, N, K) in DENSE:
        nb = lb.lowbit_gemm_w8a8_workspace_bytes(M, N, K)
        assert nb == (k.splits * M * N * 4 if k.splits > 1 else 0), (M, N, K)
        if k.splits > 1:
            call = lambda ws, n: lb.lowbit_gemm_w8a8(M, N, K, at, at, at, at, None, at, lb.LOWBIT_F16, ws, n)
            assert call(None, 0) == lb.LOWBIT_E_WORKSPACE and call(at, nb - 1) == lb.LOWBIT_E_WORKSPACE
            assert call(at + 128, nb) == lb.LOWBIT_E_INVALID_ARG


def launch_fits(c, rows, N, E=0):
    """The launch of this kernel has fewer than 2^32 threads along the grid's first side and 2^16 rows."""
    up = lambda a, b: -(-a // b)
    if c.stream:
        more = min(rows // 16, max(8, min(rows // 128, 1 << 15))) if E else 0
        return up(N, c.channels) * c.waves * 64 < 1 << 32 and E + more < 1 << 16
    tiles = (rows // c.rows + E if E else up(rows, c.rows)) * up(N, c.channels) * c.splits
    return up(tiles, 8) * 8 * c.waves * 64 < 1 << 32


def test_launches_fit_a_grid():
    """The largest sizes: a launch that a grid cannot hold is never chosen; what no kernel's grid holds is refused."""
    big = (1 << 24) - 1
    for M, N, K in ((big, 3, 8), (2, big, 8), (70, big, 8), (big, 256, 131064), (65536, 1 << 23, 64), (6016, big, 8)):
        assert launch_fits(choice(M, N, K), M, N), (M, N, K)
        assert lb.lowbit_gemm_w8a8_workspace_bytes(M, N, K) % (M * N * 4) == 0
    for E, rows, N, K in ((256, 3073, big, 8), (1024, 12289, big, 8), (1000, 50000, 1 << 22, 16), (128, 1537, big, 8),
                          (1, big, big, 64), (100, 4864, 60787 * 256, 8), (100, 4864, 60787 * 256, 1032),
                          (512, 7000, 9 << 20, 2056), (1024, big, 4096, 4096), (3, 40, big, 8)):
        for gathered in (0, 1000):
            assert launch_fits(choice(rows, N, K, E, gathered), rows, N, E), (E, rows, N, K)
    at = 1 << 20                                     # a non-null address that is not read on these paths
    call = lambda M, N, K: lb.lowbit_gemm_w8a8(M, N, K, at, at, at, at, None, at, lb.LOWBIT_F16, at, 1 << 62)
    for M, N in ((big, big), (big, 1 << 20), (1 << 20, 1 << 20), (1 << 23, 1 << 17)):     # 2^40 outputs and more
        assert call(M, N, 8) == lb.LOWBIT_E_UNSUPPORTED, (M, N)
        assert lb.lowbit_gemm_w8a8_workspace_bytes(M, N, 8) == 0
