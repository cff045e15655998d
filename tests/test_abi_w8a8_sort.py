"""Host-side checks (CPU only) of the W8A8 and sorting entry points: every
refusal comes back as a status code before anything is enqueued, and empty
calls return OK without touching memory."""
import bit_weight_only_pack_amd as lb

OK, ARG, UNS, WS = lb.LOWBIT_OK, lb.LOWBIT_E_INVALID_ARG, lb.LOWBIT_E_UNSUPPORTED, lb.LOWBIT_E_WORKSPACE
FAKE = 1 << 20  # a non-null address that must never be dereferenced on these paths
F16, BF16 = lb.LOWBIT_F16, lb.LOWBIT_BF16


def gemm(M=4, N=8, K=64, xq=FAKE, xs=FAKE, wq=FAKE, ws=FAKE, bias=None, y=FAKE, dt=F16, work=FAKE, nb=1 << 40):
    return lb.lowbit_gemm_w8a8(M, N, K, xq, xs, wq, ws, bias, y, dt, work, nb)


def test_gemm_refusals():
    assert gemm(M=-1) == ARG and gemm(N=-1) == ARG and gemm(K=-8) == ARG
    assert gemm(K=12) == ARG and gemm(K=65) == ARG
    assert gemm(K=131072) == UNS                                  # sums of codes would pass int32
    assert gemm(M=1 << 24) == UNS and gemm(N=1 << 24) == UNS
    assert gemm(dt=2) == UNS and gemm(dt=-1) == UNS
    for name in ("xq", "xs", "wq", "ws", "y"):
        assert gemm(**{name: None}) == ARG, name
    for name, at in (("xq", 8), ("wq", 8), ("xs", 2), ("ws", 2), ("bias", 2), ("y", 1)):
        assert gemm(**{name: FAKE + at}) == ARG, name
    assert gemm(M=0, xq=None, xs=None, wq=None, ws=None, y=None) == OK
    assert gemm(N=0, xq=None, xs=None, wq=None, ws=None, y=None) == OK


def test_gemm_workspace_is_checked():
    needs = [(M, N, K) for M in (1, 16, 17, 64, 128, 300) for N in (64, 1024, 4096) for K in (256, 4096, 14336)
             if lb.lowbit_gemm_w8a8_workspace_bytes(M, N, K) > 0]
    for M, N, K in needs:
        nb = lb.lowbit_gemm_w8a8_workspace_bytes(M, N, K)
        assert gemm(M, N, K, work=None, nb=0) == WS and gemm(M, N, K, nb=nb - 1) == WS
        assert gemm(M, N, K, work=FAKE + 128, nb=nb) == ARG
        assert nb % (M * N * 4) == 0                              # whole planes of int32 partial sums
    for bad in ((-1, 8, 64), (4, -8, 64), (4, 8, 60), (4, 8, 131072), (0, 8, 64), (4, 0, 64), (1 << 24, 8, 64)):
        assert lb.lowbit_gemm_w8a8_workspace_bytes(*bad) == 0


def experts(E=4, N=8, K=64, wq=FAKE, ws=FAKE, xq=FAKE, xs=FAKE, x_rows=10, slot=FAKE, div=2, offs=FAKE, rows=20,
            y=FAKE, dt=BF16):
    return lb.lowbit_moe_gemm_w8a8(E, N, K, wq, ws, xq, xs, x_rows, slot, div, offs, rows, y, dt)


def test_experts_refusals():
    assert experts(E=0) == ARG and experts(E=-1) == ARG and experts(E=1025) == UNS
    assert experts(N=-1) == ARG and experts(K=60) == ARG and experts(K=131072) == UNS and experts(N=1 << 24) == UNS
    assert experts(rows=-1) == ARG and experts(rows=1 << 24) == UNS and experts(x_rows=-1) == ARG
    assert experts(div=0) == ARG and experts(x_rows=0) == ARG
    assert experts(slot=None, x_rows=19) == ARG                   # rows in order: one of x for each of y
    assert experts(dt=5) == UNS
    for name in ("wq", "ws", "xq", "xs", "offs", "y"):
        assert experts(**{name: None}) == ARG, name
    for name, at in (("xq", 8), ("wq", 8), ("xs", 2), ("ws", 2), ("slot", 2), ("offs", 2), ("y", 1)):
        assert experts(**{name: FAKE + at}) == ARG, name
    assert experts(rows=0, slot=None, x_rows=0, wq=None, ws=None, xq=None, xs=None, offs=None, y=None) == OK
    assert experts(N=0, y=None) == OK


def sort(ids=FAKE, T=4, k=2, E=8, emap=None, El=8, rs=FAKE, sr=FAKE, of=FAKE, ws=None, nb=0):
    return lb.lowbit_moe_sort(ids, T, k, E, emap, El, rs, sr, of, ws, nb)


def test_sort_refusals():
    assert sort(T=-1) == ARG and sort(k=-1) == ARG and sort(E=0) == ARG and sort(El=0) == ARG
    assert sort(E=1025) == UNS and sort(El=1025) == UNS
    assert sort(T=1 << 24) == UNS and sort(T=1 << 23, k=256) == UNS
    for name in ("ids", "rs", "sr", "of"):
        assert sort(**{name: None}) == ARG, name
    for name in ("ids", "emap", "rs", "sr", "of"):
        assert sort(**{name: FAKE + 2}) == ARG, name
    nb = lb.lowbit_moe_sort_workspace_bytes(1 << 16, 8, 128)
    assert nb > 0 and nb % 4 == 0 and lb.lowbit_moe_sort_workspace_bytes(4, 2, 8) == 0
    big = dict(T=1 << 16, k=8, E=128, El=128)
    assert sort(**big) == WS and sort(**big, ws=FAKE, nb=nb - 1) == WS and sort(**big, ws=FAKE + 64, nb=nb) == ARG
    for bad in ((-1, 2, 8), (4, -1, 8), (4, 2, 0), (4, 2, 1025), (1 << 24, 1, 8)):
        assert lb.lowbit_moe_sort_workspace_bytes(*bad) == 0


def test_row_refusals():
    permute = lambda x=FAKE, s=None, T=4, k=2, rb=64, sr=FAKE, xp=FAKE, ps=None: lb.lowbit_moe_permute(
        x, s, T, k, rb, sr, xp, ps)
    assert permute(T=-1) == ARG and permute(k=-1) == ARG and permute(rb=-8) == ARG and permute(rb=12) == ARG
    assert permute(s=FAKE) == ARG and permute(ps=FAKE) == ARG                       # scales: both or neither
    assert permute(x=None) == ARG and permute(xp=None) == ARG and permute(sr=None) == ARG
    assert permute(x=FAKE + 8) == ARG and permute(xp=FAKE + 8) == ARG and permute(sr=FAKE + 2) == ARG
    assert permute(T=1 << 24) == UNS and permute(T=1 << 23, k=256) == UNS
    assert permute(T=0, x=None, xp=None, sr=None) == OK and permute(k=0, x=None, xp=None, sr=None) == OK
    assert permute(rb=0, x=None, xp=None, sr=None) == OK

    un = lambda yp=FAKE, dt=F16, w=None, T=4, k=2, H=64, sr=FAKE, y=FAKE: lb.lowbit_moe_unpermute(
        yp, dt, w, T, k, H, sr, y)
    assert un(T=-1) == ARG and un(k=-1) == ARG and un(H=-8) == ARG and un(H=60) == ARG and un(dt=2) == UNS
    assert un(yp=None) == ARG and un(sr=None) == ARG and un(y=None) == ARG
    assert un(yp=FAKE + 8) == ARG and un(y=FAKE + 2) == ARG and un(w=FAKE + 2) == ARG and un(sr=FAKE + 1) == ARG
    assert un(T=1 << 24) == UNS and un(T=1 << 23, k=256) == UNS
    assert un(T=0, yp=None, sr=None, y=None) == OK and un(H=0, yp=None, sr=None, y=None) == OK

    back = lambda dy=FAKE, yp=FAKE, dt=F16, w=FAKE, T=4, k=2, H=64, sr=FAKE, dyp=FAKE, dw=FAKE: \
        lb.lowbit_moe_unpermute_backward(dy, yp, dt, w, T, k, H, sr, dyp, dw)
    assert back(T=-1) == ARG and back(k=-1) == ARG and back(H=-8) == ARG and back(H=60) == ARG and back(dt=2) == UNS
    for name in ("dy", "yp", "w", "sr", "dyp", "dw"):
        assert back(**{name: None}) == ARG, name
    for name, at in (("dy", 8), ("yp", 8), ("dyp", 8), ("w", 2), ("dw", 2), ("sr", 2)):
        assert back(**{name: FAKE + at}) == ARG, name
    assert back(T=1 << 24) == UNS and back(T=1 << 23, k=256) == UNS
    assert back(T=0, dy=None, yp=None, w=None, sr=None, dyp=None, dw=None) == OK
    assert back(k=0, dy=None, yp=None, w=None, sr=None, dyp=None, dw=None) == OK
