"""Plain 64-bit implementations of the W8A8 products and of the sorting of
tokens by expert, with the error bounds of the library's binary32 steps."""
import numpy as np
import torch

import bit_weight_only_pack_amd as lb

DT = {"f16": (lb.LOWBIT_F16, torch.float16), "bf16": (lb.LOWBIT_BF16, torch.bfloat16)}
U32 = 2.0 ** -24                                   # half a step of binary32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def least(dtype):
    """Half the spacing of subnormal values: the rounding of results near zero."""
    fi = torch.finfo(dtype)
    return fi.smallest_normal * fi.eps / 2


def codes(rng, rows, K):
    """int8 codes over the whole range, -128 among them, and scales of several magnitudes."""
    q = rng.integers(-128, 128, size=(rows, K)).astype(np.int8)
    return q, (10.0 ** rng.uniform(-4, -1, size=rows)).astype(np.float32)


def product64(xq, xs, wq, ws, bias=None):
    """(y, bound of the binary32 steps) in float64; the sums are whole numbers below 2^53, so exact.
    Steps: the sum to binary32, times xs, times ws, plus bias: three roundings of the product and one of the sum."""
    s = xq.astype(np.float64) @ wq.astype(np.float64).T
    p = s * xs.astype(np.float64)[:, None] * ws.astype(np.float64)[None, :]
    y = p if bias is None else p + bias.astype(np.float64)
    mag = np.abs(p) if bias is None else np.abs(p) + np.abs(bias.astype(np.float64))
    return y, 4.01 * U32 * mag


def assert_rounded(got, y64, step32, dtype, what=""):
    """got (a torch tensor of `dtype`) is y64 within its own rounding plus the binary32 steps."""
    g = got.detach().cpu().to(torch.float64).numpy()
    bound = half_step(dtype) * (np.abs(y64) + step32) + step32 + least(dtype)
    bad = ~(np.abs(g - y64) <= bound)
    assert not bad.any(), "%s: %d of %d values off, worst %.3g of its bound at %s" % (
        what, bad.sum(), bad.size, np.nanmax(np.abs(g - y64) / bound), np.argwhere(bad)[:3].tolist())


def sort64(ids, E, emap, E_local):
    """row_slot, slot_row, offsets by the definition, in numpy."""
    flat = ids.reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < E), flat, -1)
    if emap is not None:
        key = np.where(key >= 0, np.asarray(emap, np.int64)[np.maximum(key, 0)], -1)
    key = np.where((key >= 0) & (key < E_local), key, -1)
    S = flat.size
    slots = [s for e in range(E_local) for s in np.nonzero(key == e)[0]]
    row_slot = np.full(S, S, np.int32)
    slot_row = np.full(S, -1, np.int32)
    row_slot[:len(slots)] = slots
    slot_row[slots] = np.arange(len(slots))
    offsets = np.concatenate([[0], np.cumsum([(key == e).sum() for e in range(E_local)])]).astype(np.int32)
    return row_slot, slot_row, offsets


def routing(rng, T, E, top_k, skew=0.7):
    """Distinct experts per token, some liked more than others."""
    logits = rng.standard_normal((T, E)) + skew * rng.standard_normal(E)
    return np.argsort(-logits, axis=1, kind="stable")[:, :top_k].astype(np.int32)


def gpu_sort(ids, E, emap, E_local, stream=None, fill=-7):
    """lowbit_moe_sort of a numpy [T][top_k]; outputs prefilled so that an unwritten value shows."""
    T, top_k = ids.shape
    d = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()
    S = T * top_k
    row_slot = torch.full((S,), fill, dtype=torch.int32, device="cuda")
    slot_row = torch.full((S,), fill, dtype=torch.int32, device="cuda")
    offs = torch.full((E_local + 1,), fill, dtype=torch.int32, device="cuda")
    nb = lb.lowbit_moe_sort_workspace_bytes(T, top_k, E_local)
    ws = torch.full((max(nb, 1),), 0x5A, dtype=torch.uint8, device="cuda")
    dm, di = d(emap), d(ids)
    lb.check(lb.lowbit_moe_sort(di, T, top_k, E, dm, E_local, row_slot, slot_row, offs, ws, nb, stream))
    torch.cuda.synchronize()
    return row_slot, slot_row, offs
