"""Cases that time the 8-bit integer products and the sorting of tokens by expert, and say what they return.

Five operators:
  gemm      y = x_scale * w_scale * (xq @ wq^T) + bias: int8 codes, a scale per token and per channel
  experts   the same product for rows sorted by expert, each with its expert's weights
  permute   slots sorted by expert (the index) and the tokens' rows brought into that order
  unpermute the rows back in token order, summed with the router's weights
  gradient  the backward pass of unpermute (rows and router weights) and of permute (tokens)

Where ``own`` is false ``run`` computes them from elementary torch operations in binary32; where it is true it calls
the library.  Sizes are those of the decoder and the MoE layer that the package's workloads use (projections of
4096 x 4096 up to 28672 x 4096, 128 experts of 2048 x 768 with 8 per token), and odd ones beside them.
"""
import math

import torch

own = False

F16, BF16 = torch.float16, torch.bfloat16
DTYPES = {"f16": F16, "bf16": BF16}


def listed():
    return [
        # one token through an attention output projection: latency counts
        {"name": "gemm 1 token", "op": "gemm", "M": 1, "N": 4096, "K": 4096, "dtype": "f16", "bias": False},
        # a decode batch through the stacked gate and up projections: the weights' stream counts
        {"name": "gemm 16 tokens gate+up", "op": "gemm", "M": 16, "N": 28672, "K": 4096, "dtype": "f16", "bias": False},
        # a short prompt, ragged in every size, with a bias
        {"name": "gemm ragged", "op": "gemm", "M": 77, "N": 5003, "K": 4104, "dtype": "bf16", "bias": True},
        # a prefill chunk through the down projection: the matrix cores count
        {"name": "gemm prefill down", "op": "gemm", "M": 4096, "N": 4096, "K": 14336, "dtype": "bf16", "bias": False},
        # a decode batch through the experts' gate and up: rows gathered from the tokens, about one row an expert
        {"name": "experts decode", "op": "experts", "T": 16, "top_k": 8, "E": 128, "N": 1536, "K": 2048,
         "dtype": "f16", "gather": True},
        # a prefill chunk through the experts, rows already in order, about 256 rows an expert
        {"name": "experts prefill", "op": "experts", "T": 4096, "top_k": 8, "E": 128, "N": 1536, "K": 2048,
         "dtype": "bf16", "gather": False},
        # a small batch of quantized rows with their scales
        {"name": "permute codes", "op": "permute", "T": 37, "top_k": 8, "E": 128, "E_local": 128, "H": 2048,
         "dtype": "i8"},
        # a training or prefill batch of bf16 rows
        {"name": "permute batch", "op": "permute", "T": 16384, "top_k": 8, "E": 128, "E_local": 128, "H": 2048,
         "dtype": "bf16"},
        # a decode batch back in token order
        {"name": "unpermute decode", "op": "unpermute", "T": 16, "top_k": 8, "E": 128, "E_local": 128, "H": 2048,
         "dtype": "f16"},
        # a batch on a device that holds three quarters of the experts: the other slots have no row
        {"name": "unpermute batch", "op": "unpermute", "T": 8192, "top_k": 8, "E": 128, "E_local": 96, "H": 2048,
         "dtype": "bf16"},
        # a small training step with few wide experts
        {"name": "gradient small", "op": "gradient", "T": 333, "top_k": 2, "E": 8, "E_local": 8, "H": 4096,
         "dtype": "f16"},
        # a training batch
        {"name": "gradient batch", "op": "gradient", "T": 8192, "top_k": 8, "E": 128, "E_local": 128, "H": 2048,
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("gemm", "gemm", "experts", "permute", "unpermute", "gradient"))
    dtype = rng.choice(("f16", "bf16"))
    if op == "gemm":
        # one token to a prefill chunk; K a multiple of 8, as the codes' rows are
        while True:
            M, N, K = _log(rng, 1, 4096), _log(rng, 256, 28672), 8 * _log(rng, 16, 1792)
            if M * N * K <= 4096 * 4096 * 14336:
                return {"op": op, "M": M, "N": N, "K": K, "dtype": dtype, "bias": rng.random() < 0.5}
    T, E = _log(rng, 1, 16384), _log(rng, 2, 128)
    top_k = rng.randint(1, min(8, E))
    if op == "experts":
        while True:
            N, K = _log(rng, 128, 4096), 8 * _log(rng, 16, 512)
            if E * N * K <= 1 << 29 and T * top_k <= 32768 and T * top_k * N * K <= 4096 * 8 * 1536 * 2048:
                return {"op": op, "T": T, "top_k": top_k, "E": E, "N": N, "K": K, "dtype": dtype,
                        "gather": rng.random() < 0.5}
            T = _log(rng, 1, 4096)
    while True:
        H = 8 * _log(rng, 16, 1024)
        if T * top_k * H <= 16384 * 8 * 2048:
            break
        T = _log(rng, 1, 16384)
    E_local = E if rng.random() < 0.7 else rng.randint(1, E)
    if op == "permute" and rng.random() < 0.3:
        dtype = "i8"
    return {"op": op, "T": T, "top_k": top_k, "E": E, "E_local": E_local, "H": H, "dtype": dtype}


def _generator(seed, part):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 64 + part)


def _codes(rows, K, seed, part):
    """int8 codes and fp32 scales of normal rows with a few large values, as a per-row quantizer leaves them."""
    g = _generator(seed, part)
    x = torch.randn(rows, K, generator=g, device="cuda")
    x = x * torch.where(torch.rand(1, K, generator=g, device="cuda") < 0.005, 6.0, 1.0)
    x = x * (0.5 + torch.rand(rows, 1, generator=g, device="cuda"))
    scale = x.abs().amax(1) / 127
    return torch.round(x / scale[:, None]).clamp_(-127, 127).to(torch.int8), scale


def _routing(case, seed):
    """Distinct experts for each token, some experts liked more than others, and the router's weights."""
    g = _generator(seed, 40)
    logits = torch.randn(case["T"], case["E"], generator=g, device="cuda")
    logits += 0.5 * torch.randn(1, case["E"], generator=g, device="cuda")
    top, ids = logits.topk(case["top_k"], 1)
    return ids.to(torch.int32), torch.softmax(top, 1)


def _expert_map(case, seed):
    """Local numbers of the experts that this device holds, -1 for the others; None where it holds all."""
    if case["E_local"] == case["E"]:
        return None
    held = torch.randperm(case["E"], generator=_generator(seed, 41), device="cuda")[:case["E_local"]].sort().values
    local = torch.full((case["E"],), -1, dtype=torch.int32, device="cuda")
    local[held] = torch.arange(case["E_local"], dtype=torch.int32, device="cuda")
    return local


def _sorted_slots(ids, expert_map, E_local):
    """row_slot, slot_row and expert_offsets of the routed slots, in plain torch."""
    S = ids.numel()
    key = ids.reshape(-1).long()
    if expert_map is not None:
        key = expert_map[key].long()
    key = torch.where((key >= 0) & (key < E_local), key, E_local)
    key, order = torch.sort(key, stable=True)
    has_row = key < E_local
    rows = torch.arange(S, device=ids.device)
    slot_row = torch.empty(S, dtype=torch.int32, device=ids.device)
    slot_row[order] = torch.where(has_row, rows, -1).to(torch.int32)
    row_slot = torch.where(has_row, order, S).to(torch.int32)
    bounds = torch.arange(E_local + 1, device=ids.device)
    return row_slot, slot_row.view(ids.shape), torch.searchsorted(key, bounds).to(torch.int32)


def prepare(case, seed):
    op, dtype = case["op"], DTYPES.get(case["dtype"])
    s = dict(case)
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        s["xq"], s["x_scale"] = _codes(M, K, seed, 1)
        s["wq"], s["w_scale"] = _codes(N, K, seed, 2)
        s["w_scale"] *= 0.02
        s["bias"] = torch.randn(N, generator=_generator(seed, 3), device="cuda") if case["bias"] else None
        s["y"] = torch.zeros(M, N, dtype=dtype, device="cuda")
        # room for the partial sums of any of these products, as a program keeps it
        s["workspace"] = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
        return s
    ids, weights = _routing(case, seed)
    T, top_k, S = case["T"], case["top_k"], case["T"] * case["top_k"]
    if op == "experts":
        E, N, K = case["E"], case["N"], case["K"]
        s["xq"], s["x_scale"] = _codes(T if case["gather"] else S, K, seed, 1)
        wq, w_scale = _codes(E * N, K, seed, 2)
        s["wq"], s["w_scale"] = wq.view(E, N, K), 0.02 * w_scale.view(E, N)
        s["row_slot"], _, s["offsets"] = _sorted_slots(ids, None, E)
        s["most"] = int(torch.bincount(ids.reshape(-1).long(), minlength=E).max())
        s["y"] = torch.zeros(S, N, dtype=dtype, device="cuda")
        return s
    H = case["H"]
    s["ids"], s["weights"], s["map"] = ids, weights, _expert_map(case, seed)
    g = _generator(seed, 1)
    if op == "permute":
        if dtype is None:
            s["x"], s["x_scale"] = _codes(T, H, seed, 1)
            s["xp_scale"] = torch.zeros(S, device="cuda")
        else:
            s["x"] = torch.randn(T, H, generator=g, device="cuda").to(dtype)
            s["x_scale"] = s["xp_scale"] = None
        s["xp"] = torch.zeros(S, H, dtype=s["x"].dtype, device="cuda")
        s["row_slot"] = torch.empty(S, dtype=torch.int32, device="cuda")
        s["slot_row"] = torch.empty(T, top_k, dtype=torch.int32, device="cuda")
        s["offsets"] = torch.empty(case["E_local"] + 1, dtype=torch.int32, device="cuda")
        s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
        return s
    _, s["slot_row"], _ = _sorted_slots(ids, s["map"], case["E_local"])
    s["yp"] = torch.randn(S, H, generator=g, device="cuda").to(dtype)
    if op == "unpermute":
        s["y"] = torch.zeros(T, H, dtype=dtype, device="cuda")
        return s
    s["dy"] = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    s["dxp"] = torch.randn(S, H, generator=g, device="cuda").to(dtype)
    s["dyp"] = torch.zeros(S, H, dtype=dtype, device="cuda")
    s["dw"] = torch.zeros(T, top_k, device="cuda")
    s["dx"] = torch.zeros(T, H, dtype=dtype, device="cuda")
    return s


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import bit_weight_only_pack_amd as lb
    op, dtype = s["op"], lb.LOWBIT_BF16 if s["dtype"] == "bf16" else lb.LOWBIT_F16
    if op == "gemm":
        lb.check(lb.lowbit_gemm_w8a8(s["M"], s["N"], s["K"], s["xq"], s["x_scale"], s["wq"], s["w_scale"], s["bias"],
                                     s["y"], dtype, s["workspace"], s["workspace"].numel()))
        return s["y"]
    T, top_k = s["T"], s["top_k"]
    if op == "experts":
        gather = s["gather"]
        lb.check(lb.lowbit_moe_gemm_w8a8(s["E"], s["N"], s["K"], s["wq"], s["w_scale"], s["xq"], s["x_scale"],
                                         s["xq"].shape[0], s["row_slot"] if gather else None, top_k if gather else 1,
                                         s["offsets"], T * top_k, s["y"], dtype))
        return s["y"]
    H = s["H"]
    if op == "permute":
        lb.check(lb.lowbit_moe_sort(s["ids"], T, top_k, s["E"], s["map"], s["E_local"], s["row_slot"], s["slot_row"],
                                    s["offsets"], s["workspace"], s["workspace"].numel()))
        lb.check(lb.lowbit_moe_permute(s["x"], s["x_scale"], T, top_k, H * s["x"].element_size(), s["slot_row"],
                                       s["xp"], s["xp_scale"]))
        out = {"rows": s["xp"], "row_slot": s["row_slot"], "slot_row": s["slot_row"], "offsets": s["offsets"]}
        return out if s["xp_scale"] is None else {**out, "scale": s["xp_scale"]}
    if op == "unpermute":
        lb.check(lb.lowbit_moe_unpermute(s["yp"], dtype, s["weights"], T, top_k, H, s["slot_row"], s["y"]))
        return s["y"]
    lb.check(lb.lowbit_moe_unpermute_backward(s["dy"], s["yp"], dtype, s["weights"], T, top_k, H, s["slot_row"],
                                              s["dyp"], s["dw"]))
    lb.check(lb.lowbit_moe_unpermute(s["dxp"], dtype, None, T, top_k, H, s["slot_row"], s["dx"]))
    return {"rows": s["dyp"], "weights": s["dw"], "tokens": s["dx"]}


def _plain(s):
    op, dtype = s["op"], DTYPES.get(s["dtype"])
    if op == "gemm":
        y = s["xq"].float() @ s["wq"].float().t()
        y = y * s["x_scale"][:, None] * s["w_scale"][None, :]
        return (y if s["bias"] is None else y + s["bias"]).to(dtype)
    S = s["T"] * s["top_k"]
    if op == "experts":
        # every expert's rows padded to the most that one has, one batched product, and the rows read back
        E, most, offsets = s["E"], s["most"], s["offsets"].long()
        place = torch.arange(most, device="cuda")
        row = (offsets[:-1, None] + place).clamp_(max=S - 1)
        if s["gather"]:
            row = s["row_slot"].long()[row] // s["top_k"]
        x = s["xq"][row].float()
        y = torch.bmm(x, s["wq"].float().transpose(1, 2))
        y = y * s["x_scale"][row][:, :, None] * s["w_scale"][:, None, :]
        rows = torch.arange(S, device="cuda")
        e = torch.searchsorted(offsets[1:], rows, right=True)
        return y[e, rows - offsets[e]].to(dtype)
    if op == "permute":
        row_slot, slot_row, offsets = _sorted_slots(s["ids"], s["map"], s["E_local"])
        has_row = row_slot < S
        token = torch.where(has_row, row_slot, 0).long() // s["top_k"]
        rows = s["x"][token] * has_row[:, None]
        out = {"rows": rows, "row_slot": row_slot, "slot_row": slot_row, "offsets": offsets}
        return out if s["x_scale"] is None else {**out, "scale": s["x_scale"][token] * has_row}
    row = s["slot_row"].long()
    has_row = (row >= 0).float()
    row = row.clamp(min=0)
    if op == "unpermute":
        return (s["yp"][row].float() * (s["weights"] * has_row)[:, :, None]).sum(1).to(dtype)
    dyp = torch.zeros(S + 1, s["H"], dtype=dtype, device="cuda")
    to = torch.where(s["slot_row"] >= 0, row, S)
    dy = s["dy"].float()
    dyp[to] = (s["weights"][:, :, None] * dy[:, None, :]).to(dtype)
    dw = (s["yp"][row].float() * dy[:, None, :]).sum(2) * has_row
    dx = (s["dxp"][row].float() * has_row[:, :, None]).sum(1).to(dtype)
    return {"rows": dyp[:S], "weights": dw, "tokens": dx}


def work(case):
    op = case["op"]
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + N * K + 4 * (M + N) + (4 * N if case["bias"] else 0) + 2 * M * N,
                "flops": 2 * M * N * K}
    T, top_k, E = case["T"], case["top_k"], case["E"]
    S = T * top_k
    if op == "experts":
        N, K = case["N"], case["K"]
        hit = E * (1 - (1 - top_k / E) ** T)     # experts that some token chose, were all liked alike
        rows = T if case["gather"] else S
        return {"bytes": int(hit * N * (K + 4)) + rows * (K + 4) + 4 * E + 2 * S * N, "flops": 2 * S * N * K}
    H, size = case["H"], 1 if case["dtype"] == "i8" else 2
    R = S * case["E_local"] // E                 # rows: the slots whose experts are here
    if op == "permute":
        scales = 4 * (T + R) if case["dtype"] == "i8" else 0
        return {"bytes": (T + R) * H * size + 12 * S + scales, "flops": S}
    if op == "unpermute":
        return {"bytes": (T + R) * H * 2 + 8 * S, "flops": 2 * R * H}
    return {"bytes": (T + 2 * R) * H * 2 + 12 * S + (T + R) * H * 2 + 4 * S, "flops": 4 * R * H}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gemm":
        total = torch.mm(s["xq"].double(), s["wq"].double().t())      # whole numbers below 2^53: no rounding
        total *= torch.outer(s["x_scale"].double(), s["w_scale"].double())
        if s["bias"] is not None:
            total += s["bias"].double()
        return total
    T, top_k = case["T"], case["top_k"]
    S = T * top_k
    if op == "experts":
        at, slots = s["offsets"].tolist(), s["row_slot"].long()
        source = slots.div(top_k, rounding_mode="floor") if case["gather"] else torch.arange(S, device="cuda")
        y = torch.zeros(S, case["N"], dtype=torch.float64, device="cuda")
        for e, (lo, hi) in enumerate(zip(at[:-1], at[1:])):
            mine = source[lo:hi]
            part = torch.mm(s["xq"][mine].double(), s["wq"][e].double().t())
            y[lo:hi] = part * s["x_scale"][mine].double()[:, None] * s["w_scale"][e].double()
        return y
    if op == "permute":
        # expert by expert: a token's row for every slot that chose it, slots in their order
        ids = s["ids"].reshape(-1)
        chosen = ids if s["map"] is None else s["map"][ids.long()]
        slots = torch.cat([torch.nonzero(chosen == e).view(-1) for e in range(case["E_local"])])
        rows = torch.zeros(S, case["H"], dtype=torch.float64, device="cuda")
        rows[:slots.numel()] = s["x"][slots // top_k].double()
        out = {"rows": rows, "row_slot": None, "slot_row": None, "offsets": None}
        if s["x_scale"] is None:
            return out
        scale = torch.zeros(S, dtype=torch.float64, device="cuda")
        scale[:slots.numel()] = s["x_scale"][slots // top_k].double()
        return {**out, "rows": None, "scale": scale}
    lists = {n: torch.zeros(T, case["H"], dtype=torch.float64, device="cuda") for n in ("y", "dx")}
    dyp = torch.zeros(S, case["H"], dtype=torch.float64, device="cuda")
    dw = torch.zeros(T, top_k, dtype=torch.float64, device="cuda")
    for j in range(top_k):
        here = torch.nonzero(s["slot_row"][:, j] >= 0).view(-1)
        row, w = s["slot_row"][here, j].long(), s["weights"][here, j].double()
        yp = s["yp"][row].double()
        if op == "unpermute":
            lists["y"][here] += w[:, None] * yp
            continue
        dy = s["dy"][here].double()
        lists["dx"][here] += s["dxp"][row].double()
        dyp[row] = w[:, None] * dy
        dw[here, j] = torch.linalg.vecdot(yp, dy)
    return lists["y"] if op == "unpermute" else {"rows": dyp, "weights": dw, "tokens": lists["dx"]}
