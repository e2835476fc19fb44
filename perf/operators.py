"""The routed-expert operators: what is run, on which inputs, in a plain form and through the library.

Operators (`case["op"]`):
  route       sort the tokens' slots by expert, gather the tokens into that order, return the experts' rows weighted
  route_grad  the gradients of both: d(expert rows), d(weights) of the weighted return, d(tokens) of the gather
  experts     C[p] = A[p] . W_e^T for the rows p of each expert e
  experts_grad  its gradients dA[p] = G[p] . W_e and dW_e = G_e^T . A_e
  int8        rows quantised to 8 bits by their largest value, times 8-bit weights with a scale a channel; plain or by expert
"""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # one decoded token sent to eight of 64 experts: launches and latency
        {"name": "route_token", "op": "route", "T": 1, "k": 8, "E": 64, "H": 4096, "dtype": "bf16", "drop": 0.0},
        # a ragged batch of odd width in fp32, a tenth of the slots over capacity
        {"name": "route_odd", "op": "route", "T": 1237, "k": 3, "E": 20, "H": 1031, "dtype": "f32", "drop": 0.1},
        # a training or prefill batch
        {"name": "route_batch", "op": "route", "T": 16384, "k": 4, "E": 32, "H": 2048, "dtype": "bf16", "drop": 0.02},
        # the gradients of a small ragged batch, width not a multiple of the vector
        {"name": "route_grad_odd", "op": "route_grad", "T": 2053, "k": 2, "E": 8, "H": 1002, "dtype": "f16", "drop": 0.1},
        # the gradients of the training batch
        {"name": "route_grad_batch", "op": "route_grad", "T": 16384, "k": 4, "E": 32, "H": 2048, "dtype": "bf16", "drop": 0.02},
        # eight decoded tokens over 64 experts: most experts have one row or none, the weights' bytes count
        {"name": "experts_decode", "op": "experts", "T": 8, "k": 4, "E": 64, "N": 2048, "K": 2048, "dtype": "bf16", "drop": 0.0},
        # a prefill batch
        {"name": "experts_prefill", "op": "experts", "T": 16384, "k": 2, "E": 16, "N": 4096, "K": 2048, "dtype": "bf16", "drop": 0.0},
        # a fine-tuning step's ragged batch, sizes that end inside every tile
        {"name": "experts_grad_ragged", "op": "experts_grad", "T": 1501, "k": 2, "E": 12, "N": 1000, "K": 776, "dtype": "f16", "drop": 0.05},
        # a training step
        {"name": "experts_grad_train", "op": "experts_grad", "T": 8192, "k": 2, "E": 8, "N": 2048, "K": 2048, "dtype": "bf16", "drop": 0.0},
        # one decoded token through a quantised layer
        {"name": "int8_token", "op": "int8", "T": 1, "k": 1, "E": 1, "N": 4096, "K": 4096, "dtype": "bf16", "drop": 0.0},
        # a serving batch through the same layer
        {"name": "int8_batch", "op": "int8", "T": 500, "k": 1, "E": 1, "N": 4096, "K": 4096, "dtype": "bf16", "drop": 0.0},
        # a prefill batch through quantised experts
        {"name": "int8_experts", "op": "int8", "T": 8192, "k": 2, "E": 8, "N": 4096, "K": 2048, "dtype": "bf16", "drop": 0.0},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width(lo, hi, step):  # an odd multiple of `step`, so never a round power of two
        return step * (2 * (spread(lo, hi) // (2 * step)) + 1)

    op = rng.choice(["route", "route_grad", "experts", "experts_grad", "int8"])
    dtype = rng.choice(["bf16", "f16"])
    drop = rng.choice([0.0, 0.03, 0.2])
    k = rng.choice([1, 2, 3, 4, 6, 8])
    E = rng.choice([8, 12, 16, 32, 60, 64])
    if op in ("route", "route_grad"):
        T = spread(1, 12000) | 1
        H = width(128, 4096, rng.choice([1, 2, 8]))
        return {"op": op, "T": T, "k": k, "E": E, "H": H, "dtype": rng.choice(["f32", "bf16", "f16"]), "drop": drop}
    N, K = width(256, 4096, 8), width(256, 4096, 8)
    T = spread(1, 8192) | 1
    if op == "int8" and rng.random() < 0.5:
        return {"op": op, "T": T, "k": 1, "E": 1, "N": N, "K": K, "dtype": dtype, "drop": 0.0}
    k = min(k, max(1, int(1.2e11 / (T * N * K))))  # no more than the largest listed case
    return {"op": op, "T": T, "k": k, "E": E, "N": N, "K": K, "dtype": dtype, "drop": drop}


def routing(case, g):
    """Expert ids [T, k] of a router with popular and rare experts: k distinct ones a token, some slots dropped (-1)."""
    T, k, E = case["T"], case["k"], case["E"]
    bias = -0.5 * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    bias = bias[torch.randperm(E, device="cuda", generator=g)]
    u = torch.rand(T, E, device="cuda", generator=g).clamp_(1e-7, 1 - 1e-7)
    score = bias - torch.log(-torch.log(u))
    weight, ids = torch.topk(score, k, dim=1)
    ids = ids.to(torch.int32)
    ids[torch.rand(T, k, device="cuda", generator=g) < case["drop"]] = -1
    return ids.contiguous(), torch.softmax(weight, 1).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DT[case["dtype"]]

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dt)

    T, k, E = case["T"], case["k"], case["E"]
    st = {"op": case["op"], "T": T, "k": k, "E": E, "dt": dt}
    ids, weight = routing(case, g)
    S = T * k
    if case["op"] in ("route", "route_grad"):
        H = case["H"]
        st |= {"ids": ids, "weight": weight}
        if case["op"] == "route":
            return st | {"X": normal(T, H), "Ys": normal(S, H)}
        offsets, slot, pos = plain_sort(ids, E)
        return st | {"offsets": offsets, "slot": slot, "pos": pos, "dY": normal(T, H), "Ys": normal(S, H), "dXs": normal(S, H)}
    N, K = case["N"], case["K"]
    offsets = plain_sort(ids, E)[0]
    st |= {"offsets": offsets}
    if case["op"] == "experts":
        return st | {"A": normal(S, K), "W": normal(E, N, K, scale=K ** -0.5)}
    if case["op"] == "experts_grad":
        return st | {"A": normal(S, K), "G": normal(S, N), "W": normal(E, N, K, scale=K ** -0.5)}
    X = torch.randn(S, K, device="cuda", generator=g)
    X[:, torch.randperm(K, device="cuda", generator=g)[: max(1, K // 128)]] *= 8  # the channels that activations have large values in
    Wq = torch.randint(-127, 128, (E, N, K), device="cuda", generator=g, dtype=torch.int8)
    ws = (torch.rand(E, N, device="cuda", generator=g) + 0.5) * (K ** -0.5 / 73)
    return st | {"X": X.to(dt), "Wq": Wq, "ws": ws}


# ---------------------------------------------------------------- the plain forms


def plain_sort(ids, E):
    x = ids.reshape(-1)
    S = x.numel()
    keep = (x >= 0) & (x < E)
    e = torch.where(keep, x, torch.zeros_like(x)).long()
    hot = (e == torch.arange(E, device=x.device)[:, None]) & keep
    running = torch.cumsum(hot, 1, dtype=torch.int32)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=x.device)
    offsets[1:] = torch.cumsum(running[:, -1], 0, dtype=torch.int32)
    rank = running[e, torch.arange(S, device=x.device)] - 1
    pos = torch.where(keep, offsets[e] + rank, torch.full_like(x, -1))
    slot = torch.full((S + 1,), -1, dtype=torch.int32, device=x.device)
    at = torch.where(keep, pos, torch.full_like(pos, S)).long()
    slot[at] = torch.arange(S, device=x.device, dtype=torch.int32)
    return offsets, slot[:S].contiguous(), pos


def rows_of(M, at):
    """M's rows at `at` in 32 bits, zeros where that is -1."""
    return torch.where((at >= 0)[..., None], M[at.clamp(min=0).long()].float(), 0.0)


def plain_return(pos, Ys, weight, T, k):
    r = rows_of(Ys, pos.view(T, k))
    return (r if weight is None else r * weight[..., None]).sum(1)


def padded(offsets, S):
    """Places [E, most rows an expert has] of each expert's rows, -1 past its last."""
    cap = max(1, int((offsets[1:] - offsets[:-1]).max()))
    at = offsets[:-1, None].long() + torch.arange(cap, device=offsets.device)
    return torch.where(at < offsets[1:, None], at, torch.full_like(at, -1))


def scatter_rows(P, at, S):
    out = torch.zeros(S + 1, P.shape[-1], device=P.device)
    out[torch.where(at >= 0, at, torch.full_like(at, S)).reshape(-1)] = P.reshape(-1, P.shape[-1])
    return out[:S]


def plain(st):
    op, T, k, E, dt = st["op"], st["T"], st["k"], st["E"], st["dt"]
    S = T * k
    if op == "route":
        offsets, slot, pos = plain_sort(st["ids"], E)
        Xs = rows_of(st["X"], torch.where(slot >= 0, slot // k, slot))
        Y = plain_return(pos, st["Ys"], st["weight"], T, k)
        return {"offsets": offsets, "slot": slot, "pos": pos, "Xs": Xs.to(dt), "Y": Y.to(dt)}
    if op == "route_grad":
        slot, pos = st["slot"], st["pos"]
        dY, w = st["dY"].float(), st["weight"]
        dYs = rows_of(st["dY"], torch.where(slot >= 0, slot // k, slot)) * w.reshape(-1)[slot.clamp(min=0).long()][:, None]
        dw = (rows_of(st["Ys"], pos.view(T, k)) * dY[:, None, :]).sum(-1)
        dX = plain_return(pos, st["dXs"], None, T, k)
        return {"dYs": dYs.to(dt), "dw": dw, "dX": dX.to(dt)}
    at = padded(st["offsets"], S)
    if op == "experts":
        C = torch.bmm(rows_of(st["A"], at), st["W"].float().transpose(1, 2))
        return scatter_rows(C, at, S).to(dt)
    if op == "experts_grad":
        G = rows_of(st["G"], at)
        dA = scatter_rows(torch.bmm(G, st["W"].float()), at, S)
        dW = torch.bmm(G.transpose(1, 2), rows_of(st["A"], at))
        return {"dA": dA.to(dt), "dW": dW.to(dt)}
    x = st["X"].float()
    s = x.abs().amax(1) / 127.0
    q = torch.where(s[:, None] > 0, torch.round(x / s[:, None]), 0.0)
    C = scatter_rows(torch.bmm(rows_of(q, at), st["Wq"].float().transpose(1, 2)) * st["ws"][:, None, :], at, S)
    return (C * s[:, None]).to(dt)


# ---------------------------------------------------------------- through the library


def library(st):
    from csr_bsr_spmv_gb300 import spx

    op, T, k, E = st["op"], st["T"], st["k"], st["E"]
    if op == "route":
        r = spx.spx_route_build(st["ids"], E)
        Xs = spx.spx_route_gather(r, st["X"])
        Y = spx.spx_route_combine(r, st["Ys"], st["weight"])
        return {"offsets": r.offsets, "slot": r.slot, "pos": r.pos, "Xs": Xs, "Y": Y}
    if op == "route_grad":
        r = spx.Route(T, k, E, st["offsets"], st["slot"], st["pos"])
        dYs, dw = spx.spx_route_combine_grad(r, st["dY"], st["Ys"], st["weight"])
        return {"dYs": dYs, "dw": dw, "dX": spx.spx_route_combine(r, st["dXs"])}
    if op == "experts":
        return spx.spx_gemm_grouped(st["offsets"], st["A"], st["W"])
    if op == "experts_grad":
        dA = spx.spx_gemm_grouped(st["offsets"], st["G"], st["W"], layout="kn")
        return {"dA": dA, "dW": spx.spx_gemm_grouped_wgrad(st["offsets"], st["G"], st["A"])}
    q, s = spx.spx_quant_rows_i8(st["X"])
    if E == 1:
        return spx.spx_gemm_i8(q, s, st["Wq"][0], st["ws"][0], dtype=st["dt"])
    return spx.spx_gemm_i8(q, s, st["Wq"], st["ws"], offsets=st["offsets"], dtype=st["dt"])


def run(state):
    return library(state) if own else plain(state)


# ---------------------------------------------------------------- what a pass cannot do without


def kept(case):
    return case["T"] * case["k"] * (1 - case["drop"])


def work(case):
    T, k, E, b = case["T"], case["k"], case["E"], BYTES[case["dtype"]]
    S, rows = T * k, kept(case)
    if case["op"] in ("route", "route_grad"):
        H = case["H"]
        if case["op"] == "route":  # ids, order both ways, X, Xs, Ys, weights, Y
            return {"bytes": 12 * S + 4 * E + (T * H + S * H + rows * H + T * H) * b + 4 * S, "flops": 2 * rows * H}
        return {"bytes": 8 * S + (T * H + rows * H + S * H + rows * H + T * H) * b + 8 * S, "flops": 4 * rows * H}
    N, K = case["N"], case["K"]
    used = E * (1 - (1 - 1 / E) ** rows) if E > 1 else 1  # experts that have a row, about
    if case["op"] == "experts":
        return {"bytes": (rows * K + used * N * K + S * N) * b, "flops": 2 * rows * N * K}
    if case["op"] == "experts_grad":
        return {"bytes": (rows * N + rows * K + used * N * K + S * K + E * N * K) * b, "flops": 4 * rows * N * K}
    return {"bytes": S * K * b + used * N * K + 4 * S + 4 * E * N + S * N * b, "flops": 2 * rows * N * K}


# ---------------------------------------------------------------- 64 bits, from the definitions


def exact(case, seed):
    st = prepare(case, seed)
    T, k, E = st["T"], st["k"], st["E"]
    S = T * k
    if case["op"] == "route":
        ids = st["ids"].cpu().numpy().reshape(-1).astype(np.int64)
        kept_at = np.nonzero((ids >= 0) & (ids < E))[0]
        order = kept_at[np.argsort(ids[kept_at], kind="stable")]
        pos = np.full(S, -1, np.int64)
        pos[order] = np.arange(order.size)
        o = torch.from_numpy(order).cuda()
        Xs = torch.zeros(S, case["H"], dtype=torch.float64, device="cuda")
        Xs[: order.size] = st["X"].double()[o // k]
        Y = torch.zeros(T, case["H"], dtype=torch.float64, device="cuda")
        Y.index_add_(0, o // k, st["Ys"][: order.size].double() * st["weight"].reshape(-1).double()[o][:, None])
        return {"offsets": None, "slot": None, "pos": None, "Xs": Xs, "Y": Y}
    if case["op"] == "route_grad":
        o = st["slot"][st["slot"] >= 0].long()
        n = o.numel()
        w = st["weight"].reshape(-1).double()
        t = torch.div(o, k, rounding_mode="floor")
        dYs = torch.zeros(S, case["H"], dtype=torch.float64, device="cuda")
        dYs[:n] = st["dY"].double()[t] * w[o][:, None]
        dw = torch.zeros(S, dtype=torch.float64, device="cuda")
        dw[o] = torch.einsum("nh,nh->n", st["dY"].double()[t], st["Ys"][:n].double())
        dX = torch.zeros(T, case["H"], dtype=torch.float64, device="cuda")
        dX.index_add_(0, t, st["dXs"][:n].double())
        return {"dYs": dYs, "dw": dw.view(T, k), "dX": dX}
    off = st["offsets"].tolist()
    if case["op"] == "experts":
        C = torch.zeros(S, case["N"], dtype=torch.float64, device="cuda")
        for e in range(E):
            C[off[e] : off[e + 1]] = st["A"][off[e] : off[e + 1]].double() @ st["W"][e].double().T
        return C
    if case["op"] == "experts_grad":
        dA = torch.zeros(S, case["K"], dtype=torch.float64, device="cuda")
        dW = torch.zeros(E, case["N"], case["K"], dtype=torch.float64, device="cuda")
        for e in range(E):
            G = st["G"][off[e] : off[e + 1]].double()
            dA[off[e] : off[e + 1]] = G @ st["W"][e].double()
            dW[e] = G.T @ st["A"][off[e] : off[e + 1]].double()
        return {"dA": dA, "dW": dW}
    x = st["X"].double()
    s = x.abs().max(1).values / 127
    q = torch.round(x / s[:, None])
    C = torch.zeros(S, case["N"], dtype=torch.float64, device="cuda")
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        C[lo:hi] = (q[lo:hi] @ st["Wq"][e].double().T) * s[lo:hi, None] * st["ws"][e].double()
    return C
