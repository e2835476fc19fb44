"""What a block of routed experts has around and inside it: what is run, on which inputs, in a plain form and through the library.

Operators (`case["op"]`):
  norm        root-mean-square norm of the residual stream after the layer's output was added to it; 16 or 32 bits, or 8 bits with a scale a row
  norm_grad   its gradients: d(stream), with what arrives there past the norm, and d(weights)
  gated       C[p] = act(A[p] . Wg_e^T) * (A[p] . Wu_e^T) for the rows p of each expert e; in training also both factors before the activation
  gated_grad  from dY, the weights that follow and both factors: d(factors), and the product once more for the weights' gradient
  embed       rows of a table by token id, times a factor
  embed_grad  the table's gradient: for each id the sum of its tokens' gradients
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6


def listed():
    return [
        # one decoded token before an 8-bit product: launch and latency
        {"name": "norm_token", "op": "norm", "M": 1, "H": 4096, "dtype": "bf16", "residual": True, "i8": True},
        # a training or prefill batch
        {"name": "norm_batch", "op": "norm", "M": 16384, "H": 4096, "dtype": "bf16", "residual": True, "i8": False},
        # the gradients of a small ragged batch of odd width in fp32
        {"name": "norm_grad_odd", "op": "norm_grad", "M": 1237, "H": 1031, "dtype": "f32", "residual": False},
        # the gradients of the training batch
        {"name": "norm_grad_batch", "op": "norm_grad", "M": 16384, "H": 4096, "dtype": "bf16", "residual": True},
        # eight decoded tokens over 64 experts: the weights' bytes count
        {"name": "gated_decode", "op": "gated", "T": 8, "k": 4, "E": 64, "F": 1024, "K": 2048, "dtype": "bf16", "drop": 0.0, "act": "silu", "train": False},
        # a training step's forward pass
        {"name": "gated_train", "op": "gated", "T": 16384, "k": 2, "E": 16, "F": 2048, "K": 2048, "dtype": "bf16", "drop": 0.0, "act": "silu", "train": True},
        # a fine-tuning step's ragged batch, sizes that end inside every tile
        {"name": "gated_grad_ragged", "op": "gated_grad", "T": 1501, "k": 2, "E": 12, "F": 1000, "N": 776, "dtype": "f16", "drop": 0.05, "act": "gelu"},
        # a training step's backward pass
        {"name": "gated_grad_train", "op": "gated_grad", "T": 16384, "k": 2, "E": 16, "F": 2048, "N": 2048, "dtype": "bf16", "drop": 0.0, "act": "silu"},
        # a short prompt
        {"name": "embed_prompt", "op": "embed", "T": 301, "V": 50021, "H": 1002, "dtype": "f16", "pad": 0.0},
        # a training batch, padded
        {"name": "embed_batch", "op": "embed", "T": 16384, "V": 65536, "H": 4096, "dtype": "bf16", "pad": 0.05},
        # the table's gradient from a ragged batch, in fp32
        {"name": "embed_grad_odd", "op": "embed_grad", "T": 3001, "V": 20011, "H": 1002, "dtype": "f16", "out": "f32", "pad": 0.1},
        # a training step: most of the table gets zeros, a few ids hold hundreds of tokens
        {"name": "embed_grad_train", "op": "embed_grad", "T": 16384, "V": 65536, "H": 2048, "dtype": "bf16", "out": "bf16", "pad": 0.05},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width(lo, hi, step):  # an odd multiple of `step`, so never a round power of two
        return step * (2 * (spread(lo, hi) // (2 * step)) + 1)

    op = rng.choice(["norm", "norm_grad", "gated", "gated_grad", "embed", "embed_grad"])
    any_type = rng.choice(["f32", "bf16", "f16"])
    half = rng.choice(["bf16", "f16"])
    if op in ("norm", "norm_grad"):
        H = width(64, 8192, rng.choice([1, 2, 8, 64]))
        M = spread(1, min(65536, (1 << 25) // H)) | 1
        case = {"op": op, "M": M, "H": H, "dtype": any_type, "residual": rng.random() < 0.7}
        return case | {"i8": rng.random() < 0.4} if op == "norm" else case
    if op in ("gated", "gated_grad"):
        T, k, E = spread(1, 8192) | 1, rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 8, 12, 16, 32, 60, 64])
        F, R = width(128, 4096, 8), width(256, 4096, 8)
        E = min(E, max(1, (1 << 27) // (F * R)))
        k = min(k, E)
        k = min(k, max(1, int(1.2e11 / (T * F * R))))  # no more than the largest listed case
        case = {"op": op, "T": T, "k": k, "E": E, "F": F, "dtype": half, "drop": rng.choice([0.0, 0.03, 0.2]), "act": rng.choice(["silu", "silu", "gelu", "gelu_tanh"])}
        return case | ({"K": R, "train": rng.random() < 0.5} if op == "gated" else {"N": R})
    H = width(128, 4096, rng.choice([1, 2, 8]))
    V = spread(1000, 100000)
    if op == "embed":
        return {"op": op, "T": spread(1, 16384) | 1, "V": V, "H": H, "dtype": any_type, "pad": rng.choice([0.0, 0.1])}
    V = min(V, (1 << 27) // H)
    return {"op": op, "T": spread(1, 16384) | 1, "V": V, "H": H, "dtype": any_type, "out": rng.choice(["f32", any_type]), "pad": rng.choice([0.0, 0.1])}


def routing(case, g):
    """Expert ids [T, k] of a router with popular and rare experts: k distinct ones a token, some slots dropped (-1)."""
    T, k, E = case["T"], case["k"], case["E"]
    bias = -0.5 * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    bias = bias[torch.randperm(E, device="cuda", generator=g)]
    u = torch.rand(T, E, device="cuda", generator=g).clamp_(1e-7, 1 - 1e-7)
    ids = torch.topk(bias - torch.log(-torch.log(u)), k, dim=1).indices
    ids[torch.rand(T, k, device="cuda", generator=g) < case["drop"]] = -1
    return ids


def expert_offsets(ids, E):
    counts = (ids.reshape(-1) == torch.arange(E, device=ids.device)[:, None]).sum(1)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = torch.cumsum(counts, 0)
    return offsets


def zipf(V):
    """Share of each rank: a text's words."""
    p = 1.0 / (torch.arange(V, dtype=torch.float64) + 2.7)
    return p / p.sum()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DT[case["dtype"]]

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dt)

    st = {"op": case["op"], "dt": dt}
    if case["op"] in ("norm", "norm_grad"):
        M, H = case["M"], case["H"]
        X = torch.randn(M, H, device="cuda", generator=g)
        X[:, torch.randperm(H, device="cuda", generator=g)[: max(1, H // 128)]] *= 8  # the channels that activations have large values in
        X = X.to(dt)
        w = (1 + 0.2 * torch.randn(H, device="cuda", generator=g)).to(dt)
        st |= {"X": X, "w": w, "R": normal(M, H, scale=2.0) if case["residual"] else None}
        if case["op"] == "norm":
            return st | {"i8": case["i8"]}
        rstd = torch.rsqrt(X.double().square().mean(1) + EPS).float()  # as the forward pass left it
        return st | {"dY": normal(M, H), "rstd": rstd}
    if case["op"] in ("embed", "embed_grad"):
        T, V, H = case["T"], case["V"], case["H"]
        u = torch.rand(T, device="cuda", generator=g, dtype=torch.float64)
        rank = torch.searchsorted(torch.cumsum(zipf(V).cuda(), 0), u).clamp_(max=V - 1)
        ids = torch.randperm(V, device="cuda", generator=g)[rank]
        ids[torch.rand(T, device="cuda", generator=g) < case["pad"]] = 0
        st |= {"ids": ids, "V": V, "factor": H ** 0.5}
        if case["op"] == "embed":
            return st | {"W": normal(V, H, scale=H ** -0.5)}
        return st | {"dY": normal(T, H), "out": DT[case["out"]]}
    T, k, E, F = case["T"], case["k"], case["E"], case["F"]
    S = T * k
    st |= {"offsets": expert_offsets(routing(case, g), E), "act": case["act"]}
    if case["op"] == "gated":
        K = case["K"]
        return st | {"A": normal(S, K), "W": normal(E, 2 * F, K, scale=K ** -0.5), "train": case["train"]}
    N = case["N"]
    return st | {"dY": normal(S, N), "W": normal(E, N, F, scale=F ** -0.5), "H": normal(S, 2 * F)}


# ---------------------------------------------------------------- the plain forms


def padded(offsets, S):
    """Places [E, most rows an expert has] of each expert's rows, -1 past its last."""
    cap = max(1, int((offsets[1:] - offsets[:-1]).max()))
    at = offsets[:-1, None].long() + torch.arange(cap, device=offsets.device)
    return torch.where(at < offsets[1:, None], at, torch.full_like(at, -1))


def rows_of(M, at):
    """M's rows at `at` in 32 bits, zeros where that is -1."""
    return torch.where((at >= 0)[..., None], M[at.clamp(min=0)].float(), 0.0)


def scatter_rows(P, at, S):
    out = torch.zeros(S + 1, P.shape[-1], device=P.device)
    out[torch.where(at >= 0, at, torch.full_like(at, S)).reshape(-1)] = P.reshape(-1, P.shape[-1])
    return out[:S]


def activation(kind, x):
    """act(x) and its derivative."""
    if kind == "silu":
        s = 1 / (1 + torch.exp(-x))
        return x * s, s * (1 + x * (1 - s))
    if kind == "gelu":
        p = 0.5 * (1 + torch.erf(x * 0.5 ** 0.5))
        return x * p, p + x * torch.exp(-0.5 * x * x) * (0.5 / math.pi) ** 0.5
    c = (2 / math.pi) ** 0.5
    t = torch.tanh(c * (x + 0.044715 * x * x * x))
    return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)


def plain(st):
    op, dt = st["op"], st["dt"]
    if op == "norm":
        s = st["X"].float() if st["R"] is None else st["X"].float() + st["R"].float()
        y = s * torch.rsqrt(s.square().mean(1, keepdim=True) + EPS) * st["w"].float()
        S = None if st["R"] is None else s.to(dt)
        if not st["i8"]:
            return {"Y": y.to(dt), "S": S}
        scale = y.abs().amax(1) / 127.0
        q = torch.where(scale[:, None] > 0, torch.round(y / scale[:, None]), 0.0).to(torch.int8)
        return {"Y": (q.float() * scale[:, None]).to(torch.bfloat16), "scale": scale, "S": S}
    if op == "norm_grad":
        x, dy, rstd = st["X"].float(), st["dY"].float(), st["rstd"][:, None]
        xh, h = x * rstd, dy * st["w"].float()
        dx = rstd * (h - xh * (h * xh).mean(1, keepdim=True))
        if st["R"] is not None:
            dx = dx + st["R"].float()
        return {"dX": dx.to(dt), "dw": (dy * xh).sum(0)}
    if op == "embed":
        return (st["W"][st["ids"]].float() * st["factor"]).to(dt)
    if op == "embed_grad":
        dW = torch.zeros(st["V"], st["dY"].shape[1], device=st["dY"].device)
        dW.index_add_(0, st["ids"], st["dY"].float())
        dW[0] = 0.0  # the padding's row
        return (dW * st["factor"]).to(st["out"])
    if op == "gated":
        S, F = st["A"].shape[0], st["W"].shape[1] // 2
        at = padded(st["offsets"], S)
        P = torch.bmm(rows_of(st["A"], at), st["W"].float().transpose(1, 2))
        C = activation(st["act"], P[..., :F])[0] * P[..., F:]
        return {"C": scatter_rows(C, at, S).to(dt), "H": scatter_rows(P, at, S).to(dt) if st["train"] else None}
    S, F = st["dY"].shape[0], st["W"].shape[2]
    at = padded(st["offsets"], S)
    dC = torch.bmm(rows_of(st["dY"], at), st["W"].float())
    H = rows_of(st["H"], at)
    a, da = activation(st["act"], H[..., :F])
    U = H[..., F:]
    dH = torch.cat([dC * U * da, dC * a], -1)
    return {"dH": scatter_rows(dH, at, S).to(dt), "C": scatter_rows(a * U, at, S).to(dt)}


# ---------------------------------------------------------------- through the library


def library(st):
    from csr_bsr_spmv_gb300 import spx

    op = st["op"]
    if op == "norm":
        if st["i8"]:
            q, scale, S = spx.spx_rms_norm_i8(st["X"], st["w"], st["R"], eps=EPS)
            return {"Y": (q.float() * scale[:, None]).to(torch.bfloat16), "scale": scale, "S": S}
        Y, S, _ = spx.spx_rms_norm(st["X"], st["w"], st["R"], eps=EPS)
        return {"Y": Y, "S": S}
    if op == "norm_grad":
        dX, dw = spx.spx_rms_norm_grad(st["dY"], st["X"], st["rstd"], st["w"], dS=st["R"])
        return {"dX": dX, "dw": dw}
    if op == "embed":
        return spx.spx_embed(st["ids"], st["W"], st["factor"])
    if op == "embed_grad":
        return spx.spx_embed_grad(st["ids"], st["dY"], st["V"], st["factor"], padding=0, dtype=st["out"])
    if op == "gated":
        C, H = spx.spx_gemm_grouped_gated(st["offsets"], st["A"], st["W"], act=st["act"], grad=st["train"])
        return {"C": C, "H": H}
    dH, C = spx.spx_gemm_grouped_gated_grad(st["offsets"], st["dY"], st["W"], st["H"], act=st["act"])
    return {"dH": dH, "C": C}


def run(state):
    return library(state) if own else plain(state)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    b = BYTES[case["dtype"]]
    if case["op"] == "norm":
        n = case["M"] * case["H"]
        rows = 3 if case["residual"] else 1  # X, R, S
        return {"bytes": n * rows * b + n * (1 if case["i8"] else b) + case["H"] * b + 4 * case["M"] * case["i8"], "flops": 5 * n}
    if case["op"] == "norm_grad":
        n = case["M"] * case["H"]
        return {"bytes": n * (4 if case["residual"] else 3) * b + case["H"] * (b + 4) + 4 * case["M"], "flops": 9 * n}
    if case["op"] in ("embed", "embed_grad"):
        T, V, H = case["T"], case["V"], case["H"]
        if case["op"] == "embed":
            distinct = float((1 - (1 - zipf(V)) ** T).sum())
            return {"bytes": 8 * T + (distinct + T) * H * b, "flops": T * H}
        return {"bytes": 8 * T + T * (1 - case["pad"]) * H * b + V * H * BYTES[case["out"]], "flops": T * H}
    S, E, F = case["T"] * case["k"], case["E"], case["F"]
    rows = S * (1 - case["drop"])
    used = E * (1 - (1 - 1 / E) ** rows) if E > 1 else 1  # experts that have a row, about
    if case["op"] == "gated":
        K = case["K"]
        return {"bytes": (rows * K + used * 2 * F * K + S * F * (3 if case["train"] else 1)) * b, "flops": 4 * rows * F * K}
    N = case["N"]
    return {"bytes": (rows * N + used * F * N + rows * 2 * F + 3 * S * F) * b, "flops": 2 * rows * F * N}


# ---------------------------------------------------------------- 64 bits, from the definitions


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        s = st["X"].double() + (0 if st["R"] is None else st["R"].double())
        y = s / torch.sqrt((s * s).sum(1, keepdim=True) / case["H"] + EPS) * st["w"].double()
        S = s if st["R"] is not None else None
        if not case["i8"]:
            return {"Y": y, "S": S}
        scale = y.abs().max(1).values / 127
        return {"Y": torch.round(y / scale[:, None]) * scale[:, None], "scale": scale, "S": S}
    if case["op"] == "norm_grad":
        x, dy, w, r = st["X"].double(), st["dY"].double(), st["w"].double(), st["rstd"].double()
        dot = torch.einsum("mh,mh,h->m", dy, x, w)
        dx = r[:, None] * dy * w - (r ** 3 * dot / case["H"])[:, None] * x
        return {"dX": dx if st["R"] is None else dx + st["R"].double(), "dw": torch.einsum("mh,mh,m->h", dy, x, r)}
    if case["op"] == "embed":
        return st["W"].double().index_select(0, st["ids"]) * st["factor"]
    if case["op"] == "embed_grad":
        order = torch.argsort(st["ids"], stable=True)
        sums = torch.cat([torch.zeros(1, case["H"], dtype=torch.float64, device="cuda"), torch.cumsum(st["dY"].double()[order], 0)])
        ids = st["ids"][order]
        edge = torch.searchsorted(ids, torch.arange(case["V"] + 1, device="cuda"))
        dW = torch.empty(case["V"], case["H"], dtype=torch.float64, device="cuda")
        torch.sub(sums[edge[1:]], sums[edge[:-1]], out=dW)
        dW[0] = 0
        return dW * st["factor"]
    off, F, E = st["offsets"].tolist(), case["F"], case["E"]
    S = case["T"] * case["k"]

    def act(x):
        if case["act"] == "silu":
            return x * torch.sigmoid(x)
        if case["act"] == "gelu":
            return x * torch.special.ndtr(x)
        return x * torch.sigmoid((8 / math.pi) ** 0.5 * (x + 0.044715 * x ** 3))  # (1 + tanh z) / 2 = sigmoid(2 z)

    if case["op"] == "gated":
        C = torch.zeros(S, F, dtype=torch.float64, device="cuda")
        H = torch.zeros(S, 2 * F, dtype=torch.float64, device="cuda") if case["train"] else None
        for e in range(E):
            rows = slice(off[e], off[e + 1])
            P = st["A"][rows].double() @ st["W"][e].double().T
            C[rows] = act(P[:, :F]) * P[:, F:]
            if H is not None:
                H[rows] = P
        return {"C": C, "H": H}
    dH = torch.zeros(S, 2 * F, dtype=torch.float64, device="cuda")
    C = torch.zeros(S, F, dtype=torch.float64, device="cuda")
    for e in range(E):
        rows = slice(off[e], off[e + 1])
        with torch.enable_grad():
            h = st["H"][rows].double().requires_grad_()
            c = act(h[:, :F]) * h[:, F:]
            dH[rows] = torch.autograd.grad(c, h, st["dY"][rows].double() @ st["W"][e].double())[0]
        C[rows] = c.detach()
    return {"dH": dH, "C": C}
