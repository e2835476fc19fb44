"""A block with gated routed experts between its table and its output: trained in bf16, its output then served in 8 bits.

Tokens look up their rows of a table; a norm and a layer of routed experts with a gate follow, whose result is added to
the rows; a second norm and the table itself give the scores of the next token:

    python examples/gated_block.py [--tokens 4096 --vocab 4096 --width 512 --inner 768 --experts 8 --k 2 --steps 40]

trains it for a few steps on a made-up language, in which a token's successor is mostly a fixed one (every lookup, norm,
product and gradient runs in the library), and compares the scores from the 8-bit norm and table with those in bf16.
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from csr_bsr_spmv_gb300 import spx  # noqa: E402


class Embed(torch.autograd.Function):
    """Y[t] = scale * W[ids[t]]."""

    @staticmethod
    def forward(ctx, ids, W, scale):
        ctx.save_for_backward(ids)
        ctx.rows, ctx.scale = W.shape[0], scale
        return spx.spx_embed(ids, W, scale)

    @staticmethod
    def backward(ctx, dY):
        ids, = ctx.saved_tensors
        return None, spx.spx_embed_grad(ids, dY.contiguous(), ctx.rows, ctx.scale), None


class AddNorm(torch.autograd.Function):
    """The stream S = X + R and its norm Y; without R the stream is X."""

    @staticmethod
    def forward(ctx, X, R, weight):
        Y, S, rstd = spx.spx_rms_norm(X, weight, R, grad=True)
        S = X if S is None else S
        ctx.save_for_backward(S, rstd, weight)
        ctx.residual = R is not None
        return Y, S

    @staticmethod
    def backward(ctx, dY, dS):
        S, rstd, weight = ctx.saved_tensors
        dX, dweight = spx.spx_rms_norm_grad(dY.contiguous(), S, rstd, weight, dS=dS.contiguous())
        return dX, dX if ctx.residual else None, dweight.to(weight.dtype)


class GatedExperts(torch.autograd.Function):
    """Y[t] = sum_j weight[t, j] * W2_e (silu(Wg_e X[t]) * Wu_e X[t]), e = expert[t, j]; W1 = [Wg; Wu]."""

    @staticmethod
    def forward(ctx, X, expert, weight, W1, W2):
        r = spx.spx_route_build(expert, W1.shape[0])
        Xs = spx.spx_route_gather(r, X)
        C, H = spx.spx_gemm_grouped_gated(r.offsets, Xs, W1, grad=True)
        Ys = spx.spx_gemm_grouped(r.offsets, C, W2)
        ctx.route = r
        ctx.save_for_backward(Xs, H, Ys, weight, W1, W2)
        return spx.spx_route_combine(r, Ys, weight)

    @staticmethod
    def backward(ctx, dY):
        r = ctx.route
        Xs, H, Ys, weight, W1, W2 = ctx.saved_tensors
        dYs, dweight = spx.spx_route_combine_grad(r, dY.contiguous(), Ys, weight)
        dH, C = spx.spx_gemm_grouped_gated_grad(r.offsets, dYs, W2, H)
        dW2 = spx.spx_gemm_grouped_wgrad(r.offsets, dYs, C)
        dW1 = spx.spx_gemm_grouped_wgrad(r.offsets, dH, Xs)
        dXs = spx.spx_gemm_grouped(r.offsets, dH, W1, layout="kn")
        return spx.spx_route_combine(r, dXs), None, dweight, dW1, dW2


def route(X, Wr, k):
    """The router: expert ids [T, k] and their weights, which carry the gradient to Wr."""
    top, expert = torch.topk(X.float() @ Wr, k, dim=1)
    return expert, torch.softmax(top, dim=1)


def stream(ids, table, norm1, norm2, Wr, W1, W2, k):
    """The last norm's output and the stream before it."""
    X = Embed.apply(ids, table, table.shape[1] ** 0.5)
    Y, X = AddNorm.apply(X, None, norm1)
    expert, weight = route(Y, Wr, k)
    return AddNorm.apply(GatedExperts.apply(Y, expert, weight, W1, W2), X, norm2)


def main(tokens=4096, vocab=4096, width=512, inner=768, experts=8, k=2, steps=40, seed=0, say=print):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale):
        return torch.randn(*shape, device="cuda", generator=g) * scale

    table = normal(vocab, width, scale=width ** -0.5).bfloat16().requires_grad_()
    norm1, norm2 = (torch.ones(width, device="cuda", dtype=torch.bfloat16).requires_grad_() for _ in range(2))
    Wr = normal(width, experts, scale=width ** -0.5).requires_grad_()
    W1 = normal(experts, 2 * inner, width, scale=width ** -0.5).bfloat16().requires_grad_()
    W2 = normal(experts, width, inner, scale=inner ** -0.5).bfloat16().requires_grad_()
    weights = [table, norm1, norm2, Wr, W1, W2]
    successor = torch.randperm(vocab, device="cuda", generator=g)
    opt = torch.optim.Adam(weights, lr=1e-3)
    losses = []

    def batch():
        ids = torch.randint(0, vocab, (tokens,), device="cuda", generator=g)
        noise = torch.randint(0, vocab, (tokens,), device="cuda", generator=g)
        return ids, torch.where(torch.rand(tokens, device="cuda", generator=g) < 0.9, successor[ids], noise)

    for step in range(steps):
        ids, target = batch()
        Y, _ = stream(ids, *weights, k)
        loss = F.cross_entropy((Y @ table.t()).float(), target)
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        losses.append(loss.detach())
        if step % 10 == 0 or step == steps - 1:
            say(f"step {step:3d}  loss {loss.item():.4f}")
    with torch.no_grad():
        codes, scales = spx.spx_quant_rows_i8(table)
        ids, _ = batch()
        Y, S = stream(ids, *weights, k)
        want = (Y @ table.t()).float()
        q, qs, _ = spx.spx_rms_norm_i8(S, norm2)
        got = spx.spx_gemm_i8(q, qs, codes, scales)
        off = ((got - want).norm() / want.norm()).item()
        say(f"8-bit output: {100 * off:.2f}% off the bf16 scores")
    torch.cuda.synchronize()
    assert spx.spx_last_device_error() == 0
    return [float(x) for x in losses], off


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 4096), ("vocab", 4096), ("width", 512), ("inner", 768), ("experts", 8), ("k", 2), ("steps", 40)):
        p.add_argument(f"--{name}", type=int, default=value)
    main(**vars(p.parse_args()))
