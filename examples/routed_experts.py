"""A layer of routed experts: trained in bf16, then served from 8-bit weights.

A router sends each token to k of E experts; an expert is two matrices with a
SiLU between them.  The tokens' slots are sorted by expert, gathered into that
order, multiplied by their experts' matrices and returned weighted:

    python examples/routed_experts.py [--tokens 4096 --width 1024 --inner 2048 --experts 16 --k 2 --steps 40]

trains the layer on a made-up target for a few steps (every product, gather,
return and gradient runs in the library), quantises the experts to 8 bits with
a scale a channel, and compares the quantised layer with the trained one on a
batch and on a single token.
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from csr_bsr_spmv_gb300 import spx  # noqa: E402


class RoutedExperts(torch.autograd.Function):
    """Y[t] = sum_j weight[t, j] * W2_e silu(W1_e X[t]), e = expert[t, j]; an expert id of -1 drops the slot."""

    @staticmethod
    def forward(ctx, X, expert, weight, W1, W2):
        r = spx.spx_route_build(expert, W1.shape[0])
        Xs = spx.spx_route_gather(r, X)
        h = spx.spx_gemm_grouped(r.offsets, Xs, W1)
        a = F.silu(h)
        Ys = spx.spx_gemm_grouped(r.offsets, a, W2)
        ctx.route = r
        ctx.save_for_backward(Xs, h, a, Ys, weight, W1, W2)
        return spx.spx_route_combine(r, Ys, weight)

    @staticmethod
    def backward(ctx, dY):
        r = ctx.route
        Xs, h, a, Ys, weight, W1, W2 = ctx.saved_tensors
        dYs, dweight = spx.spx_route_combine_grad(r, dY.contiguous(), Ys, weight)
        da = spx.spx_gemm_grouped(r.offsets, dYs, W2, layout="kn")
        dW2 = spx.spx_gemm_grouped_wgrad(r.offsets, dYs, a)
        s = torch.sigmoid(h.float())
        dh = (da.float() * s * (1 + h.float() * (1 - s))).to(h.dtype)
        dXs = spx.spx_gemm_grouped(r.offsets, dh, W1, layout="kn")
        dW1 = spx.spx_gemm_grouped_wgrad(r.offsets, dh, Xs)
        return spx.spx_route_combine(r, dXs), None, dweight, dW1, dW2


def route(X, Wr, k):
    """The router: expert ids [T, k] and their weights, which carry the gradient to Wr."""
    logits = X.float() @ Wr
    top, expert = torch.topk(logits, k, dim=1)
    return expert, torch.softmax(top, dim=1)


def quantise(W):
    """[E, N, K] -> 8-bit codes of the same shape and a scale for each expert's channels."""
    E, N, K = W.shape
    q, s = spx.spx_quant_rows_i8(W.reshape(E * N, K))
    return q.view(E, N, K), s.view(E, N)


def serve(X, expert, weight, W1, W2):
    """The layer's forward pass on quantised experts (W1 and W2: codes and scales), activations quantised a token."""
    r = spx.spx_route_build(expert, W1[0].shape[0])
    q, s = spx.spx_quant_rows_i8(spx.spx_route_gather(r, X))
    h = spx.spx_gemm_i8(q, s, *W1, offsets=r.offsets, dtype=X.dtype)
    q, s = spx.spx_quant_rows_i8(F.silu(h))
    return spx.spx_route_combine(r, spx.spx_gemm_i8(q, s, *W2, offsets=r.offsets, dtype=X.dtype), weight)


def main(tokens=4096, width=1024, inner=2048, experts=16, k=2, steps=40, seed=0, say=print):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale):
        return torch.randn(*shape, device="cuda", generator=g) * scale

    Wr = normal(width, experts, scale=width ** -0.5).requires_grad_()
    W1 = normal(experts, inner, width, scale=width ** -0.5).bfloat16().requires_grad_()
    W2 = normal(experts, width, inner, scale=inner ** -0.5).bfloat16().requires_grad_()
    target = normal(width, width, scale=width ** -0.5)
    opt = torch.optim.Adam([Wr, W1, W2], lr=1e-3)
    losses = []
    for step in range(steps):
        X = normal(tokens, width, scale=1.0).bfloat16()
        expert, weight = route(X, Wr, k)
        Y = RoutedExperts.apply(X, expert, weight, W1, W2)
        loss = F.mse_loss(Y.float(), torch.relu(X.float() @ target))
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        losses.append(loss.detach())
        if step % 10 == 0 or step == steps - 1:
            say(f"step {step:3d}  loss {loss.item():.4f}")
    with torch.no_grad():
        Q1, Q2 = quantise(W1), quantise(W2)
        off = {}
        for name, n in (("batch", tokens), ("single token", 1)):
            X = normal(n, width, scale=1.0).bfloat16()
            expert, weight = route(X, Wr, k)
            Y = RoutedExperts.apply(X, expert, weight, W1, W2).float()
            Y8 = serve(X, expert, weight, Q1, Q2).float()
            off[name] = ((Y8 - Y).norm() / Y.norm()).item()
            say(f"8-bit experts, {name}: {100 * off[name]:.2f}% off the bf16 layer")
    torch.cuda.synchronize()
    assert spx.spx_last_device_error() == 0
    return [float(x) for x in losses], off


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 4096), ("width", 1024), ("inner", 2048), ("experts", 16), ("k", 2), ("steps", 40)):
        p.add_argument(f"--{name}", type=int, default=value)
    main(**vars(p.parse_args()))
