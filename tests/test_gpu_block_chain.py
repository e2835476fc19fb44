"""The norm, the gated products and the embedding together, as a block uses them."""
import importlib.util
import math
import os

import pytest
import torch

from block_util import BF16, F16, normal, offsets_of, whole
from csr_bsr_spmv_gb300 import spx

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "gated_block.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("gated_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_the_example_runs(example):
    losses, off = example.main(tokens=300, vocab=200, width=64, inner=96, experts=4, k=2, steps=3, say=lambda *a: None)
    assert len(losses) == 3 and all(math.isfinite(x) for x in losses) and math.isfinite(off)


@pytest.mark.parametrize("T,V,width,inner,E,k", [(1, 7, 64, 48, 3, 2), (130, 50, 72, 40, 4, 2), (700, 90, 66, 37, 5, 3)])
def test_the_blocks_gradients(example, T, V, width, inner, E, k):
    """Against autograd in 64 bits on the same weights and routing.  On the way from the loss back to the table there are
    16 roundings to fp16 (2^-11 each, relative to values of one size) and as many on the way there; what follows one
    enlarges it less than fourfold for rows of unit size: 32 * 4 * 2^-11 of the gradient's norm."""
    torch.manual_seed(T)
    table = normal(1, V, width, dtype=F16, scale=width ** -0.5).requires_grad_()
    n1, n2 = ((1 + 0.2 * normal(i, width)).to(F16).requires_grad_() for i in (2, 3))
    W1 = normal(4, E, 2 * inner, width, dtype=F16, scale=width ** -0.5).requires_grad_()
    W2 = normal(5, E, width, inner, dtype=F16, scale=inner ** -0.5).requires_grad_()
    ids = torch.randint(0, V, (T,), device="cuda")
    expert = torch.stack([torch.randperm(E, device="cuda")[:k] for _ in range(T)])
    weight = torch.softmax(normal(6, T, k), 1).requires_grad_()
    out = normal(7, T, width)
    X = example.Embed.apply(ids, table, width ** 0.5)
    Y, X = example.AddNorm.apply(X, None, n1)
    Z, S = example.AddNorm.apply(example.GatedExperts.apply(Y, expert, weight, W1, W2), X, n2)
    leaves = [table, n1, n2, weight, W1, W2]
    got = torch.autograd.grad((Z.float() * out).sum() + (S.float() * out).sum(), leaves)
    assert spx.spx_last_device_error() == 0

    wide = [t.detach().double().requires_grad_() for t in leaves]
    tab, m1, m2, wt, V1, V2 = wide

    def norm(x, w):
        return x / torch.sqrt(x.square().mean(1, keepdim=True) + 1e-6) * w

    x = tab[ids] * width ** 0.5
    y = norm(x, m1)
    h = torch.einsum("tkfc,tc->tkf", V1[expert], y)
    c = torch.nn.functional.silu(h[..., :inner]) * h[..., inner:]
    s = x + (torch.einsum("tkcf,tkf->tkc", V2[expert], c) * wt[..., None]).sum(1)
    want = torch.autograd.grad((norm(s, m2) * out.double()).sum() + (s * out.double()).sum(), wide)
    for g, w, what in zip(got, want, ("table", "norm1", "norm2", "weight", "W1", "W2")):
        rel = ((g.double() - w).norm() / w.norm()).item()
        assert rel <= 32 * 4 * 2.0 ** -11, (what, rel)


@pytest.mark.parametrize("graph", [False, True])
def test_back_to_back_calls_see_the_arrays_of_their_own_turn(graph):
    """Lookup, norm, gated product, its gradient and the table's gradient over the same buffers again and again, nothing
    else on the stream: each turn's results are those of its own ids.  Every kernel starts before the one ahead of it
    has ended, so a read ahead of its wait would show here."""
    T, V, H, F, E, turns = 500, 300, 64, 48, 3, 12
    off = offsets_of([100, 0, 350])
    torch.manual_seed(V)
    table, w = normal(1, V, H, dtype=BF16), (1 + 0.2 * normal(2, H)).to(BF16)
    W1, W2 = normal(3, E, 2 * F, H, dtype=BF16, scale=0.1), normal(4, E, H, F, dtype=BF16, scale=0.1)
    all_ids = torch.randint(0, V, (turns, T), device="cuda")
    ids = torch.zeros(T, dtype=torch.int64, device="cuda")

    def turn():
        X = spx.spx_embed(ids, table, 2.0)
        Y, S, rstd = spx.spx_rms_norm(X, w, X, grad=True)
        C, Hf = spx.spx_gemm_grouped_gated(off, Y, W1, grad=True)
        Z = spx.spx_gemm_grouped(off, C, W2)
        dH, C2 = spx.spx_gemm_grouped_gated_grad(off, Z, W2, Hf)
        dY = spx.spx_gemm_grouped(off, dH, W1, layout="kn")
        dX, dw = spx.spx_rms_norm_grad(dY, S, rstd, w, dS=Z)
        q, qs, _ = spx.spx_rms_norm_i8(S, w)
        return [Y, C, dH, C2, dX, dw, q, qs, spx.spx_embed_grad(ids, dX, V, 2.0, padding=5)]

    want = []
    for i in range(turns):
        ids.copy_(all_ids[i])
        torch.cuda.synchronize()
        got = turn()
        torch.cuda.synchronize()
        want.append([t.clone() for t in got])
    if graph:
        turn()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = []
            for i in range(turns):
                ids.copy_(all_ids[i])
                out.append([t.clone() for t in turn()])
        all_ids.copy_(all_ids.clone())
        g.replay()
        g.replay()
    else:
        out = []
        for i in range(turns):
            ids.copy_(all_ids[i])
            out.append(turn())
    torch.cuda.synchronize()
    for i in range(turns):
        for n, (a, b) in enumerate(zip(want[i], out[i])):
            assert torch.equal(a, b), (i, n)


def test_two_graphs_over_one_scratch():
    """Two captured gradients that the caller gives the same workspace, replayed in turn."""
    T, V, H = 3000, 400, 72
    torch.manual_seed(V)
    ids = [torch.randint(0, V, (T,), device="cuda") for _ in range(2)]
    dY = [whole(i, T, H, dtype=BF16) for i in range(2)]
    lib = spx._lib()
    scratch = torch.empty(max(lib.spx_embed_grad_scratch_bytes(T, H), lib.spx_rms_norm_grad_scratch_bytes(T, H)), dtype=torch.uint8, device="cuda")
    rstd = torch.ones(T, device="cuda")

    def run(i):
        return [spx.spx_embed_grad(ids[i], dY[i], V, scratch=scratch), *spx.spx_rms_norm_grad(dY[i], dY[1 - i], rstd, scratch=scratch)]

    want = [run(i) for i in range(2)]
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run(i)
        graphs.append((g, out))
    for _ in range(3):
        for g, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    for w, (_, out) in zip(want, graphs):
        assert all(torch.equal(a, b) for a, b in zip(w, out))


def test_wrong_offsets_are_reported_by_the_checked_build():
    S, E, H, F = 200, 3, 64, 48
    A, W1, W2 = normal(1, S, H, dtype=BF16), normal(2, E, 2 * F, H, dtype=BF16), normal(3, E, H, F, dtype=BF16)
    Hf = normal(4, S, 2 * F, dtype=BF16)

    def calls(off):
        return [*spx.spx_gemm_grouped_gated(off, A, W1, grad=True), *spx.spx_gemm_grouped_gated_grad(off, A, W2, Hf),
                *spx.spx_gemm_grouped_gated(off, A[:, 1:], W1[:, :, 1:], grad=True),
                *spx.spx_gemm_grouped_gated_grad(off, A[:, 1:], W2[:, 1:], Hf)]

    right = offsets_of([50, 0, 120])
    want = calls(right)
    with spx.checked_build():
        got = calls(right)
        assert spx.spx_last_device_error() == 0
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        for wrong in ([0, 50, 300, 300], [0, 80, 40, 170], [-1, 50, 60, 170]):
            off = torch.tensor(wrong, dtype=torch.int32, device="cuda")
            for fn in (lambda: spx.spx_gemm_grouped_gated(off, A, W1), lambda: spx.spx_gemm_grouped_gated_grad(off, A, W2, Hf),
                       lambda: spx.spx_gemm_grouped_gated(off, A[:, 1:], W1[:, :, 1:])):
                fn()
                assert spx.spx_last_device_error() == -2, wrong
                assert spx.spx_last_device_error() == 0
