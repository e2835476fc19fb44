"""The root-mean-square norm and its gradient on the GPU against 64-bit formulas.

Tolerances, fixed from the formats before any run, u = 2^-24.  The fp32 sum of H squares is off by at most H u of itself
in any order, which its root halves; the root, the quotients and the three products of y = s rstd w add 8 u, s itself one:
(H / 2 + 10) u |y|, then the output's rounding.  In the gradient, with g = dy w and n = s rstd, the mean of H products is
off by (H + 4) u mean|g n|, and the rest by 8 u of each term.  The weights' gradient sums M products.  A code of the
8-bit output is the quotient y / scale, at most 127, rounded: off by half, and by 127 (H + 24) u where the quotient is
(the errors of y and of the largest y)."""
import numpy as np
import pytest
import torch

from block_util import BF16, F16, F32, TINY, U, between, close, gen, normal, padded
from csr_bsr_spmv_gb300 import spx

pytestmark = pytest.mark.gpu
EPS = 1e-5


def norm64(X, R, w, eps=EPS):
    s = X.double() + (R.double() if R is not None else 0)
    rstd = 1 / torch.sqrt((s * s).sum(1) / X.shape[1] + eps)
    return s, rstd, s * rstd[:, None] * (w.double() if w is not None else 1)


def grad64(dY, S, rstd, w, dS):
    n, g = S.double() * rstd.double()[:, None], dY.double() * (w.double() if w is not None else 1)
    r = rstd.double()[:, None]
    dX = r * (g - n * (g * n).mean(1, keepdim=True))
    near = r * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    if dS is not None:
        dX, near = dX + dS.double(), near + dS.double().abs()
    return dX, near, (dY.double() * n).sum(0), (dY.double() * n).abs().sum(0)


SIZES = [(1, 1), (1, 4096), (3, 7), (2, 64), (1, 128), (5, 130), (700, 128), (33, 1002), (2, 1031), (64, 2048), (3, 4096), (1217, 72),
         (9, 4097), (2, 5000), (4, 8192), (2, 16384), (3, 16385), (2, 20000), (1, 32768), (40000, 16), (3000, 4104), (5, 8195), (500, 33), (3, 20001), (2, 9001), (2, 32767)]


@pytest.mark.parametrize("M,H", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_is_the_formula(M, H, dtype, residual):
    X, R = normal(M + H, M, H, dtype=dtype), normal(H, M, H, dtype=dtype, scale=2) if residual else None
    w = (1 + 0.3 * normal(1, H)).to(dtype)
    Y, S, rstd = spx.spx_rms_norm(X, w, R, eps=EPS, grad=True)
    s, r, y = norm64(X, R, w)
    close(Y, y, (H / 2 + 10) * U * y.abs(), "Y")
    close(rstd, r, (H / 2 + 8) * U * r, "rstd")
    assert (S is None) == (not residual)
    if residual:
        close(S, s, U * s.abs(), "S")
    Q, scale, S8 = spx.spx_rms_norm_i8(X, w, R, eps=EPS)
    top = y.abs().max(1).values / 127
    close(scale, top, (H / 2 + 12) * U * top, "scale")
    assert ((Q.double() - y / top[:, None]).abs() <= 0.5 + 127 * (H + 24) * U).all()
    assert Q.abs().max() <= 127 and (not residual or torch.equal(S8, S))


@pytest.mark.parametrize("M,H", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("residual", [False, True])
def test_gradient_is_the_formula(M, H, dtype, residual):
    S, dY, w = normal(M, M, H, dtype=dtype), normal(H + 1, M, H, dtype=dtype), (1 + 0.3 * normal(2, H)).to(dtype)
    dS = normal(7, M, H, dtype=dtype) if residual else None
    rstd = (1 / torch.sqrt(S.double().square().mean(1) + EPS)).float()
    dX, dw = spx.spx_rms_norm_grad(dY, S, rstd, w, dS=dS)
    ref, near, rw, nw = grad64(dY, S, rstd, w, dS)
    close(dX, ref, (H + 12) * U * near, "dX")
    close(dw, rw, (M + 4) * U * nw, "dweight")
    again, dw2 = spx.spx_rms_norm_grad(dY, S, rstd, w, dS=dS)
    assert torch.equal(again, dX) and torch.equal(dw, dw2)
    only, none = spx.spx_rms_norm_grad(dY, S, rstd, w, dS=dS, dweight=False)
    assert none is None and torch.equal(only, dX)


@pytest.mark.parametrize("dtype,wide", [(F32, False), (BF16, False), (BF16, True), (F16, True)])
@pytest.mark.parametrize("pad", [1, 2, 4, 8, 24])
@pytest.mark.parametrize("H", [264, 1002, 5, 4500])
def test_pitches_and_bases_of_any_alignment(dtype, wide, pad, H):
    M = 37
    X, R, dY = (padded(normal(i, M, H, dtype=dtype), pad) for i in range(3))
    w = padded((1 + 0.3 * normal(3, 1, H)).to(F32 if wide else dtype), pad)[0]
    Y, S = (padded(torch.zeros(M, H, dtype=dtype, device="cuda"), pad) for _ in range(2))
    Q = padded(torch.zeros(M, H, dtype=torch.int8, device="cuda"), pad)
    edges = [between(t, pad) for t in (Y, S, Q)]
    _, _, rstd = spx.spx_rms_norm(X, w, R, eps=EPS, Y=Y, S=S, grad=True)
    s, r, y = norm64(X, R, w)
    close(Y, y, (H / 2 + 10) * U * y.abs(), "Y")
    close(S, s, U * s.abs(), "S")
    spx.spx_rms_norm_i8(X, w, R, eps=EPS, Q=Q)
    Q0, _, _ = spx.spx_rms_norm_i8(X.contiguous(), w.clone(), R.contiguous(), eps=EPS)
    assert (Q.int() - Q0.int()).abs().max() <= 1
    dX = padded(torch.zeros(M, H, dtype=dtype, device="cuda"), pad)
    edges.append(between(dX, pad))
    _, dw = spx.spx_rms_norm_grad(dY, S, rstd, w, dS=R, dX=dX)
    ref, near, rw, nw = grad64(dY, S, rstd, w, R)
    close(dX, ref, (H + 12) * U * near, "dX")
    close(dw, rw, (M + 4) * U * nw, "dweight")
    for t, e in zip((Y, S, Q, dX), edges):
        assert torch.equal(between(t, pad).nan_to_num(5), e.nan_to_num(5))


@pytest.mark.parametrize("dtype,wide", [(F32, False), (BF16, True)])
@pytest.mark.parametrize("pad", [1, 2, 4])
@pytest.mark.parametrize("H", [9000, 16384, 17000])
def test_long_rows_of_any_alignment(dtype, wide, pad, H):
    test_pitches_and_bases_of_any_alignment(dtype, wide, pad, H)


@pytest.mark.parametrize("H", [7, 40, 41, 1000, 1001, 1002, 4095, 6000, 6001, 9001, 16401, 20000])
def test_outputs_over_their_inputs(H):
    """S over R, Y over X; dX over dY, over dS and over S: rows on 16- and 4-byte boundaries and on neither."""
    M = 900 if H < 2000 else 320
    X, R, w = normal(1, M, H, dtype=BF16), normal(2, M, H, dtype=BF16), normal(3, H, dtype=BF16)
    Y, S, rstd = spx.spx_rms_norm(X, w, R, grad=True)
    x, r = X.clone(), R.clone()
    spx.spx_rms_norm(x, w, r, Y=x, S=r)
    assert torch.equal(x, Y) and torch.equal(r, S)
    x, r = X.clone(), R.clone()
    spx.spx_rms_norm(x, w, r, Y=r, S=x)
    assert torch.equal(r, Y) and torch.equal(x, S)
    r = R.clone()
    Q, scale, _ = spx.spx_rms_norm_i8(X, w, r, S=r)
    assert torch.equal(r, S) and torch.equal(Q, spx.spx_rms_norm_i8(X, w, R)[0])
    dY, dS = normal(4, M, H, dtype=BF16), normal(5, M, H, dtype=BF16)
    dX, dw = spx.spx_rms_norm_grad(dY, S, rstd, w, dS=dS)
    for i in range(3):
        t = [dY.clone(), S.clone(), dS.clone()]
        out, dw2 = spx.spx_rms_norm_grad(t[0], t[1], rstd, w, dS=t[2], dX=t[i])
        assert out is t[i] and torch.equal(out, dX) and torch.equal(dw, dw2)


def test_no_weights_and_no_rows():
    X = normal(1, 9, 300)
    Y, _, _ = spx.spx_rms_norm(X, eps=EPS)
    _, r, y = norm64(X, None, None)
    close(Y, y, 160 * U * y.abs())
    dX, dw = spx.spx_rms_norm_grad(X, X, r.float(), None)
    ref, near, rw, nw = grad64(X, X, r.float(), None, None)
    close(dX, ref, 312 * U * near)
    close(dw, rw, 13 * U * nw)
    E = torch.empty(0, 300, device="cuda")
    before = spx.launch_count()
    assert spx.spx_rms_norm(E)[0].shape == (0, 300)
    dw = spx.spx_rms_norm_grad(E, E, torch.empty(0, device="cuda"))[1]
    assert torch.equal(dw, torch.zeros(300, device="cuda"))
    assert spx.launch_count() == before


def test_copied_sum_without_a_residual():
    X = normal(1, 9, 300, dtype=F16)
    S = torch.zeros_like(X)
    assert spx.spx_rms_norm(X, S=S)[1] is S and torch.equal(S, X)


def test_rows_of_zeros_infinities_and_nan():
    """Other rows are not touched by a bad one; a row of zeros is zeros, with scale 0."""
    X = normal(1, 6, 520, dtype=BF16)
    clean = spx.spx_rms_norm(X)[0]
    Qc, sc, _ = spx.spx_rms_norm_i8(X)
    X[1], X[3, 7], X[4, 519] = 0, float("inf"), float("nan")
    Y = spx.spx_rms_norm(X)[0]
    Q, scale, _ = spx.spx_rms_norm_i8(X)
    for i in (0, 2, 5):
        assert torch.equal(Y[i], clean[i]) and torch.equal(Q[i], Qc[i]) and scale[i] == sc[i]
    assert not Y[1].any() and not Q[1].any() and scale[1] == 0
    assert Y[3, 7].isnan() and not Y[3, :7].any()       # infinity times a root of zero
    assert Y[4].isnan().all()
    assert scale[3].isnan() and scale[4].isnan() and not Q[3].any() and not Q[4].any()


def test_gradient_by_differences():
    """(L(x + h) - L(x - h)) / 2h of L = <Y, dY> + <S, dS> in 64 bits: off by h^2 / 6 times the third derivative, here
    below 1e-7, and by the roundoff 1e-16 / h."""
    M, H, h = 4, 23, 1e-5
    X, w = normal(1, M, H), 1 + 0.3 * normal(2, H)
    dY, dS = normal(3, M, H), normal(4, M, H)
    _, _, rstd = spx.spx_rms_norm(X, w, eps=EPS, grad=True)
    dX, dw = spx.spx_rms_norm_grad(dY, X, rstd, w, dS=dS)

    def loss(x, v):
        s = x
        return ((s / torch.sqrt(s.square().mean(1, keepdim=True) + EPS) * v) * dY.double()).sum() + (s * dS.double()).sum()

    x, v = X.double(), w.double()
    for i, j in [(0, 0), (1, 5), (3, 22)]:
        d = torch.zeros_like(x)
        d[i, j] = h
        assert abs((loss(x + d, v) - loss(x - d, v)) / (2 * h) - dX[i, j]) <= 1e-5
        e = torch.zeros_like(v)
        e[j] = h
        assert abs((loss(x, v + e) - loss(x, v - e)) / (2 * h) - dw[j]) <= 1e-5


def test_offsets_past_32_bits():
    """A matrix of more than 2^31 values: the last rows are right."""
    M, H = (1 << 31) // 4096 + 40, 4096
    X = torch.zeros(M, H, dtype=BF16, device="cuda")
    X[-3:] = normal(1, 3, H, dtype=BF16)
    Y, _, _ = spx.spx_rms_norm(X, eps=EPS, Y=X)
    assert not Y[0].any()
    X3 = normal(1, 3, H, dtype=BF16)
    close(Y[-3:], norm64(X3, None, None)[2], (H / 2 + 10) * U * norm64(X3, None, None)[2].abs())


@pytest.mark.parametrize("M,H", [(7, 600), (3000, 512)])
def test_streams_and_graphs(M, H):
    """On another stream, and captured with inputs that change between replays; two graphs with their own scratch."""
    X, R, w = normal(1, M, H, dtype=BF16), normal(2, M, H, dtype=BF16), normal(3, H, dtype=BF16)
    dY = normal(4, M, H, dtype=BF16)

    def run():
        Y, S, rstd = spx.spx_rms_norm(X, w, R, grad=True)
        Q, scale, _ = spx.spx_rms_norm_i8(X, w, R)
        return [Y, S, rstd, Q, scale, *spx.spx_rms_norm_grad(dY, S, rstd, w, dS=R)]

    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Y2, S2, r2 = spx.spx_rms_norm(X, w, R, grad=True, stream=side)
    dX2, dw2 = spx.spx_rms_norm_grad(dY, S2, r2, w, dS=R, stream=side)
    side.synchronize()
    assert torch.equal(Y2, want[0]) and torch.equal(dX2, want[5]) and torch.equal(dw2, want[6])
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
        graphs.append((g, out))
    for seed in (10, 20):
        X.copy_(normal(seed, M, H, dtype=BF16))
        dY.copy_(normal(seed + 1, M, H, dtype=BF16))
        for g, out in graphs:
            g.replay()
        torch.cuda.synchronize()
        for a, *rest in zip(run(), *(out for _, out in graphs)):
            assert all(torch.equal(a, b) for b in rest)
