"""Experts with a gate and their gradient on the GPU against 64-bit formulas.

Tolerances, fixed from the formats before any run, u = 2^-24.  A sum of n products is off by n u sum|products| in any
order, twice that where additions are cut instead of rounded: the tensor cores' bound of the routed experts' tests.  The
activations are x p(x) with |act'| <= 1.13; CUDA's expf and normcdff are off by 2 and 5 units in the last place, so act
is off by 16 u |act| + 2 u |x| and its slope by 16 u (1 + |x dz|), dz the slope of the logistic function's argument.
What is stored is rounded once to its type."""
import numpy as np
import pytest
import torch

from block_util import BF16, F16, F32, U, between, close, normal, offsets_of, padded
from csr_bsr_spmv_gb300 import spx

pytestmark = pytest.mark.gpu
ACTS = ["silu", "gelu", "gelu_tanh"]


def act64(kind, x):
    """act, act' and the slope of the logistic function's argument (1 for the others), in 64 bits."""
    one = torch.ones_like(x)
    if kind == "gelu":
        p = torch.special.erfc(-x / 2 ** 0.5) / 2  # torch's ndtr loses the left tail: 0 at -12 for 1.8e-33
        return x * p, p + x * torch.exp(-x * x / 2) / (2 * np.pi) ** 0.5, one
    c = (8 / np.pi) ** 0.5
    z, dz = (x, one) if kind == "silu" else (c * (x + 0.044715 * x ** 3), c * (1 + 3 * 0.044715 * x * x))
    p = torch.sigmoid(z)
    return x * p, p * (1 + x * dz * torch.sigmoid(-z)), dz


def forward64(counts, A, W, act):
    """C, and the errors its and the factors' sums may have; H."""
    S, F = A.shape[0], W.shape[1] // 2
    H = torch.zeros(S, 2 * F, dtype=torch.float64, device="cuda")
    near = torch.zeros_like(H)
    p = 0
    for e, n in enumerate(counts):
        a, w = A[p:p + n].double(), W[e].double()
        H[p:p + n], near[p:p + n] = a @ w.T, a.abs() @ w.abs().T
        p += n
    eh = 2 * (A.shape[1] + 1) * U * near
    G, Uf, eg, eu = H[:, :F], H[:, F:], eh[:, :F], eh[:, F:]
    a, _, _ = act64(act, G)
    ea = 1.13 * eg + 16 * U * a.abs() + 2 * U * G.abs()
    return a * Uf, ea * Uf.abs() + (a.abs() + ea) * eu + 2 * U * (a * Uf).abs(), H, eh


def grad64(counts, dY, W, layout, H, act):
    S, F = dY.shape[0], H.shape[1] // 2
    dC = torch.zeros(S, F, dtype=torch.float64, device="cuda")
    near = torch.zeros_like(dC)
    live = torch.zeros(S, 1, dtype=torch.bool, device="cuda")
    p = 0
    for e, n in enumerate(counts):
        g, w = dY[p:p + n].double(), W[e].double() if layout == "kn" else W[e].double().T
        dC[p:p + n], near[p:p + n] = g @ w, g.abs() @ w.abs()
        p += n
    live[:p] = True
    H = torch.where(live, H.double(), 0.0)
    G, Uf = H[:, :F], H[:, F:]
    a, s, dz = act64(act, G)
    ec = 2 * (dY.shape[1] + 1) * U * near
    ea = 16 * U * a.abs() + 2 * U * G.abs()
    es = 16 * U * (1 + (G * dz).abs())
    dG, dU = dC * Uf * s, dC * a
    err = torch.cat([ec * (Uf * s).abs() + (dC.abs() + ec) * Uf.abs() * es + 4 * U * dG.abs(), ec * a.abs() + (dC.abs() + ec) * ea + 2 * U * dU.abs()], 1)
    return torch.cat([dG, dU], 1), err, a * Uf, ea * Uf.abs() + 2 * U * (a * Uf).abs()


def counts_of(load, E, S):
    if load == "one":
        return [S] + [0] * (E - 1)
    if load == "last":
        return [0] * (E - 1) + [S]
    rng = np.random.default_rng(E + S)
    share = rng.dirichlet(np.full(E, 0.5)) if load == "uneven" else np.full(E, 1 / E)
    return list(rng.multinomial(S - S // 10, share))  # the last tenth belongs to no expert


def forward(counts, F, K, dtype, act, pad=0, out=None):
    """The product of all experts, checked; both factors."""
    E, S = len(counts), int(sum(counts) + sum(counts) // 9)
    off = offsets_of(counts)
    A, W = padded(normal(S, S, K, dtype=dtype), pad), padded(normal(F, E, 2 * F, K, dtype=dtype, scale=K ** -0.5), pad)
    C, H = spx.spx_gemm_grouped_gated(off, A, W, act=act, grad=True, dtype=out)
    c, ec, h, eh = forward64(counts, A, W, act)
    close(H, h, eh, "H")
    close(C, c, ec, "C")
    again, none = spx.spx_gemm_grouped_gated(off, A, W, act=act, dtype=out)
    assert none is None and torch.equal(again, C)
    assert not C[sum(counts):].any() and not H[sum(counts):].any()
    assert spx.spx_last_device_error() == 0
    return H


def backward(counts, N, dtype, act, layout, H, pad=0):
    E, S, F = len(counts), H.shape[0], H.shape[1] // 2
    off = offsets_of(counts)
    dY = padded(normal(N, S, N, dtype=dtype), pad)
    W2 = normal(E, E, N, F, dtype=dtype, scale=F ** -0.5)
    W2 = padded(W2 if layout == "kn" else W2.transpose(1, 2).contiguous(), pad)
    Hn = H.clone()
    Hn[sum(counts):] = float("nan")  # what lies behind the last expert's rows does not matter
    Hn = padded(Hn, pad)
    dH, C2 = spx.spx_gemm_grouped_gated_grad(off, dY, W2, Hn, act=act, layout=layout)
    d, ed, c, ec = grad64(counts, dY, W2, layout, H, act)
    close(dH, d, ed, "dH")
    close(C2, c, ec, "C again")
    only, none = spx.spx_gemm_grouped_gated_grad(off, dY, W2, Hn, act=act, layout=layout, product=False)
    assert none is None and torch.equal(only, dH)
    assert not dH[sum(counts):].any() and not C2[sum(counts):].any()
    assert spx.spx_last_device_error() == 0


def check(load, E, S, F, R, dtype, act, layout, pad=0, out=None):
    counts = counts_of(load, E, S)
    backward(counts, R, dtype, act, layout, forward(counts, F, R, dtype, act, pad, out), pad)


@pytest.mark.parametrize("load,E,S,F,R", [("even", 1, 1, 1, 1), ("even", 1, 11, 16, 64), ("uneven", 3, 40, 24, 72), ("one", 4, 33, 72, 64),
                                          ("last", 4, 130, 136, 200), ("uneven", 60, 300, 40, 136), ("even", 8, 1000, 264, 72),
                                          ("uneven", 12, 3002, 1000, 776), ("uneven", 5, 700, 9, 1031), ("one", 2, 600, 520, 2064)])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_formulas(load, E, S, F, R, dtype, act, layout):
    check(load, E, S, F, R, dtype, act, layout)


@pytest.mark.parametrize("pad", [1, 3, 8])
@pytest.mark.parametrize("F,R", [(64, 72), (40, 33), (7, 64)])
def test_pitches_and_bases_of_any_alignment(pad, F, R):
    check("uneven", 3, 90, F, R, BF16, "silu", "kn", pad)


@pytest.mark.parametrize("F,R", [(64, 128), (40, 33)])
def test_fp32_product(F, R):
    check("uneven", 3, 190, F, R, BF16, "silu", "kn", out=F32)


def test_values_far_from_zero():
    """The activations' tails: no infinity meets a zero, small values keep their digits."""
    x = torch.tensor([-3e38, -1e4, -120.0, -60.0, -12.0, -5.0, -1e-30, 0.0, 1e-30, 5.0, 60.0, 120.0, 1e4, 3e38], device="cuda").to(BF16)
    n = x.numel()
    H = torch.stack([x, torch.ones_like(x)], 1)
    one = torch.ones(1, 1, 1, dtype=BF16, device="cuda")
    for act in ACTS:
        dH, C = spx.spx_gemm_grouped_gated_grad(offsets_of([n]), torch.ones(n, 1, dtype=BF16, device="cuda"), one, H, act=act)
        a, s, dz = act64(act, x.double().clamp(-1e4, 1e4))
        a = torch.where(x.abs().double() > 1e4, torch.where(x > 0, x.double(), 0.0), a)
        close(C[:, 0], a, 16 * U * a.abs() + 1e-37)
        dz = dz.clamp(max=200) * (x.abs() < 100)
        close(dH[:, 0], s, 16 * U * (1 + (x.double() * dz).abs()))
        close(dH[:, 1], a, 16 * U * a.abs() + 1e-37)
        ends = torch.tensor([[float("-inf"), 1], [float("inf"), 1], [float("nan"), 1]], dtype=F16, device="cuda")
        dE, E = spx.spx_gemm_grouped_gated_grad(None, torch.ones(3, 1, dtype=F16, device="cuda"), one[0].to(F16), ends, act=act)
        assert E[0, 0] == 0 and E[1, 0] == float("inf") and dE[0, 0] == 0 and dE[1, 0] == 1 and dE[2, 0].isnan() and E[2, 0].isnan()
        A = torch.stack([x, torch.ones_like(x)], 1)
        C2, _ = spx.spx_gemm_grouped_gated(None, A, torch.eye(2, dtype=BF16, device="cuda"), act=act)
        assert torch.equal(C2, C)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("K", [16, 18])
def test_activations_of_every_16_bit_value(act, dtype, K):
    """C in fp32 for G = x and U = 1: the activation itself, on the tensor cores and (K = 18) on the CUDA cores.  16 u of the
    activation as above, and: p below fp32's normal numbers, 2^-126, may be 0, which is |x| 2^-126 of x p; the tanh form's z comes
    from two rounded constants and three roundings, 5 u |z| in all, which its p = 1 / (1 + exp(-z)) passes on as 5 u |z| (1 - p) p."""
    x = torch.arange(-2 ** 15, 2 ** 15, device="cuda", dtype=torch.int32).to(torch.int16).view(dtype)
    x = x[x.abs().float() < 1e4]
    x = torch.cat([x, x[:-x.numel() % 8]]).view(-1, 8)
    A = torch.zeros(x.shape[0], K, device="cuda", dtype=dtype)
    A[:, :8], A[:, 8:16] = x, 1
    C, _ = spx.spx_gemm_grouped_gated(None, A, torch.eye(16, K, device="cuda", dtype=dtype), act=act, dtype=F32)
    a = act64(act, x.double())[0]
    err = 16 * U * a.abs() + x.double().abs() * 2.0 ** -126
    if act == "gelu_tanh":
        z = (8 / np.pi) ** 0.5 * (x.double() + 0.044715 * x.double() ** 3)
        err += 5 * U * z.abs() * torch.sigmoid(-z) * a.abs()
    close(C, a, err)
    assert not C[x == 0].any()


def test_no_offsets_no_rows_and_no_reduction():
    A, W = normal(1, 70, 64, dtype=BF16), normal(2, 48, 64, dtype=BF16)
    C, H = spx.spx_gemm_grouped_gated(None, A, W, grad=True)
    C1, H1 = spx.spx_gemm_grouped_gated(offsets_of([70]), A, W[None], grad=True)
    assert torch.equal(C, C1) and torch.equal(H, H1)
    W2, dY = normal(3, 32, 24, dtype=BF16), normal(4, 70, 32, dtype=BF16)
    a, b = spx.spx_gemm_grouped_gated_grad(None, dY, W2, H), spx.spx_gemm_grouped_gated_grad(offsets_of([70]), dY, W2[None], H)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    E = torch.empty(0, 64, dtype=BF16, device="cuda")
    assert spx.spx_gemm_grouped_gated(None, E, W)[0].shape == (0, 24)
    C, H0 = spx.spx_gemm_grouped_gated(None, torch.empty(5, 0, dtype=BF16, device="cuda"), torch.empty(8, 0, dtype=BF16, device="cuda"), grad=True)
    assert C.shape == (5, 4) and not C.any() and not H0.any()
    H5 = normal(6, 5, 8, dtype=BF16)
    dH, C5 = spx.spx_gemm_grouped_gated_grad(None, torch.empty(5, 0, dtype=BF16, device="cuda"), torch.empty(0, 4, dtype=BF16, device="cuda"), H5)
    a = act64("silu", H5[:, :4].double())[0] * H5[:, 4:].double()
    assert not dH.any()
    close(C5, a, 32 * U * a.abs())


@pytest.mark.parametrize("F,R", [(24, 64), (136, 200), (7, 9)])
def test_gradient_over_its_factors(F, R):
    """dH over H."""
    off = offsets_of([20, 0, 41])
    dY, W, H = normal(1, 61, R, dtype=BF16), normal(2, 3, R, F, dtype=BF16), normal(3, 61, 2 * F, dtype=BF16)
    dH, C = spx.spx_gemm_grouped_gated_grad(off, dY, W, H)
    h = H.clone()
    d2, C2 = spx.spx_gemm_grouped_gated_grad(off, dY, W, h, dH=h)
    assert d2 is h and torch.equal(h, dH) and torch.equal(C, C2)


@pytest.mark.parametrize("act", ACTS)
def test_gradients_by_differences(act):
    """The whole layer's gradients against (L(x + h) - L(x - h)) / 2h of L = <Y, dY> in 64 bits.  What the library rounds
    on the way (H, dH, C to fp16, 2^-11 each, and the gradient's own rounding) bounds the difference: 8 roundings of the
    terms' magnitudes, which are below 40 here."""
    S, K, F, N = 5, 16, 16, 16
    A, W1, W2, dY = normal(1, S, K, dtype=F16), normal(2, 1, 2 * F, K, dtype=F16, scale=0.25), normal(3, 1, N, F, dtype=F16, scale=0.25), normal(4, S, N, dtype=F16)
    off = offsets_of([S])
    C, H = spx.spx_gemm_grouped_gated(off, A, W1, act=act, grad=True)
    dH, C2 = spx.spx_gemm_grouped_gated_grad(off, dY, W2, H, act=act)
    dA = spx.spx_gemm_grouped(off, dH, W1, layout="kn")
    dW1, dW2 = spx.spx_gemm_grouped_wgrad(off, dH, A), spx.spx_gemm_grouped_wgrad(off, dY, C2)

    def loss(a, w1, w2):
        h = a @ w1[0].T
        return ((act64(act, h[:, :F])[0] * h[:, F:]) @ w2[0].T * dY.double()).sum()

    args, step = [A.double(), W1.double(), W2.double()], 1e-5
    for which, got, at in [(0, dA, (0, 3)), (0, dA, (4, 15)), (1, dW1, (0, 5, 2)), (1, dW1, (0, 20, 7)), (2, dW2, (0, 1, 1)), (2, dW2, (0, 15, 9))]:
        d = torch.zeros_like(args[which])
        d[at] = step
        up, down = list(args), list(args)
        up[which], down[which] = args[which] + d, args[which] - d
        assert abs((loss(*up) - loss(*down)) / (2 * step) - got[at].double()) <= 40 * 8 * 2.0 ** -11


def test_infinities_stay_in_their_rows():
    off = offsets_of([50, 14])
    A, W = normal(1, 64, 128, dtype=BF16), normal(2, 2, 64, 128, dtype=BF16)
    clean = spx.spx_gemm_grouped_gated(off, A, W, grad=True)
    A[49, 3] = float("nan")
    bad = spx.spx_gemm_grouped_gated(off, A, W, grad=True)
    keep = [i for i in range(64) if i != 49]
    for x, y in zip(clean, bad):
        assert torch.equal(x[keep], y[keep]) and y[49].isnan().all()


def test_offsets_past_32_bits():
    """A table of factors of more than 2^31 values: the last rows are right."""
    F, R = 4096, 64
    S = (1 << 31) // (2 * F) + 300
    A = torch.zeros(S, R, dtype=BF16, device="cuda")
    A[-100:] = normal(1, 100, R, dtype=BF16)
    W = normal(2, 1, 2 * F, R, dtype=BF16)
    C, H = spx.spx_gemm_grouped_gated(None, A, W[0], grad=True)
    c, ec, h, eh = forward64([100], A[-100:], W, "silu")
    close(H[-100:], h, eh)
    close(C[-100:], c, ec)
    assert not H[:1000].any()
    W2 = normal(3, 1, R, F, dtype=BF16)
    dH, C2 = spx.spx_gemm_grouped_gated_grad(None, A, W2[0], H, dH=H, C=C)
    # H is overwritten: the factors again, from the same sums
    h0 = spx.spx_gemm_grouped_gated(None, A[-100:], W[0], grad=True)[1]
    d, ed, c, ec = grad64([100], A[-100:], W2, "kn", h0, "silu")
    close(dH[-100:], d, ed)
    close(C2[-100:], c, ec)


def test_streams_and_graphs():
    S, F, R, E = 300, 136, 200, 4
    off = offsets_of(counts_of("uneven", E, S))
    A, W, W2, dY = normal(1, S, R, dtype=BF16), normal(2, E, 2 * F, R, dtype=BF16), normal(3, E, R, F, dtype=BF16), normal(4, S, R, dtype=BF16)

    def run(stream=None):
        C, H = spx.spx_gemm_grouped_gated(off, A, W, grad=True, stream=stream)
        return [C, H, *spx.spx_gemm_grouped_gated_grad(off, dY, W2, H, stream=stream)]

    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
        graphs.append((g, out))
    for seed in (10, 20):
        A.copy_(normal(seed, S, R, dtype=BF16))
        off.copy_(offsets_of(counts_of("uneven", E, S - seed)))
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for a, *rest in zip(run(), *(out for _, out in graphs)):
            assert all(torch.equal(a, b) for b in rest)
