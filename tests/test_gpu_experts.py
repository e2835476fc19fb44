"""The routed-expert operators on the GPU against plain 64-bit implementations.

Tolerances, fixed from the formats before any run.  u = 2^-24 is the fp32 unit
roundoff, v the output type's (half a unit in the last of 24, 8 and 11
significand bits: 2^-24, 2^-8 for bf16, 2^-11 for fp16 -- whose subnormals
round by up to 2^-25).  A sum of n fp32 products, in any order and
with each addition rounded or cut (a cut costs 2u, and the tensor cores add 16
products a step), is off by at most n * u * sum |products|; the last rounding
adds v * |value|.  Copies, places and 8-bit codes are exact; the 8-bit product
is an exact integer, converted to fp32 and scaled once, so it is compared bit
for bit.
"""
import numpy as np
import pytest
import torch

from csr_bsr_spmv_gb300 import spx

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
ROUND = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}
TINY = {F32: 1e-38, BF16: 1e-38, F16: 2.0 ** -25}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def ids_of(T, k, E, seed, drop=0.1, dtype=torch.int32):
    g = gen(seed)
    ids = torch.randint(0, E, (T, k), device="cuda", generator=g)
    ids[torch.rand(T, k, device="cuda", generator=g) < drop] = -1
    return ids.to(dtype)


def sort_ref(ids, E):
    x = ids.cpu().numpy().reshape(-1).astype(np.int64)
    kept = np.nonzero((x >= 0) & (x < E))[0]
    order = kept[np.argsort(x[kept], kind="stable")]
    slot = np.full(x.size, -1)
    slot[:order.size] = order
    pos = np.full(x.size, -1)
    pos[order] = np.arange(order.size)
    return np.concatenate([[0], np.cumsum(np.bincount(x[kept], minlength=E))]), slot, pos


def padded(t, pad):
    """The same rows with `pad` values between them (and the base moved by `pad` values)."""
    if not pad:
        return t
    flat = torch.full((t[..., 0].numel() * (t.shape[-1] + pad) + pad,), float("nan") if t.is_floating_point() else 77,
                      dtype=t.dtype, device=t.device)
    strides, s = [], t.shape[-1] + pad
    for n in reversed(t.shape[:-1]):
        strides.append(s)
        s *= n
    v = flat.as_strided(t.shape, tuple(reversed(strides)) + (1,), pad)
    v.copy_(t)
    return v


def close(got, ref, bound, n, what=""):
    """|got - ref| <= v |ref| + n u bound, every value; NaN counts as wrong."""
    got64 = got.double()
    tol = ROUND[got.dtype] * ref.abs() + n * 2.0 ** -24 * bound + TINY[got.dtype]
    bad = ~((got64 - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first {bad.nonzero()[0].tolist()}: " \
                          f"{got64[bad][0].item()} for {ref[bad][0].item()}"


# ---------------------------------------------------------------- the sort

@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 64), (5, 3, 2), (31, 1, 7), (33, 2, 2048), (1000, 8, 3),
                                   (2731, 3, 60), (8192, 1, 64), (8193, 1, 64), (20000, 6, 129), (70001, 4, 2048),
                                   (512, 4, 64), (513, 4, 64), (4096, 4, 33), (4097, 4, 33), (200000, 4, 50)])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_route_build_is_the_stable_sort(T, k, E, dtype):
    ids = ids_of(T, k, E, T + E, dtype=dtype)
    r = spx.spx_route_build(ids, E)
    off, slot, pos = sort_ref(ids, E)
    assert np.array_equal(r.offsets.cpu().numpy(), off)
    assert np.array_equal(r.slot.cpu().numpy(), slot)
    assert np.array_equal(r.pos.cpu().numpy(), pos)


@pytest.mark.parametrize("case", ["none kept", "one expert", "last expert", "out of range", "no tokens", "strided"])
def test_route_build_edges(case):
    T, k, E = 700, 3, 9
    ids = ids_of(T, k, E, 5)
    if case == "none kept":
        ids[:] = -1
    elif case == "one expert":
        ids[:] = 4
    elif case == "last expert":
        ids[:] = E - 1
    elif case == "out of range":
        ids[::3] = E
        ids[1::3] = 2 ** 31 - 1
        ids[2::7] = -2 ** 31
    elif case == "no tokens":
        ids = ids[:0]
    else:
        wide = torch.full((T, k + 4), 1, dtype=torch.int32, device="cuda")
        wide[:, :k] = ids
        ids = wide[:, :k]
    r = spx.spx_route_build(ids, E)
    off, slot, pos = sort_ref(ids, E)
    assert np.array_equal(r.offsets.cpu().numpy(), off)
    assert np.array_equal(r.slot.cpu().numpy(), slot) and np.array_equal(r.pos.cpu().numpy(), pos)


def test_route_build_wide_ids_do_not_wrap():
    """An int64 id of 2^32 + 1 is no expert, not expert 1."""
    ids = torch.tensor([[2 ** 32 + 1, 1], [0, -2 ** 32]], device="cuda")
    r = spx.spx_route_build(ids, 2)
    assert r.pos.tolist() == [-1, 1, 0, -1] and r.offsets.tolist() == [0, 1, 2]


# ---------------------------------------------------------------- gather, return, gradient

SHAPES = [(1, 8, 64, 4096), (3, 1, 2, 1), (7, 2, 4, 8), (65, 3, 5, 33), (130, 5, 16, 1002), (257, 9, 8, 264),
          (1000, 4, 32, 2048)]


def routed(T, k, E, seed=1, drop=0.15):
    ids = ids_of(T, k, E, seed, drop)
    r = spx.spx_route_build(ids, E)
    slot = r.slot.cpu().long()
    return r, slot[slot >= 0].cuda(), torch.rand(T, k, device="cuda", generator=gen(seed + 1)) - 0.3


@pytest.mark.parametrize("T,k,E,H", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16, torch.int8])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_gather_copies_rows(T, k, E, H, dtype, pad):
    r, order, _ = routed(T, k, E)
    X = (torch.randn(T, H, device="cuda", generator=gen(3)) * 30).to(dtype)
    out = padded(torch.full((T * k, H), 99, device="cuda").to(dtype), pad)
    got = spx.spx_route_gather(r, padded(X, pad), out if pad else None)
    want = torch.zeros(T * k, H, dtype=dtype, device="cuda")
    want[:order.numel()] = X[order // k]
    assert torch.equal(got, want)


@pytest.mark.parametrize("T,k,E,H", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("pad", [0, 1, 8])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(T, k, E, H, dtype, pad, weighted):
    r, order, w = routed(T, k, E)
    n = order.numel()
    Ys = torch.randn(T * k, H, device="cuda", generator=gen(4)).to(dtype)
    Ys[n:] = float("nan")  # rows of no slot are not read
    Y = spx.spx_route_combine(r, padded(Ys, pad), w if weighted else None)
    wd = w.double().reshape(-1)[order] if weighted else torch.ones(n, dtype=torch.float64, device="cuda")
    terms = Ys[:n].double() * wd[:, None]
    ref = torch.zeros(T, H, dtype=torch.float64, device="cuda").index_add_(0, order // k, terms)
    bound = torch.zeros(T, H, dtype=torch.float64, device="cuda").index_add_(0, order // k, terms.abs())
    close(Y, ref, bound, k + 1, "combine")


@pytest.mark.parametrize("T,k,E,H", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("pad", [0, 1, 8])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_grad_is_the_formula(T, k, E, H, dtype, pad, weighted):
    r, order, w = routed(T, k, E)
    n = order.numel()
    dY = torch.randn(T, H, device="cuda", generator=gen(5)).to(dtype)
    Ys = torch.randn(T * k, H, device="cuda", generator=gen(6)).to(dtype)
    Ys[n:] = float("nan")
    out = padded(torch.full((T * k, H), 99.0, device="cuda").to(dtype), pad)
    dYs, dw = spx.spx_route_combine_grad(r, padded(dY, pad), padded(Ys, pad), w if weighted else None, out)
    g = dY.double()[order // k]
    ref = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
    ref[:n] = g * w.double().reshape(-1)[order][:, None] if weighted else g
    close(dYs, ref, ref.abs(), 1, "dYs")
    refw = torch.zeros(T * k, dtype=torch.float64, device="cuda")
    bound = torch.zeros(T * k, dtype=torch.float64, device="cuda")
    refw[order] = (g * Ys[:n].double()).sum(1)
    bound[order] = (g * Ys[:n].double()).abs().sum(1)
    close(dw.reshape(-1), refw, bound, H, "dw")
    only, none = spx.spx_route_combine_grad(r, dY, None, w if weighted else None)
    assert none is None and torch.equal(only, dYs)


def test_return_gradients_match_differences():
    """Whole numbers small enough that fp32 holds every sum: differences of the forward pass give the
    gradients exactly (the return is linear in the rows and in the weights)."""
    T, k, E, H = 40, 3, 6, 20
    ids = ids_of(T, k, E, 11, 0.2)
    r = spx.spx_route_build(ids, E)
    g = gen(12)

    def whole(*s):
        return torch.randint(-4, 5, s, device="cuda", generator=g).float()

    Ys, w, dY, X = whole(T * k, H), whole(T, k), whole(T, H), whole(T, H)
    dYs, dw = spx.spx_route_combine_grad(r, dY, Ys, w)
    D, d = whole(T * k, H), whole(T, k)
    up, down = spx.spx_route_combine(r, Ys + D, w), spx.spx_route_combine(r, Ys - D, w)
    assert ((up - down) * dY).sum().item() / 2 == (dYs * D).sum().item()
    up, down = spx.spx_route_combine(r, Ys, w + d), spx.spx_route_combine(r, Ys, w - d)
    assert ((up - down) * dY).sum().item() / 2 == (dw * d).sum().item()
    G, D = whole(T * k, H), whole(T, H)
    up, down = spx.spx_route_gather(r, X + D), spx.spx_route_gather(r, X - D)
    assert ((up - down) * G).sum().item() / 2 == (spx.spx_route_combine(r, G) * D).sum().item()


def test_infinities_stay_in_their_token():
    T, k, E, H = 50, 2, 4, 40
    r, order, w = routed(T, k, E, 21, 0.0)
    Ys = torch.randn(T * k, H, device="cuda", generator=gen(22))
    base = spx.spx_route_combine(r, Ys, w)
    p = int(r.pos[2 * 7 + 1])
    Ys[p, 3], Ys[p, 4] = float("inf"), float("nan")
    Y = spx.spx_route_combine(r, Ys, w)
    assert torch.isinf(Y[7, 3]) and torch.isnan(Y[7, 4])
    Y[7, 3:5] = base[7, 3:5]
    assert torch.equal(Y, base)


def test_gather_past_32_bit_offsets():
    T, k, E, H = 560000, 2, 4, 2048  # 2.3e9 values in the sorted array
    ids = ids_of(T, k, E, 31, 0.01)
    r = spx.spx_route_build(ids, E)
    X = torch.randint(-100, 100, (T, H), device="cuda", generator=gen(32), dtype=torch.int8)
    Xs = spx.spx_route_gather(r, X)
    n = int(r.offsets[-1])
    for lo in range(0, T * k, 1 << 18):
        sl = r.slot[lo:lo + (1 << 18)].long()
        want = X[sl.clamp(min=0) // k] * (sl >= 0)[:, None]
        assert torch.equal(Xs[lo:lo + (1 << 18)], want)
    assert n < T * k


# ---------------------------------------------------------------- the experts' products

def counts_case(name, E, S, seed=0):
    """offsets[E + 1] of a few shapes of load: spread, with empty experts, all on one, single rows, rows past the last."""
    rng = np.random.default_rng(seed)
    if name == "spread":
        c = rng.multinomial(S, rng.dirichlet(np.ones(E)))
    elif name == "gaps":
        c = rng.multinomial(S - S // 5, rng.dirichlet(np.ones(E)))
        c[rng.random(E) < 0.4] = 0
    elif name == "one":
        c = np.zeros(E, int)
        c[E // 2] = S
    elif name == "single":
        c = np.minimum(np.arange(E) % 2, 1)
        c[c.cumsum() > S] = 0
    else:
        c = np.zeros(E, int)
    return torch.tensor(np.concatenate([[0], np.cumsum(c)]), dtype=torch.int32, device="cuda")


def product_ref(off, A, W):
    """In 64 bits, with the sums of magnitudes; W as E x N x K."""
    S, N = A.shape[0], W.shape[1]
    ref = torch.zeros(S, N, dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(ref)
    o = off.tolist()
    for e in range(len(o) - 1):
        if o[e + 1] > o[e]:
            a, w = A[o[e]:o[e + 1]].double(), W[e].double()
            ref[o[e]:o[e + 1]] = a @ w.T
            bound[o[e]:o[e + 1]] = a.abs() @ w.abs().T
    return ref, bound


PRODUCTS = [("spread", 4, 300, 128, 64), ("spread", 3, 1000, 1000, 776), ("gaps", 12, 700, 264, 520),
            ("one", 5, 600, 96, 200), ("single", 64, 40, 512, 1024), ("empty", 3, 20, 72, 40),
            ("spread", 1, 1, 8, 8), ("spread", 2, 5, 1, 16), ("gaps", 40, 4097, 136, 72), ("spread", 8, 2000, 513, 257),
            ("spread", 300, 90, 40, 24), ("one", 2, 257, 256, 4096),
            ("spread", 200, 900, 200, 264), ("gaps", 7, 5000, 392, 648),
            # few tiles and a long reduction: shared by four CTAs
            ("spread", 1, 16, 512, 8192), ("spread", 1, 100, 640, 4104), ("gaps", 2, 33, 384, 6000)]


@pytest.mark.parametrize("load,E,S,N,K", PRODUCTS)
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F16, F16), (BF16, F32), (F16, F32)])
@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("pad", ["dense", "wide", "odd"])
def test_grouped_product(load, E, S, N, K, dtype, out, layout, pad):
    """Every layout and load; NaN in the rows of no expert must not show anywhere."""
    off = counts_case(load, E, S, N)
    g = gen(N + K)
    A = torch.randn(S, K, device="cuda", generator=g).to(dtype)
    W = torch.randn(E, N, K, device="cuda", generator=g).to(dtype)
    ref, bound = product_ref(off, A, W)
    A[int(off[-1]):] = float("nan")
    Wl = W if layout == "nk" else W.transpose(1, 2).contiguous()
    p = {"dense": 0, "wide": 8 + (-A.shape[1]) % 8, "odd": 1}[pad]
    q = {"dense": 0, "wide": 8 + (-Wl.shape[2]) % 8, "odd": 3}[pad]
    C = padded(torch.full((S, N), 7.0, device="cuda").to(out), p)
    got = spx.spx_gemm_grouped(off, padded(A, p), padded(Wl, q), C, layout=layout)
    close(got, ref, bound, K, "product")
    assert spx.spx_last_device_error() == 0


@pytest.mark.parametrize("load,E,S,N,K", PRODUCTS)
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F16, F16), (BF16, F32)])
@pytest.mark.parametrize("pad", ["dense", "wide", "odd"])
def test_grouped_weight_gradient(load, E, S, N, K, dtype, out, pad):
    off = counts_case(load, E, S, N)
    g = gen(N + K + 1)
    G = torch.randn(S, N, device="cuda", generator=g).to(dtype)
    A = torch.randn(S, K, device="cuda", generator=g).to(dtype)
    o = off.tolist()
    ref = torch.zeros(E, N, K, dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(ref)
    for e in range(E):
        ge, ae = G[o[e]:o[e + 1]].double(), A[o[e]:o[e + 1]].double()
        ref[e] = ge.T @ ae
        bound[e] = ge.abs().T @ ae.abs()
    G[o[-1]:], A[o[-1]:] = float("nan"), float("inf")
    p = {"dense": 0, "wide": 8 + (-N) % 8, "odd": 1}[pad]
    q = {"dense": 0, "wide": 8 + (-K) % 8, "odd": 3}[pad]
    dW = padded(torch.full((E, N, K), 7.0, device="cuda").to(out), q)
    got = spx.spx_gemm_grouped_wgrad(off, padded(G, p), padded(A, q), dW)
    close(got, ref, bound, S, "weight gradient")
    assert spx.spx_last_device_error() == 0


@pytest.mark.parametrize("E,S,N,K", [(4, 200, 256, 128), (3, 333, 72, 200)])
def test_nan_rows_stay_with_their_expert(E, S, N, K):
    """A NaN in one expert's rows must not reach the products or gradients of its neighbours."""
    off = counts_case("spread", E, S, 3)
    o = off.tolist()
    g = gen(41)
    A = torch.randn(S, K, device="cuda", generator=g).to(BF16)
    G = torch.randn(S, N, device="cuda", generator=g).to(BF16)
    W = torch.randn(E, N, K, device="cuda", generator=g).to(BF16)
    C0, dW0 = spx.spx_gemm_grouped(off, A, W), spx.spx_gemm_grouped_wgrad(off, G, A)
    A2, G2 = A.clone(), G.clone()
    A2[o[1]:o[2]], G2[o[1]:o[2]] = float("nan"), float("inf")
    C, dW = spx.spx_gemm_grouped(off, A2, W), spx.spx_gemm_grouped_wgrad(off, G2, A2)
    keep = [e for e in range(E) if e != 1]
    for e in keep:
        assert torch.equal(C[o[e]:o[e + 1]], C0[o[e]:o[e + 1]]) and torch.equal(dW[e], dW0[e])
    assert torch.isnan(C[o[1]:o[2]]).all() and torch.isnan(dW[1]).all()


@pytest.mark.parametrize("E,S,N,K", [(5, 300, 136, 200), (3, 64, 256, 64)])
def test_product_gradients_match_differences(E, S, N, K):
    """Whole numbers: every product and sum is exact, so are the differences."""
    off = counts_case("gaps", E, S, 2)
    g = gen(51)

    def whole(*s):
        return torch.randint(-2, 3, s, device="cuda", generator=g).to(BF16)

    A, W, G = whole(S, K), whole(E, N, K), whole(S, N)
    n = int(off[-1])
    dA = spx.spx_gemm_grouped(off, G, W, layout="kn", dtype=F32)
    dW = spx.spx_gemm_grouped_wgrad(off, G, A, dtype=F32)
    D = whole(S, K)
    diff = spx.spx_gemm_grouped(off, A + D, W, dtype=F32) - spx.spx_gemm_grouped(off, A - D, W, dtype=F32)
    assert (diff.double() * G.double()).sum().item() / 2 == (dA.double() * D.double())[:n].sum().item()
    D = whole(E, N, K)
    diff = spx.spx_gemm_grouped(off, A, W + D, dtype=F32) - spx.spx_gemm_grouped(off, A, W - D, dtype=F32)
    assert (diff.double() * G.double()).sum().item() / 2 == (dW.double() * D.double()).sum().item()


def test_shared_weights_have_stride_zero():
    """All experts reading one matrix (stride 0 between them) is the plain product."""
    A = torch.randn(100, 64, device="cuda", generator=gen(61)).to(BF16)
    W = torch.randn(1, 96, 64, device="cuda", generator=gen(62)).to(BF16)
    off = counts_case("one", 1, 100)
    many = torch.tensor([0, 30, 30, 100], dtype=torch.int32, device="cuda")
    assert torch.equal(spx.spx_gemm_grouped(many, A, W.expand(3, -1, -1)), spx.spx_gemm_grouped(off, A, W))


def test_wrong_offsets_stay_inside_the_arrays():
    """Offsets out of order or past S: values are unspecified, accesses stay inside and nothing hangs."""
    A = torch.randn(300, 64, device="cuda", generator=gen(63)).to(BF16)
    W = torch.randn(3, 128, 64, device="cuda", generator=gen(64)).to(BF16)
    G = torch.randn(300, 128, device="cuda", generator=gen(65)).to(BF16)
    q, s = spx.spx_quant_rows_i8(A)
    w8 = torch.ones(3, 128, 64, dtype=torch.int8, device="cuda")
    for bad in ([0, 500, 100, 900], [-7, -3, 200, 10 ** 9], [300, 200, 100, 0]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        spx.spx_gemm_grouped(off, A, W)
        spx.spx_gemm_grouped(off, G, W, layout="kn")
        spx.spx_gemm_grouped_wgrad(off, G, A)
        spx.spx_gemm_i8(q, s, w8, torch.ones(3, 128, device="cuda"), offsets=off)
        assert spx.spx_last_device_error() == 0


def test_product_past_32_bit_offsets():
    S, N, K = 70000, 32768, 64  # 2.3e9 values in C
    A = torch.randn(S, K, device="cuda", generator=gen(71)).to(BF16)
    W = torch.randn(2, N, K, device="cuda", generator=gen(72)).to(BF16)
    off = torch.tensor([0, 100, S], dtype=torch.int32, device="cuda")
    C = spx.spx_gemm_grouped(off, A, W)
    for lo, e in ((0, 0), (65500, 1), (S - 64, 1)):
        a, w = A[lo:lo + 64].double(), W[e].double()
        close(C[lo:lo + 64], a @ w.T, a.abs() @ w.abs().T, K, "far rows")


def test_weights_past_32_bit_offsets():
    E, N, K = 36, 8192, 8192  # 2.4e9 weights
    W = torch.empty(E, N, K, device="cuda", dtype=BF16)
    for e in range(E):
        W[e].normal_(generator=gen(200 + e))
    S = 3 * E
    A = torch.randn(S, K, device="cuda", generator=gen(201)).to(BF16)
    off = torch.arange(0, S + 1, 3, dtype=torch.int32, device="cuda")
    G = torch.randn(S, N, device="cuda", generator=gen(202)).to(BF16)
    C, dA = spx.spx_gemm_grouped(off, A, W), spx.spx_gemm_grouped(off, G, W, layout="kn")
    W8 = torch.randint(-127, 128, (E, N, K), device="cuda", generator=gen(203), dtype=torch.int8)
    Q, rs = spx.spx_quant_rows_i8(A)
    ws = torch.rand(E, N, device="cuda", generator=gen(204))
    C8 = spx.spx_gemm_i8(Q, rs, W8, ws, offsets=off)
    dW = spx.spx_gemm_grouped_wgrad(off, G, A)
    for e in (0, 31, 32, 35):
        a, g, w = A[3 * e:3 * e + 3].double(), G[3 * e:3 * e + 3].double(), W[e].double()
        close(C[3 * e:3 * e + 3], a @ w.T, a.abs() @ w.abs().T, K, "far weights")
        close(dA[3 * e:3 * e + 3], g @ w, g.abs() @ w.abs(), N, "far weights")
        close(dW[e], g.T @ a, g.abs().T @ a.abs(), 3, "far gradient")
        acc = (Q[3 * e:3 * e + 3].double() @ W8[e].double().T).long()
        assert torch.equal(C8[3 * e:3 * e + 3], acc.float() * (rs[3 * e:3 * e + 3, None] * ws[e]))


def test_experts_on_another_stream():
    """Calls on a side stream, their outputs read there, while the main stream reuses memory."""
    T, k, E, H, N = 600, 2, 6, 256, 384
    side = torch.cuda.Stream()
    ids = ids_of(T, k, E, 81)
    X = torch.randn(T, H, device="cuda", generator=gen(82)).to(BF16)
    W = torch.randn(E, N, H, device="cuda", generator=gen(83)).to(BF16)
    r = spx.spx_route_build(ids, E)
    want = spx.spx_route_combine(r, spx.spx_gemm_grouped(r.offsets, spx.spx_route_gather(r, X), W))
    torch.cuda.synchronize()
    for _ in range(5):
        r2 = spx.spx_route_build(ids, E, stream=side)
        Xs = spx.spx_route_gather(r2, X, stream=side)
        C = spx.spx_gemm_grouped(r2.offsets, Xs, W, stream=side)
        Y = spx.spx_route_combine(r2, C, stream=side)
        junk = torch.full((T * k, N), float("nan"), device="cuda", dtype=BF16)  # main-stream memory
        del Xs, C
        side.synchronize()
        assert torch.equal(Y, want)
        del junk


def test_experts_in_a_graph():
    """Capture of route, gather, product, return; replays follow the contents of the captured buffers."""
    T, k, E, H = 64, 2, 8, 128
    ids = ids_of(T, k, E, 91)
    X = torch.randn(T, H, device="cuda", generator=gen(92)).to(BF16)
    W = torch.randn(E, H, H, device="cuda", generator=gen(93)).to(BF16)

    def step():
        r = spx.spx_route_build(ids, E)
        return spx.spx_route_combine(r, spx.spx_gemm_grouped(r.offsets, spx.spx_route_gather(r, X), W))

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for seed in (94, 95):
        ids.copy_(ids_of(T, k, E, seed))
        X.copy_(torch.randn(T, H, device="cuda", generator=gen(seed)))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, step())


# ---------------------------------------------------------------- 8 bits

@pytest.mark.parametrize("M,K", [(1, 1), (1, 4096), (3, 17), (100, 776), (65, 1003), (2, 20000)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("pad", [0, 1, 16])
def test_quant_rows(M, K, dtype, pad):
    X = (torch.randn(M, K, device="cuda", generator=gen(K)) * 3).to(dtype)
    if M > 2:
        X[1] = 0
        X[2, :] = 0
        X[2, K // 2] = -1e-3
    Q, s = spx.spx_quant_rows_i8(padded(X, pad), padded(torch.zeros(M, K, dtype=torch.int8, device="cuda"), pad))
    x = X.float().cpu().numpy()
    sn = (np.abs(x).max(1) / np.float32(127)).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        qn = np.where(sn[:, None] > 0, np.rint(x / sn[:, None]), 0).astype(np.int8)
    assert np.array_equal(s.cpu().numpy(), sn) and np.array_equal(Q.cpu().numpy(), qn)


def test_quant_rows_subnormal_and_not_finite():
    X = torch.zeros(5, 300, device="cuda")
    X[0, 7], X[0, 9] = 3e-45, -1e-43        # a subnormal scale: codes stay inside -127..127
    X[1, 299] = float("inf")
    X[2, 0] = float("nan")
    X[3, 5], X[3, 6] = float("-inf"), float("nan")
    X[4, 1] = 3.0e38
    X[1:4, 20] = 5.0
    Q, s = spx.spx_quant_rows_i8(X)
    assert Q.abs().max() <= 127 and torch.isnan(s[1:4]).all() and not Q[1:4].any()
    assert torch.isfinite(s[0]) and torch.isfinite(s[4]) and Q[4, 1] == 127
    C = spx.spx_gemm_i8(Q, s, torch.ones(16, 300, dtype=torch.int8, device="cuda"), torch.ones(16, device="cuda"))
    assert torch.isnan(C[1:4]).all() and torch.isfinite(C[[0, 4]]).all()


def i8_ref(off, Q, rs, W, ws, out):
    """The exact integers (64 bits), as fp32, times the fp32 product of the scales, rounded to `out`."""
    S, N = Q.shape[0], W.shape[1]
    C = torch.zeros(S, N, device="cuda")
    o = off.tolist()
    for e in range(len(o) - 1):
        lo, hi = o[e], o[e + 1]
        if hi > lo:
            acc = (Q[lo:hi].double() @ W[e].double().T).long()
            C[lo:hi] = acc.float() * (rs[lo:hi, None] * ws[e][None, :])
    return C.to(out)


I8 = [("spread", 1, 1, 4096, 4096), ("spread", 1, 5, 100, 300), ("spread", 1, 64, 256, 512), ("spread", 1, 300, 1000, 776),
      ("spread", 4, 500, 264, 1040), ("gaps", 12, 800, 128, 96), ("single", 64, 40, 512, 256), ("one", 3, 400, 513, 129),
      # one or two rows in all, up to 8, 16 and 32 an expert, and on to 128: each with long and short reductions
      ("one", 3, 2, 72, 4096), ("spread", 1, 2, 1030, 208), ("spread", 1, 8, 300, 4112), ("spread", 1, 16, 520, 9216),
      ("spread", 40, 200, 136, 2048), ("gaps", 40, 480, 100, 1040), ("spread", 1, 24, 512, 4096),
      ("spread", 5, 170, 260, 4112), ("gaps", 6, 300, 264, 2320), ("spread", 2, 250, 640, 3000), ("one", 4, 100, 136, 520),
      ("empty", 3, 20, 72, 40), ("spread", 2, 17, 1, 1), ("spread", 1, 2, 40, 5000), ("spread", 3, 900, 272, 2064)]


@pytest.mark.parametrize("load,E,S,N,K", I8)
@pytest.mark.parametrize("out", [F32, BF16, F16])
@pytest.mark.parametrize("pad", ["dense", "wide", "odd"])
def test_int8_product_is_exact(load, E, S, N, K, out, pad):
    off = counts_case(load, E, S, N)
    g = gen(N + K)
    Q = torch.randint(-128, 128, (S, K), device="cuda", generator=g, dtype=torch.int8)
    W = torch.randint(-128, 128, (E, N, K), device="cuda", generator=g, dtype=torch.int8)
    rs = torch.rand(S, device="cuda", generator=g) / 1000
    ws = torch.rand(E, N, device="cuda", generator=g) / 100
    want = i8_ref(off, Q, rs, W, ws, out)
    p = {"dense": 0, "wide": 16 + (-K) % 16, "odd": 1}[pad]
    Qp, Wp = padded(Q, p), padded(W, p)
    C = padded(torch.full((S, N), 7.0, device="cuda").to(out), 0 if pad == "dense" else 5)
    if E == 1:
        got = spx.spx_gemm_i8(Qp, rs, Wp[0], ws[0], C=C)
        assert torch.equal(spx.spx_gemm_i8(Qp, rs, Wp, ws, offsets=off, dtype=out), want)
    else:
        got = spx.spx_gemm_i8(Qp, rs, Wp, ws, offsets=off, C=C)
    assert torch.equal(got, want)
    assert spx.spx_last_device_error() == 0


@pytest.mark.parametrize("S,N,K", [(1, 64, 65536), (64, 128, 8192), (300, 256, 131071 - 15), (9, 300, 1025), (200, 256, 2048)])
@pytest.mark.parametrize("a,b", [(-128, -128), (127, -128), (127, 127)])
def test_int8_product_is_exact_at_the_extremes(S, N, K, a, b):
    """Every code at its largest: sums far past 2^24, where an fp32 sum would round."""
    Q = torch.full((S, K), a, dtype=torch.int8, device="cuda")
    W = torch.full((N, K), b, dtype=torch.int8, device="cuda")
    Q[0, 0], W[0, K - 1] = 1, 1  # and odd ones
    one = torch.ones(max(S, N), device="cuda")
    C = spx.spx_gemm_i8(Q, one[:S], W, one[:N])
    row = torch.full((S, N), float(a * b * K), dtype=torch.float64, device="cuda")
    row[0] += (1 - a) * b
    row[:, 0] += (1 - b) * a
    assert torch.equal(C, row.float())


# ---------------------------------------------------------------- the layer

def test_layer_end_to_end():
    """Sort, gather, two products with a ReLU between them, weighted return, and every gradient, against
    the same layer in 64 bits.  Whole-number inputs with small sums, so the 16-bit steps are exact."""
    T, k, E, H, F = 150, 2, 5, 64, 72
    g = gen(101)

    def whole(lo, hi, *s):
        return torch.randint(lo, hi + 1, s, device="cuda", generator=g).float()

    ids = ids_of(T, k, E, 102, 0.1)
    X, W1, W2 = whole(-1, 1, T, H), whole(-1, 1, E, F, H), whole(-1, 1, E, H, F)
    W1 *= torch.rand(E, F, H, device="cuda", generator=g) < 0.2
    W2 *= torch.rand(E, H, F, device="cuda", generator=g) < 0.1
    wt, dY = whole(1, 2, T, k), whole(-1, 1, T, H)
    r = spx.spx_route_build(ids, E)
    Xs = spx.spx_route_gather(r, X.to(F16))
    h = spx.spx_gemm_grouped(r.offsets, Xs, W1.to(F16))
    a = torch.relu(h)
    Ys = spx.spx_gemm_grouped(r.offsets, a, W2.to(F16))
    Y = spx.spx_route_combine(r, Ys, wt)
    dYs, dwt = spx.spx_route_combine_grad(r, dY.to(F16), Ys, wt)
    da = spx.spx_gemm_grouped(r.offsets, dYs, W2.to(F16), layout="kn")
    dW2 = spx.spx_gemm_grouped_wgrad(r.offsets, dYs, a, dtype=F32)
    dh = da * (h > 0)
    dW1 = spx.spx_gemm_grouped_wgrad(r.offsets, dh, Xs, dtype=F32)
    dX = spx.spx_route_combine(r, spx.spx_gemm_grouped(r.offsets, dh, W1.to(F16), layout="kn"))

    P = [t.double().requires_grad_() for t in (X, W1, W2, wt)]
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if e >= 0:
                out[t] = out[t] + P[3][t, j] * (P[2][e] @ torch.relu(P[1][e] @ P[0][t]))
    out.backward(dY.double())
    assert torch.equal(Y.double(), out.detach())
    for got, p in ((dX, P[0]), (dW1, P[1]), (dW2, P[2]), (dwt, P[3])):
        assert torch.equal(got.double(), p.grad)


def test_example_trains_and_serves():
    """examples/routed_experts.py: the loss falls, and 8-bit experts stay within 5% of the bf16 layer (codes of
    7 bits a value round by about 0.5% of a row's largest, four roundings in a row)."""
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "routed_experts.py")
    spec = importlib.util.spec_from_file_location("routed_experts", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses, off = m.main(tokens=512, width=128, inner=256, experts=8, k=2, steps=30, say=lambda *_: None)
    assert losses[-1] < 0.8 * losses[0]
    assert all(v < 0.05 for v in off.values())
