"""Routed-expert calls at the sizes where another form of a kernel takes over.  References and tolerances are those
of tests/test_gpu_experts.py (fp32 sums within n u sum |products|, one rounding to the output's type; 8-bit products
and codes bit for bit)."""
import pytest
import torch

import experts_forms
import test_gpu_experts as base
from csr_bsr_spmv_gb300 import spx
from test_gpu_experts import close, counts_case, gen, padded

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def test_a_gradient_over_hundreds_of_millions_of_rows_is_waited_for():
    """One expert with 4e8 rows and one tile: its reduction takes longer than a second, the limit of a wait that does
    not grow with it.  Zeros but for a few rows of small whole numbers, so the gradient is exact."""
    S, N, K = 400_000_003, 8, 8
    G = torch.zeros(S, N, device="cuda", dtype=BF16)
    A = torch.zeros(S, K, device="cuda", dtype=BF16)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    rows = torch.cat([torch.arange(0, S, 2_000_003, device="cuda"), torch.tensor([S - 2, S - 1], device="cuda")])
    G[rows] = torch.randint(-2, 3, (rows.numel(), N), device="cuda", generator=g).to(BF16)
    A[rows] = torch.randint(-2, 3, (rows.numel(), K), device="cuda", generator=g).to(BF16)
    off = torch.tensor([0, S], dtype=torch.int32, device="cuda")
    dW = spx.spx_gemm_grouped_wgrad(off, G, A, dtype=torch.float32)
    assert spx.spx_last_device_error() == 0
    assert torch.equal(dW[0].double(), G[rows].double().T @ A[rows].double())


@pytest.mark.parametrize("E,S,N,K", [(1, 700, 8, 2048), (8, 3000, 16, 1024), (5, 900, 64, 128), (3, 500, 1, 72), (60, 4000, 40, 264),
                                     (4, 1000, 65, 520)])
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (torch.float16, torch.float32)])
def test_gradients_of_few_output_rows(E, S, N, K, dtype, out):
    """dW of N <= 64 rows (adapters of low rank): one 128-row tile, on a single CTA where K is short."""
    off = counts_case("spread", E, S, N)
    g = gen(N + K)
    G = torch.randn(S, N, device="cuda", generator=g).to(dtype)
    A = torch.randn(S, K, device="cuda", generator=g).to(dtype)
    p = (-N) % 8  # rows the copy engine can read
    dW = spx.spx_gemm_grouped_wgrad(off, padded(G, p), A, dtype=out)
    o = off.tolist()
    for e in range(E):
        ge, ae = G[o[e]:o[e + 1]].double(), A[o[e]:o[e + 1]].double()
        close(dW[e], ge.T @ ae, ge.abs().T @ ae.abs(), S, "gradient")
    assert spx.spx_last_device_error() == 0


# ---------------------------------------------------------------- every tile and every way to share a reduction

@pytest.mark.parametrize("case", experts_forms.PRODUCTS)
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F16, F32)])
@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("pad", ["dense", "wide"])
def test_product_in_every_form(case, dtype, out, layout, pad):
    base.test_grouped_product(*case, dtype, out, layout, pad)


@pytest.mark.parametrize("case", experts_forms.GRADIENTS)
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F16, F32)])
@pytest.mark.parametrize("pad", ["dense", "wide"])
def test_gradient_in_every_form(case, dtype, out, pad):
    base.test_grouped_weight_gradient(*case, dtype, out, pad)


@pytest.mark.parametrize("case", experts_forms.COPIED)
@pytest.mark.parametrize("out", [F32, BF16, F16])
def test_int8_product_through_copies(case, out):
    base.test_int8_product_is_exact(*case, out, "dense")


@pytest.mark.parametrize("case", experts_forms.PRODUCTS)
def test_int8_product_through_copies_of_odd_rows(case):
    """Rows off 16 bytes take the copies at any number of rows: all the product's tiles."""
    base.test_int8_product_is_exact(*case, F32, "odd")


@pytest.mark.parametrize("case", experts_forms.WIDENED)
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("pad", ["dense", "wide"])
def test_int8_product_widened_on_the_way(case, out, pad):
    base.test_int8_product_is_exact(*case, out, pad)


# as many channel blocks as keep the memory busy: a warp each, nothing shared
@pytest.mark.parametrize("case", [("spread", 64, 256, 4096, 272), ("gaps", 64, 640, 4096, 272), ("spread", 64, 960, 5000, 272)])
def test_int8_product_of_few_rows_and_many_experts(case):
    base.test_int8_product_is_exact(*case, BF16, "dense")


def test_int8_prefill_batch_is_exact():
    """16384 rows over 8 uneven experts on 256-row tiles of CTA pairs, a ragged last tile of columns."""
    base.test_int8_product_is_exact("spread", 8, 16384, 4088, 2048, BF16, "dense")


@pytest.mark.parametrize("S,N,K", [(4000, 264, 8192), (1000, 2000, 65536)])
@pytest.mark.parametrize("a,b", [(-128, -128), (127, -128)])
def test_int8_product_of_pairs_is_exact_at_the_extremes(S, N, K, a, b):
    base.test_int8_product_is_exact_at_the_extremes(S, N, K, a, b)


# ---------------------------------------------------------------- rows

@pytest.mark.parametrize("M,K", [(1216, 2048), (1216, 256), (3001, 776), (2000, 1024), (1300, 1001), (1217, 2047), (1500, 17),
                                 (1216, 4096), (1300, 2049)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("pad", [0, 1])
def test_quantisation_a_warp_a_row(M, K, dtype, pad):
    base.test_quant_rows(M, K, dtype, pad)


ROWS = [(2432, 3, 16, 2048), (2433, 2, 8, 1002), (3001, 8, 16, 130), (2500, 4, 8, 1031), (2450, 5, 12, 515), (2431, 3, 5, 1000)]


@pytest.mark.parametrize("T,k,E,H", ROWS)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("pad", [0, 1])
def test_many_tokens_there_and_back(T, k, E, H, dtype, pad):
    """Tokens enough for a warp each in the return's gradient."""
    base.test_gather_copies_rows(T, k, E, H, dtype, pad)
    base.test_combine(T, k, E, H, dtype, pad, True)
    base.test_combine_grad_is_the_formula(T, k, E, H, dtype, pad, True)


@pytest.mark.parametrize("dtype", [F32, BF16, torch.int8])
@pytest.mark.parametrize("H,pad", [(2064, 0), (516, 0), (515, 1), (8192, 4)])
@pytest.mark.parametrize("kept", [0.0, 0.5])
def test_gather_clears_the_rows_of_dropped_slots(dtype, H, pad, kept):
    T, k, E = 301, 3, 7
    g = gen(7)
    ids = torch.randint(0, E, (T, k), device="cuda", generator=g)
    ids[torch.rand(T, k, device="cuda", generator=g) >= kept] = -1
    r = spx.spx_route_build(ids, E)
    n = int(r.offsets[-1])
    X = (torch.randn(T, H, device="cuda", generator=g) * 30).to(dtype)
    out = padded(torch.full((T * k, H), 99, device="cuda").to(dtype), pad)
    spx.spx_route_gather(r, padded(X, pad), out)
    assert not out[n:].any() and torch.equal(out[:n], X[r.slot[:n].long() // k])
    if dtype != torch.int8:
        dYs = padded(torch.full((T * k, H), 99, device="cuda").to(dtype), pad)
        spx.spx_route_combine_grad(r, padded(X, pad), dYs=dYs)
        assert not dYs[n:].any()


# ---------------------------------------------------------------- what a call does not depend on

@pytest.mark.parametrize("case", experts_forms.PRODUCTS[::3] + [("spread", 8, 4096, 1024, 2048)])
def test_results_are_the_same_from_run_to_run(case):
    load, E, S, N, K = case
    off, g = counts_case(load, E, S, N), gen(3)
    A, W = (torch.randn(*s, device="cuda", generator=g).to(BF16) for s in ((S, K), (E, N, K)))
    G = torch.randn(S, N, device="cuda", generator=g).to(BF16)
    Q, s = spx.spx_quant_rows_i8(A)
    W8, ws = W.to(torch.int8), torch.rand(E, N, device="cuda", generator=g)

    def all_of_it():
        return (spx.spx_gemm_grouped(off, A, W), spx.spx_gemm_grouped(off, G, W, layout="kn"), spx.spx_gemm_grouped_wgrad(off, G, A),
                spx.spx_gemm_i8(Q, s, W8, ws, offsets=off))

    first = all_of_it()
    for _ in range(4):
        assert all(torch.equal(x, y) for x, y in zip(all_of_it(), first))


@pytest.mark.parametrize("gap", [16, 48, 3])
def test_experts_any_distance_apart(gap):
    """An expert stride that is no multiple of the row pitch."""
    E, S, N, K = 5, 400, 136, 208
    off, g = counts_case("spread", E, S, 5), gen(9)

    def apart(t):
        flat = torch.zeros(E * (N * K + gap), dtype=t.dtype, device="cuda")
        v = flat.as_strided((E, N, K), (N * K + gap, K, 1))
        v.copy_(t)
        return v

    A, G = torch.randn(S, K, device="cuda", generator=g).to(BF16), torch.randn(S, N, device="cuda", generator=g).to(BF16)
    W = torch.randn(E, N, K, device="cuda", generator=g).to(BF16)
    ref, bound = base.product_ref(off, A, W)
    close(spx.spx_gemm_grouped(off, A, apart(W)), ref, bound, K, "product")
    ref, bound = base.product_ref(off, G, W.transpose(1, 2))
    close(spx.spx_gemm_grouped(off, G, apart(W), layout="kn"), ref, bound, N, "its gradient")
    dense = spx.spx_gemm_grouped_wgrad(off, G, A)
    assert torch.equal(spx.spx_gemm_grouped_wgrad(off, G, A, apart(torch.zeros_like(W))), dense)
    W8 = torch.randint(-127, 128, (E, N, K), device="cuda", generator=g, dtype=torch.int8)
    ws = torch.rand(E, N, device="cuda", generator=g)
    for rows in (60, S):  # straight from memory, and widened on the way
        Q, s = spx.spx_quant_rows_i8(A[:rows])
        o = off.clamp(max=rows)
        assert torch.equal(spx.spx_gemm_i8(Q, s, apart(W8), ws, offsets=o), base.i8_ref(o, Q, s, W8, ws, F32))
    assert spx.spx_last_device_error() == 0
