"""Routed-expert calls at the sizes where another form of a kernel takes over.  References and tolerances are those
of tests/test_gpu_experts.py (fp32 sums within n u sum |products|, one rounding to the output's type; 8-bit products
and codes bit for bit)."""
import pytest
import torch

from csr_bsr_spmv_gb300 import spx
from test_gpu_experts import close, counts_case, gen, padded

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


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
