"""Routed-expert calls at the sizes where another form of a kernel takes over.  References and tolerances are those
of tests/test_gpu_experts.py (fp32 sums within n u sum |products|, one rounding to the output's type; 8-bit products
and codes bit for bit)."""
import pytest
import torch

from csr_bsr_spmv_gb300 import spx

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
