"""A builder, a check or an upload that CUDA refuses on the host -- on a stream whose capture was broken off -- leaves nothing
for the product that follows it."""
import pytest
import torch

from csr_bsr_spmv_gb300 import spx
from test_gpu_refused_calls import broken  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
M, K = 96, 128


def matrix():
    g = torch.Generator().manual_seed(3)
    D = torch.randint(-3, 4, (M, K), generator=g).float() * (torch.rand(M, K, generator=g) < 0.1)
    row, col = (t.int().cuda() for t in D.nonzero().t())
    val = D[D != 0].cuda()
    return D.cuda(), row.contiguous(), col.contiguous(), val


@pytest.mark.parametrize("name", ["build", "transpose", "bsr", "wcsr", "check", "plan"])
def test_the_next_product_is_not_refused(broken, name):  # noqa: F811
    D, row, col, val = matrix()
    rp, col, val = spx.spx_build_csr(M, K, row, col, val)
    A, B = spx.Csr(M, K, rp, col, val), torch.randint(-3, 4, (K, 32), device="cuda").float()
    spx.spx_spmm_csr(A, B, torch.zeros(M, 32, device="cuda"))
    refused = {"build": lambda s: spx.spx_build_csr(M, K, row, col, val, stream=s),
               "transpose": lambda s: spx.spx_transpose_csr(M, K, rp, col, val, stream=s),
               "bsr": lambda s: spx.spx_build_bsr(M, K, rp, col, val, 4, 4, stream=s),
               "wcsr": lambda s: spx.spx_build_wcsr(M, K, rp, col, val, stream=s),
               "check": lambda s: spx._check(spx.spx_check_csr(M, K, rp, col, stream=s), "spx_check_csr"),
               "plan": lambda s: spx.spx_plan_csr(M, K, val.numel(), rp, stream=s)}[name]
    with pytest.raises(spx.SpxError, match="SPX_ERR_CUDA|SPX_ERR_NOMEM"):
        refused(broken)
    C = spx.spx_spmm_csr(A, B, torch.full((M, 32), 7.0, device="cuda"))
    assert torch.equal(C, D @ B)
