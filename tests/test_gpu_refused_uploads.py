"""An upload, or a product on host vectors, that CUDA refuses on the host -- on a stream whose capture was broken off -- leaves
nothing for the product that follows it."""
import numpy as np
import pytest
import torch

from csr_bsr_spmv_gb300 import spx
from test_gpu_refused_builds import K, M, matrix
from test_gpu_refused_calls import broken  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["sell", "sell built on the device", "wcsr plan", "bsr plan", "hostio"])
def test_the_next_product_is_not_refused(broken, name):  # noqa: F811
    D, row, col, val = matrix()
    rp, col, val = spx.spx_build_csr(M, K, row, col, val)
    A, B = spx.Csr(M, K, rp, col, val), torch.randint(-3, 4, (K, 32), device="cuda").float()
    plan = spx.spx_plan_csr(M, K, val.numel(), rp)
    spx.spx_spmm_csr(A, B, torch.zeros(M, 32, device="cuda"))
    host, windows = [t.cpu().numpy() for t in (rp, col, val)], np.array([0, 200, 300], np.int32)
    refused = {"sell": lambda s: spx.Sell(M, K, *host, stream=s),
               "sell built on the device": lambda s: spx.Sell(M, K, rp, col, val, stream=s),
               "wcsr plan": lambda s: spx.WcsrPlan(128, 300, windows, max_chunks=16, device="cuda", stream=s),
               "bsr plan": lambda s: spx.BsrPlan(128, 300, windows, max_chunks=16, device="cuda", stream=s),
               "hostio": lambda s: spx.spx_spmv_csr_hostio(plan, A, torch.ones(1, K), torch.zeros(1, M), stream=s)}[name]
    with pytest.raises(spx.SpxError, match="SPX_ERR_CUDA"):
        refused(broken)
    C = spx.spx_spmm_csr(A, B, torch.full((M, 32), 7.0, device="cuda"))
    assert torch.equal(C, D @ B)
