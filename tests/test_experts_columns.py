"""The documented limit of the experts' products on the CUDA cores (no GPU): beyond 4194240 output columns they are refused,
and nothing is launched."""
import ctypes

import pytest

from csr_bsr_spmv_gb300 import spx

P = ctypes.c_void_p(4096)   # never dereferenced: every call here is refused on the host
MOST = 65535 * 64


@pytest.mark.parametrize("columns", [MOST + 1, 2 * MOST])
@pytest.mark.parametrize("depth", [0, 9])  # rows of 9 values lie off 16-byte boundaries; without any there is nothing to copy
def test_columns_past_the_limit_are_refused(columns, depth):
    lib, N, K = spx._lib(), columns, depth
    W = N | 1  # an odd pitch
    before = spx.launch_count()
    for rc in (lib.spx_gemm_grouped(1, 8, N, K, P, P, 9, P, 9, 0, 0, 1, P, N, 1, None),
               lib.spx_gemm_grouped(1, 8, N, K, P, P, 9, P, W, 0, 1, 1, P, N, 1, None),
               lib.spx_gemm_grouped_wgrad(1, 8, 9, N, P, P, 9, P, W, 1, P, W, 0, 1, None),
               lib.spx_gemm_grouped_gated(1, 8, N, K, None, P, 9, P, 9, 0, 0, 1, P, 2 * N, P, N, 1, None),
               lib.spx_gemm_grouped_gated_grad(1, 8, N, K, None, P, 9, P, W, 0, 1, 0, 1, P, 2 * N, P, 2 * N, P, N, None)):
        assert spx.STATUS[rc] == "SPX_ERR_UNSUPPORTED"
    assert spx.launch_count() == before
