"""Sizes near 2^31 of the routed-expert calls (no GPU): beyond 2^31 - 2^23 - 1 an int index that steps past its end
by a grid could wrap, so such sizes are refused before anything is launched."""
import ctypes

import pytest

from csr_bsr_spmv_gb300 import spx

P = ctypes.c_void_p(4096)  # never dereferenced: every call here is refused on the host
OVER = 2 ** 31 - 2 ** 23

CALLS = {
    "spx_route_gather": ([10, 1, 64, 1, P, P, P, OVER, P, OVER, None], (0, 1, 2)),
    "spx_route_combine": ([10, 1, 64, 1, P, P, P, OVER, P, OVER, None], (0, 1, 2)),
    "spx_route_combine_grad": ([10, 1, 64, 2, P, P, P, P, OVER, P, OVER, P, OVER, P, None], (0, 1, 2)),
    "spx_gemm_grouped": ([1, 100, 64, 32, P, P, OVER, P, OVER, 0, 0, 1, P, OVER, 1, None], (1, 2, 3)),
    "spx_gemm_grouped_wgrad": ([1, 100, 64, 32, P, P, OVER, P, OVER, 1, P, OVER, 0, 1, None], (1, 2, 3)),
    "spx_quant_rows_i8": ([10, 32, 1, P, OVER, P, OVER, P, None], (0, 1)),
    "spx_gemm_i8": ([1, 100, 64, 32, None, P, 32, P, P, 32, 0, P, P, OVER, 1, P, 1 << 60, None], (1, 2)),
    "spx_route_build": ([100, 1, 8, P, 4, OVER, P, P, P, P, 1 << 60, None], (0, 1)),
}


@pytest.mark.parametrize("name,at", [(n, i) for n, (_, where) in CALLS.items() for i in where])
@pytest.mark.parametrize("size", [OVER, 2 ** 31 - 1])
def test_sizes_that_could_wrap_are_refused(name, at, size):
    args = list(CALLS[name][0])
    if name.startswith("spx_route") and at < 2:
        args[0] = args[1] = 1  # the product of the two is the number of slots
    args[at] = size
    if name == "spx_route_build" and at == 1:
        args[5] = size
    before = spx.launch_count()
    rc = getattr(spx._lib(), name)(*args)
    assert spx.STATUS.get(rc, rc) == "SPX_ERR_INDEX_RANGE"
    assert spx.launch_count() == before
