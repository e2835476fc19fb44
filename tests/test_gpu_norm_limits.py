"""Where the norm's arithmetic ends: sums of squares at fp32's largest number, and eps 0.  No sums are compared here but those
that are exact or lie 2% from the border, of fp32 sums that are off by less than H u = 2^-9."""
import pytest
import torch

from block_util import BF16, F16, F32
from csr_bsr_spmv_gb300 import spx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H", [1, 4096, 4097, 32768, 32767])
def test_sums_of_squares_past_the_range_give_zeros(H, dtype):
    """Rows of one value v: H v^2 at 0.98 of 2^128 is a sum, at 1.02 there is none, though the mean is far inside the range."""
    root = (2.0 ** 128 / H) ** 0.5
    X = torch.zeros(3, H, dtype=F32, device="cuda")
    X[0], X[1], X[2] = root * 0.98 ** 0.5, root * 1.02 ** 0.5, 1
    X = X.to(dtype)
    sums = H * X.double()[:, 0].square() / 2.0 ** 128
    assert 0.97 < sums[0] < 0.99 and 1.01 < sums[1] < 1.03  # bf16's step moves them by less than 1%
    Y, _, rstd = spx.spx_rms_norm(X, grad=True)
    assert ((Y[[0, 2]].double() - 1).abs() <= 2 ** -7).all() and (rstd[[0, 2]] > 0).all()
    assert not Y[1].any() and rstd[1] == 0
    Q, scale, _ = spx.spx_rms_norm_i8(X)
    assert (Q[[0, 2]] == 127).all() and not Q[1].any() and scale[1] == 0


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("H", [5, 520, 4097, 20000])
def test_rows_of_zeros_need_an_eps(H, dtype):
    """The formula divides 0 by 0 for a row of zeros and eps 0: NaN, codes 0 and a scale of NaN.  Other rows do not mind."""
    X = torch.ones(4, H, dtype=dtype, device="cuda")
    X[2] = 0
    for eps in (0.0, 2.0 ** -30):
        Y, _, rstd = spx.spx_rms_norm(X, eps=eps, grad=True)
        Q, scale, _ = spx.spx_rms_norm_i8(X, eps=eps)
        for i in (0, 1, 3):
            assert (Y[i] == 1).all() and rstd[i] == 1 and (Q[i] == 127).all()
        assert not Q[2].any()
        if eps:
            assert not Y[2].any() and rstd[2] == 2.0 ** 15 and scale[2] == 0
        else:
            assert Y[2].isnan().all() and rstd[2] == float("inf") and scale[2].isnan()
