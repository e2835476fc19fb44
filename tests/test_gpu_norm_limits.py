"""Where the norm's arithmetic ends: sums of squares at fp32's largest number.  The sums lie 2% from the border, and
fp32 sums are off by less than H u = 2^-9."""
import pytest
import torch

from block_util import BF16, F32
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
