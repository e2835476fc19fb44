"""Gated products at the sizes where another form of their kernels takes over; references and tolerances are those of
tests/test_gpu_gated.py."""
import pytest
import torch

import gated_forms
from block_util import BF16, F16, close, normal, offsets_of, padded
from csr_bsr_spmv_gb300 import spx
from test_gpu_gated import backward, counts_of, forward, grad64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", gated_forms.GATE)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("pad", ["dense", "wide"])
def test_product_in_every_form(case, dtype, pad):
    """Dense rows of K on 16-byte boundaries; wide ones leave 8 values between them."""
    E, S, F, K = case
    forward(counts_of("even" if E > 20 else "uneven", E, S), F, K, dtype, "silu", 8 if pad == "wide" else 0)


@pytest.mark.parametrize("case", gated_forms.BACK)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_gradient_in_every_form(case, dtype, layout):
    E, S, F, N = case
    counts = counts_of("even" if E > 20 else "uneven", E, S)
    if layout == "kn" and F % 8:
        F += 8 - F % 8 if S < 1000 else 0  # rows of F on 16-byte boundaries, or the CUDA cores
    backward(counts, N, dtype, "gelu_tanh", layout, normal(F, S, 2 * F, dtype=dtype))


@pytest.mark.parametrize("F", [35, 43, 264, 520])
@pytest.mark.parametrize("S", [300, 9000])
def test_factors_off_their_boundaries(F, S):
    """Weights on 16-byte boundaries, but H, dH and C on rows of any width: stored value by value."""
    counts = counts_of("uneven", 4, S)
    for pad in (1, 3):
        W2 = normal(5, 4, 136, F + (-F) % 8, dtype=BF16, scale=F ** -0.5)[:, :, :F]
        H, dY = padded(normal(F, S, 2 * F, dtype=BF16), pad), normal(S, S, 136, dtype=BF16)
        out, C = padded(torch.zeros(S, 2 * F, dtype=BF16, device="cuda"), pad), padded(torch.zeros(S, F, dtype=BF16, device="cuda"), pad)
        dH, C2 = spx.spx_gemm_grouped_gated_grad(offsets_of(counts), dY, W2, H, dH=out, C=C)
        d, ed, c, ec = grad64(counts, dY, W2, "kn", H, "silu")
        close(dH, d, ed, "dH")
        close(C2, c, ec, "C")
