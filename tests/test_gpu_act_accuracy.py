"""The activations' stated accuracy, by every 16-bit value: C = act(x) of the gated product in fp32, on the tensor cores and
(K = 18) on the CUDA cores.

Stated: the logistic function within 2^-21 of itself, which its product with x, rounded by half a step (u = 2^-24), passes on
to SiLU; GELU within 2^-20.9 in all; the tanh form as SiLU, and besides 5 u |z| (1 - p) for its argument z (two rounded
constants, three roundings).  p below fp32's normal numbers, 2^-126, may be 0: |x| 2^-126."""
import numpy as np
import pytest
import torch

from block_util import BF16, F16, F32, U
from csr_bsr_spmv_gb300 import spx
from test_gpu_gated import act64

pytestmark = pytest.mark.gpu
STATED = {"silu": 2.0 ** -21 + U, "gelu": 2.0 ** -20.9, "gelu_tanh": 2.0 ** -21 + U}


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("K", [64, 18])
def test_activations_are_as_near_as_stated(act, dtype, K):
    x = torch.arange(-2 ** 15, 2 ** 15, device="cuda", dtype=torch.int32).to(torch.int16).view(dtype)
    x = x[x.abs().float() < 1e4]
    x = torch.cat([x, x[:-x.numel() % 8]]).view(-1, 8)
    A = torch.zeros(x.shape[0], K, device="cuda", dtype=dtype)
    A[:, :8], A[:, 8:16] = x, 1
    C, _ = spx.spx_gemm_grouped_gated(None, A, torch.eye(16, K, device="cuda", dtype=dtype), act=act, dtype=F32)
    a = act64(act, x.double())[0]
    err = STATED[act] * a.abs() + x.double().abs() * 2.0 ** -126 + 2.0 ** -126
    if act == "gelu_tanh":
        z = (8 / np.pi) ** 0.5 * (x.double() + 0.044715 * x.double() ** 3)
        err += 5 * U * z.abs() * torch.sigmoid(-z) * a.abs()
    off = (C.double() - a).abs()
    assert (off <= err).all(), (off / a.abs().clamp(min=1e-300))[a.abs() > 2.0 ** -100].max().log2().item()
