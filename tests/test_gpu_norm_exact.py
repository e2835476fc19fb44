"""The norm's sums value by value, at lengths where a bound that grows with the length would hide a lost one.

Whole numbers (up to 6) and roots of two keep every sum exact in fp32: below 2^24 of its unit.  Then the norm's root, its
rows and its codes are single fp32 operations and one rounding to the type, compared bit for bit, and so are the weights'
gradients.  u = 2^-24."""
import pytest
import torch

from block_util import BF16, F16, F32, U, close, padded, whole
from csr_bsr_spmv_gb300 import spx

pytestmark = pytest.mark.gpu
SIZES = [(1, 1), (3, 7), (2, 64), (33, 1002), (2, 1031), (3, 4096), (9, 4097), (2, 5000), (3000, 4104), (4, 8192), (5, 8195), (2, 9001), (2, 16383), (2, 16384),
         (3, 16385), (2, 20000), (3, 20001), (3, 32766), (2, 32767), (2, 32768), (40000, 16), (5000, 130)]
TYPES = [F32, BF16, F16]


def positive(seed, *shape, dtype):
    """Whole numbers 1 to 3 with a sign, so that every one counts in a sum of squares."""
    return whole(seed, *shape, most=1).mul(2).add(whole(seed + 1, *shape, most=1)).add(0.5).sign().to(dtype) * whole(seed + 2, *shape, most=1).add(2).to(dtype)


@pytest.mark.parametrize("pad", [0, 1, 2])
@pytest.mark.parametrize("M,H", SIZES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_bit_for_bit(M, H, dtype, residual, pad):
    """rstd = 1 / sqrt(sum / H + eps) and y = (s rstd) w, each operation rounded once; a value left out of the sum, or counted
    twice, changes it by 1 of at most 36 H, which is 2^-20.2 of it or more: at least 3 steps of the root."""
    X = padded(positive(M + H, M, H, dtype=dtype), pad)
    R = padded(positive(H, M, H, dtype=dtype), pad) if residual else None
    w = padded((1 + whole(3, 1, H, most=2) / 4).to(dtype), pad)[0]
    s = X.float() + (R.float() if residual else 0)
    sums = s.double().square().sum(1)
    assert sums.max() < 2 ** 24
    eps = torch.tensor(2.0 ** -10, device="cuda")
    rstd = 1 / torch.sqrt(sums.float() / torch.tensor(float(H), device="cuda") + eps)
    y = s * rstd[:, None] * w.float()
    Y, S, r = spx.spx_rms_norm(X, w, R, eps=2.0 ** -10, grad=True)
    assert torch.equal(r, rstd) and torch.equal(Y, y.to(dtype))
    assert not residual or torch.equal(S, s.to(dtype))
    Q, scale, _ = spx.spx_rms_norm_i8(X, w, R, eps=2.0 ** -10)
    top = y.abs().max(1).values / torch.tensor(127.0, device="cuda")
    assert torch.equal(scale, top)
    assert torch.equal(Q, torch.where(top[:, None] > 0, torch.round(y / top[:, None]), 0.0).to(torch.int8))


@pytest.mark.parametrize("pad", [0, 1, 2])
@pytest.mark.parametrize("M,H", SIZES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("residual", [False, True])
def test_gradient_of_whole_numbers(M, H, dtype, residual, pad):
    """dweight is exact: at most 40000 products of up to 9.  So is the sum of dy w n (27 each, H of them, in units of 1/2); the
    mean's factor -1 / H and the product with it are rounded, then n mean + g once and, with dS, that sum once more: 3 u of
    n mean, u of the first sum, u of the result; the type's half step is of what was computed, so 2^-8 of all that more."""
    S, dY = padded(whole(M, M, H, dtype=dtype), pad), padded(whole(H + 1, M, H, dtype=dtype), pad)
    w = padded(positive(5, 1, H, dtype=dtype), pad)[0]
    dS = padded(whole(7, M, H, dtype=dtype), pad) if residual else None
    rstd = 2.0 ** -(torch.arange(M, device="cuda") % 2).float()
    dX, dw = spx.spx_rms_norm_grad(dY, S, rstd, w, dS=dS)
    n, g, r = S.double() * rstd.double()[:, None], dY.double() * w.double(), rstd.double()[:, None]
    assert ((g * n).abs().sum(1) < 2 ** 23).all()
    c = (g * n).sum(1, keepdim=True) / H
    want = r * (g - n * c)
    err = r * (3 * U * (n * c).abs() + U * (g - n * c).abs())
    if residual:
        want = want + dS.double()
    close(dX, want, (err + U * want.abs()) * (1 + 2 ** -8), "dX")
    assert torch.equal(dw.double(), (dY.double() * n).sum(0))


@pytest.mark.parametrize("pad", [0, 1, 2])
@pytest.mark.parametrize("H", [7, 64, 1002, 1031, 2048, 4095, 4096, 5000, 8192, 8195, 9001, 16383, 16384, 16385, 20001, 32767, 32768])
@pytest.mark.parametrize("dtype", TYPES)
def test_every_value_counts_in_the_gradients_sum(H, dtype, pad):
    """One value of dY a row, stepped over the row's ends and the ends of pieces and warps: the sum is that one product, and
    what is not 0 elsewhere in dX is n times its mean.  Left out, dX is 0 there; counted twice, twice as large."""
    at = {j for j in list(range(48)) + [H - 1 - i for i in range(48)] if 0 <= j < H}
    for step in (32, 128, 256, 512, 1024, 2048, 4096, 8192, 16384):
        for k in range(step, H, max(step, H // 16 // step * step)):
            at |= {j for j in (k - 1, k, k + 1) if j < H}
    at = torch.tensor(sorted(at), device="cuda")
    M = at.numel()
    S, w = padded(positive(1, M, H, dtype=dtype), pad), padded(positive(2, 1, H, dtype=dtype), pad)[0]
    dY = torch.zeros(M, H, dtype=dtype, device="cuda")
    dY[torch.arange(M, device="cuda"), at] = positive(3, M, dtype=dtype)
    dY = padded(dY, pad)
    rstd = torch.full((M,), 0.5, device="cuda")
    dX, dw = spx.spx_rms_norm_grad(dY, S, rstd, w)
    n, g = S.double() / 2, dY.double() * w.double()
    c = (g * n).sum(1, keepdim=True) / H
    assert (c != 0).all()
    want = (g - n * c) / 2
    close(dX, want, (3 * U * (n * c).abs() + U * (g - n * c).abs()) / 2 * (1 + 2 ** -8), "dX")
    assert torch.equal(dw.double(), (dY.double() * n).sum(0))
