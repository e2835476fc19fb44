"""Outputs of the norm and its gradient over their inputs, in every type: rows on 16-byte boundaries, in 4-byte pieces and
in shifted words, whose threads read words that other threads write, rows that are read twice, moved bases and pitches."""
import pytest
import torch

from block_util import BF16, F16, F32, between, normal, padded
from csr_bsr_spmv_gb300 import spx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pad", [0, 1, 3])
@pytest.mark.parametrize("H", [7, 40, 41, 1000, 1001, 1002, 4095, 6001, 8195, 9001, 16383, 16401, 20000, 20001])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_outputs_over_their_inputs(H, dtype, pad):
    M = 900 if H < 2000 else 320

    def at(t):
        return padded(t.clone(), pad)

    def same_pads(t, edges):
        return not pad or torch.equal(between(t, pad).nan_to_num(5), edges.nan_to_num(5))

    X, R, w = normal(1, M, H, dtype=dtype), normal(2, M, H, dtype=dtype), normal(3, H, dtype=dtype)
    Y, S, rstd = spx.spx_rms_norm(at(X), w, at(R), grad=True)
    for y, s in ((0, 1), (1, 0)):
        t = [at(X), at(R)]
        edges = [between(v, pad) for v in t] if pad else [None] * 2
        spx.spx_rms_norm(t[0], w, t[1], Y=t[y], S=t[s])
        assert torch.equal(t[y], Y) and torch.equal(t[s], S)
        assert all(same_pads(v, e) for v, e in zip(t, edges))
    r = at(R)
    Q, scale, _ = spx.spx_rms_norm_i8(at(X), w, r, S=r)
    Q0, scale0, _ = spx.spx_rms_norm_i8(at(X), w, at(R))
    assert torch.equal(r, S) and torch.equal(Q, Q0) and torch.equal(scale, scale0)
    dY, dS = normal(4, M, H, dtype=dtype), normal(5, M, H, dtype=dtype)
    dX, dw = spx.spx_rms_norm_grad(at(dY), at(S), rstd, w, dS=at(dS), dX=at(torch.zeros_like(S)))
    for i in range(3):
        t = [at(dY), at(S), at(dS)]
        edges = [between(v, pad) for v in t] if pad else [None] * 3
        out, dw2 = spx.spx_rms_norm_grad(t[0], t[1], rstd, w, dS=t[2], dX=t[i])
        assert out is t[i] and torch.equal(out, dX) and torch.equal(dw, dw2)
        assert all(same_pads(v, e) for v, e in zip(t, edges))
