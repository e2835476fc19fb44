"""The bindings of the norm, the gated products and the embedding refuse operands of two devices and of a device that is
not the current one, on which the library would launch (no GPU: the operands are stand-ins)."""
import pytest
import torch

from csr_bsr_spmv_gb300 import spx
from test_experts_devices import BF16, F32, I32, Far, Library

S, E, H, F, V = 12, 3, 16, 8, 40
CALLS = [
    ("spx_rms_norm", dict(X=((S, H), BF16), weight=((H,), BF16), R=((S, H), BF16), Y=((S, H), BF16), S=((S, H), BF16)), {}),
    ("spx_rms_norm_i8", dict(X=((S, H), BF16), weight=((H,), F32), R=((S, H), BF16), Q=((S, H), torch.int8), scale=((S,), F32),
                             S=((S, H), BF16)), {}),
    ("spx_rms_norm_grad", dict(dY=((S, H), BF16), S=((S, H), BF16), rstd=((S,), F32), weight=((H,), BF16), dS=((S, H), BF16),
                               dX=((S, H), BF16)), dict(dweight=False)),
    ("spx_gemm_grouped_gated", dict(offsets=((E + 1,), I32), A=((S, H), BF16), W=((E, 2 * F, H), BF16), C=((S, F), BF16),
                                    H=((S, 2 * F), BF16)), {}),
    ("spx_gemm_grouped_gated_grad", dict(offsets=((E + 1,), I32), dY=((S, H), BF16), W=((E, H, F), BF16), H=((S, 2 * F), BF16),
                                         dH=((S, 2 * F), BF16), C=((S, F), BF16)), {}),
    ("spx_embed", dict(ids=((S,), torch.int64), W=((V, H), BF16), Y=((S, H), BF16)), {}),
    ("spx_embed_grad", dict(ids=((S,), torch.int64), dY=((S, H), BF16), dW=((V, H), BF16), scratch=((64,), torch.uint8)), dict(V=V)),
]


@pytest.fixture
def current(monkeypatch):
    monkeypatch.setattr(spx, "_lib", Library)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)


def call(name, operands, more, where):
    fn = getattr(spx, name)
    return fn(**{k: Far(shape, dtype, where.get(k, where[None])) for k, (shape, dtype) in operands.items()}, **more)


@pytest.mark.parametrize("name,operands,more", CALLS)
def test_operands_of_the_current_device_are_taken(current, name, operands, more):
    before = Library.calls
    call(name, operands, more, {None: 0})
    assert Library.calls == before + 1


@pytest.mark.parametrize("name,operands,more", CALLS)
def test_another_device_is_refused(current, name, operands, more):
    before = Library.calls
    with pytest.raises(ValueError):
        call(name, operands, more, {None: 1})
    for k in operands:
        with pytest.raises(ValueError):
            call(name, operands, more, {None: 0, k: 1})
    assert Library.calls == before
