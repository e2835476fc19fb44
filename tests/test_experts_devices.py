"""The routed-expert bindings refuse operands of two devices and of a device that is not the current one, on which the
library would launch (no GPU: the operands are stand-ins that only know their shape and device)."""
import pytest
import torch

from csr_bsr_spmv_gb300 import spx

I32, F32, I8, BF16 = torch.int32, torch.float32, torch.int8, torch.bfloat16


class Far:
    """What the bindings ask of a tensor."""

    def __init__(self, shape, dtype, device):
        self.shape, self.dtype, self.device, self.is_cuda = tuple(shape), dtype, torch.device("cuda", device), True

    def stride(self):
        out = [1]
        for n in reversed(self.shape[1:]):
            out.insert(0, out[0] * n)
        return tuple(out)

    def numel(self):
        n = 1
        for m in self.shape:
            n *= m
        return n

    def get_device(self):
        return self.device.index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()


class Library:
    """Counts calls; every one succeeds."""
    calls = 0

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return lambda *a: 64

        def call(*a):
            Library.calls += 1
            return 0

        return call


T, K, E, H, N = 6, 2, 3, 16, 32
S = T * K


def calls(d):
    """Every binding, `d(i)` giving the device of its i-th operand: (number of operands, call)."""
    def route(i):
        return spx.Route(T, K, E, Far([E + 1], I32, d(i)), Far([S], I32, d(i)), Far([S], I32, d(i)))

    m = Far
    return {
        "build": (2, lambda s: spx.spx_route_build(m([T, K], I32, d(0)), E, scratch=m([64], I32, d(1)), stream=s)),
        "gather": (3, lambda s: spx.spx_route_gather(route(0), m([T, H], BF16, d(1)), m([S, H], BF16, d(2)), stream=s)),
        "combine": (4, lambda s: spx.spx_route_combine(route(0), m([S, H], BF16, d(1)), m([T, K], F32, d(2)),
                                                       m([T, H], BF16, d(3)), stream=s)),
        "grad": (5, lambda s: spx.spx_route_combine_grad(route(0), m([T, H], BF16, d(1)), m([S, H], BF16, d(2)),
                                                         m([T, K], F32, d(3)), m([S, H], BF16, d(4)), stream=s)),
        "product": (4, lambda s: spx.spx_gemm_grouped(m([E + 1], I32, d(0)), m([S, H], BF16, d(1)), m([E, N, H], BF16, d(2)),
                                                      m([S, N], BF16, d(3)), stream=s)),
        "gradient": (4, lambda s: spx.spx_gemm_grouped_wgrad(m([E + 1], I32, d(0)), m([S, N], BF16, d(1)), m([S, H], BF16, d(2)),
                                                             m([E, N, H], BF16, d(3)), stream=s)),
        "quant": (3, lambda s: spx.spx_quant_rows_i8(m([S, H], BF16, d(0)), m([S, H], I8, d(1)), m([S], F32, d(2)), stream=s)),
        "int8": (7, lambda s: spx.spx_gemm_i8(m([S, H], I8, d(0)), m([S], F32, d(1)), m([E, N, H], I8, d(2)), m([E, N], F32, d(3)),
                                              offsets=m([E + 1], I32, d(4)), C=m([S, N], F32, d(5)),
                                              scratch=m([64], torch.uint8, d(6)), stream=s)),
    }


@pytest.fixture
def fake(monkeypatch):
    monkeypatch.setattr(spx, "_lib", lambda lib=Library(): lib)
    monkeypatch.setattr(spx, "_new", lambda shape, dtype, like, stream: Far(
        [shape] if isinstance(shape, int) else shape, dtype, like.device.index))
    monkeypatch.setattr(spx, "_empty", lambda shape, dtype=None, device=None: Far(
        [shape] if isinstance(shape, int) else shape, dtype, device.index))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    Library.calls = 0


class Stream:
    cuda_stream = 0

    def __init__(self, device):
        self.device_index = device


@pytest.mark.parametrize("name", list(calls(lambda i: 0)))
def test_operands_of_another_device_are_refused(fake, name):
    n = calls(lambda i: 0)[name][0]
    calls(lambda i: 0)[name][1](None)
    calls(lambda i: 0)[name][1](Stream(0))
    assert Library.calls == 2
    for odd in range(n):
        with pytest.raises(ValueError):
            calls(lambda i: 1 if i == odd else 0)[name][1](None)
    with pytest.raises(ValueError):  # all together on a device that is not the current one
        calls(lambda i: 1)[name][1](None)
    with pytest.raises(ValueError):
        calls(lambda i: 0)[name][1](Stream(1))
    assert Library.calls == 2
