"""Refusals of the routed-expert calls (no GPU): a rejected argument gives the documented status and
launches nothing; the binding refuses operands whose layout it would have to copy."""
import ctypes

import pytest
import torch

from csr_bsr_spmv_gb300 import spx

P = ctypes.c_void_p(4096)   # never dereferenced: every call here is refused on the host
ODD = ctypes.c_void_p(4097)
BIG = 2 ** 31 - 1


def refused(name, args, status):
    lib = spx._lib()
    before = spx.launch_count()
    rc = getattr(lib, name)(*args)
    assert spx.STATUS[rc] == status, (name, args, spx.STATUS.get(rc, rc))
    assert spx.launch_count() == before


@pytest.mark.parametrize("change,status", [
    ({0: -1}, "SPX_ERR_ARG"), ({1: 0}, "SPX_ERR_ARG"), ({2: 0}, "SPX_ERR_ARG"), ({2: 2049}, "SPX_ERR_UNSUPPORTED"),
    ({3: None}, "SPX_ERR_ARG"), ({4: 2}, "SPX_ERR_ARG"), ({5: 1}, "SPX_ERR_ARG"), ({6: None}, "SPX_ERR_ARG"),
    ({7: None}, "SPX_ERR_ARG"), ({8: None}, "SPX_ERR_ARG"), ({0: BIG, 1: 2}, "SPX_ERR_INDEX_RANGE"),
    ({0: 70000, 9: None}, "SPX_ERR_ARG"), ({0: 70000, 10: 16}, "SPX_ERR_ARG"), ({3: ODD}, "SPX_ERR_ALIGN"),
    ({8: ODD}, "SPX_ERR_ALIGN")])
def test_route_build_refuses(change, status):
    a = [100, 2, 8, P, 4, 2, P, P, P, P, 1 << 20, None]
    for i, v in change.items():
        a[i] = v
    refused("spx_route_build", a, status)


def test_route_scratch_bytes():
    lib = spx._lib()
    assert lib.spx_route_scratch_bytes(1, 8, 64) == 0
    assert lib.spx_route_scratch_bytes(-1, 8, 64) == 0 and lib.spx_route_scratch_bytes(8, 0, 64) == 0
    assert 0 < lib.spx_route_scratch_bytes(1 << 20, 8, 64) <= 1 << 20


@pytest.mark.parametrize("change,status", [
    ({0: -1}, "SPX_ERR_ARG"), ({1: 0}, "SPX_ERR_ARG"), ({2: -1}, "SPX_ERR_ARG"), ({3: 4}, "SPX_ERR_ARG"),
    ({4: None}, "SPX_ERR_ARG"), ({5: None}, "SPX_ERR_ARG"), ({6: None}, "SPX_ERR_ARG"), ({7: 63}, "SPX_ERR_ARG"),
    ({8: None}, "SPX_ERR_ARG"), ({9: 0}, "SPX_ERR_ARG"), ({6: ODD}, "SPX_ERR_ALIGN"), ({4: ODD}, "SPX_ERR_ALIGN"),
    ({0: BIG}, "SPX_ERR_INDEX_RANGE")])
def test_route_gather_refuses(change, status):
    a = [10, 2, 64, 1, P, P, P, 64, P, 64, None]
    for i, v in change.items():
        a[i] = v
    refused("spx_route_gather", a, status)


@pytest.mark.parametrize("change,status", [
    ({0: -1}, "SPX_ERR_ARG"), ({3: 3}, "SPX_ERR_ARG"), ({4: None}, "SPX_ERR_ARG"), ({6: None}, "SPX_ERR_ARG"),
    ({7: 63}, "SPX_ERR_ARG"), ({8: None}, "SPX_ERR_ARG"), ({9: 63}, "SPX_ERR_ARG"), ({5: ODD}, "SPX_ERR_ALIGN"),
    ({8: ODD}, "SPX_ERR_ALIGN"), ({1: BIG}, "SPX_ERR_INDEX_RANGE")])
def test_route_combine_refuses(change, status):
    a = [10, 2, 64, 1, P, P, P, 64, P, 64, None]
    for i, v in change.items():
        a[i] = v
    refused("spx_route_combine", a, status)


@pytest.mark.parametrize("change,status", [
    ({0: -1}, "SPX_ERR_ARG"), ({3: 3}, "SPX_ERR_ARG"), ({4: None}, "SPX_ERR_ARG"), ({5: None}, "SPX_ERR_ARG"),
    ({7: None}, "SPX_ERR_ARG"), ({8: 1}, "SPX_ERR_ARG"), ({9: None}, "SPX_ERR_ARG"), ({10: 63}, "SPX_ERR_ARG"),
    ({11: None}, "SPX_ERR_ARG"), ({12: 63}, "SPX_ERR_ARG"), ({13: ODD}, "SPX_ERR_ALIGN"), ({7: ODD}, "SPX_ERR_ALIGN")])
def test_route_combine_grad_refuses(change, status):
    a = [10, 2, 64, 2, P, P, P, P, 64, P, 64, P, 64, P, None]
    for i, v in change.items():
        a[i] = v
    refused("spx_route_combine_grad", a, status)


@pytest.mark.parametrize("change,status", [
    ({0: 0}, "SPX_ERR_ARG"), ({0: 2049}, "SPX_ERR_UNSUPPORTED"), ({1: -1}, "SPX_ERR_ARG"), ({2: -1}, "SPX_ERR_ARG"),
    ({3: -1}, "SPX_ERR_ARG"), ({4: None}, "SPX_ERR_ARG"), ({5: None}, "SPX_ERR_ARG"), ({6: 31}, "SPX_ERR_ARG"),
    ({7: None}, "SPX_ERR_ARG"), ({8: 31}, "SPX_ERR_ARG"), ({9: -1}, "SPX_ERR_ARG"), ({10: 2}, "SPX_ERR_ARG"),
    ({10: 1, 8: 63}, "SPX_ERR_ARG"), ({11: 0}, "SPX_ERR_ARG"), ({11: 3}, "SPX_ERR_ARG"), ({12: None}, "SPX_ERR_ARG"),
    ({13: 63}, "SPX_ERR_ARG"), ({14: 2}, "SPX_ERR_ARG"), ({5: ODD}, "SPX_ERR_ALIGN"), ({4: ODD}, "SPX_ERR_ALIGN")])
def test_gemm_grouped_refuses(change, status):
    a = [4, 100, 64, 32, P, P, 32, P, 32, 2048, 0, 1, P, 64, 1, None]
    for i, v in change.items():
        a[i] = v
    refused("spx_gemm_grouped", a, status)


@pytest.mark.parametrize("change,status", [
    ({0: 0}, "SPX_ERR_ARG"), ({0: 2049}, "SPX_ERR_UNSUPPORTED"), ({1: -1}, "SPX_ERR_ARG"), ({4: None}, "SPX_ERR_ARG"),
    ({5: None}, "SPX_ERR_ARG"), ({6: 63}, "SPX_ERR_ARG"), ({7: None}, "SPX_ERR_ARG"), ({8: 31}, "SPX_ERR_ARG"),
    ({9: 0}, "SPX_ERR_ARG"), ({10: None}, "SPX_ERR_ARG"), ({11: 31}, "SPX_ERR_ARG"), ({12: 0}, "SPX_ERR_ARG"),
    ({13: 2}, "SPX_ERR_ARG"), ({10: ODD}, "SPX_ERR_ALIGN")])
def test_gemm_grouped_wgrad_refuses(change, status):
    a = [4, 100, 64, 32, P, P, 64, P, 32, 1, P, 32, 2048, 1, None]
    for i, v in change.items():
        a[i] = v
    refused("spx_gemm_grouped_wgrad", a, status)


@pytest.mark.parametrize("change,status", [
    ({0: -1}, "SPX_ERR_ARG"), ({1: -1}, "SPX_ERR_ARG"), ({2: 3}, "SPX_ERR_ARG"), ({3: None}, "SPX_ERR_ARG"),
    ({4: 31}, "SPX_ERR_ARG"), ({5: None}, "SPX_ERR_ARG"), ({6: 31}, "SPX_ERR_ARG"), ({7: None}, "SPX_ERR_ARG"),
    ({3: ODD}, "SPX_ERR_ALIGN"), ({7: ODD}, "SPX_ERR_ALIGN")])
def test_quant_rows_refuses(change, status):
    a = [10, 32, 1, P, 32, P, 32, P, None]
    for i, v in change.items():
        a[i] = v
    refused("spx_quant_rows_i8", a, status)


@pytest.mark.parametrize("change,status", [
    ({0: 0}, "SPX_ERR_ARG"), ({0: 2049}, "SPX_ERR_UNSUPPORTED"), ({3: 131072, 6: 131072, 9: 131072}, "SPX_ERR_UNSUPPORTED"),
    ({4: None}, "SPX_ERR_ARG"), ({5: None}, "SPX_ERR_ARG"), ({6: 31}, "SPX_ERR_ARG"), ({7: None}, "SPX_ERR_ARG"),
    ({8: None}, "SPX_ERR_ARG"), ({9: 31}, "SPX_ERR_ARG"), ({10: -1}, "SPX_ERR_ARG"), ({11: None}, "SPX_ERR_ARG"),
    ({12: None}, "SPX_ERR_ARG"), ({13: 63}, "SPX_ERR_ARG"), ({14: 3}, "SPX_ERR_ARG"), ({11: ODD}, "SPX_ERR_ALIGN")])
def test_gemm_i8_refuses(change, status):
    a = [4, 100, 64, 32, P, P, 32, P, P, 32, 2048, P, P, 64, 1, P, 1 << 40, None]
    for i, v in change.items():
        a[i] = v
    refused("spx_gemm_i8", a, status)


def test_sizes_of_zero_launch_nothing():
    lib = spx._lib()
    before = spx.launch_count()
    assert lib.spx_route_gather(0, 2, 64, 1, None, None, None, 64, None, 64, None) == 0
    assert lib.spx_route_combine(10, 2, 0, 1, None, None, None, 0, None, 0, None) == 0
    assert lib.spx_gemm_grouped(4, 0, 64, 32, None, None, 32, None, 32, 0, 0, 1, None, 64, 1, None) == 0
    assert lib.spx_gemm_grouped_wgrad(4, 10, 0, 32, None, None, 0, None, 32, 1, None, 32, 0, 1, None) == 0
    assert lib.spx_gemm_i8(1, 0, 64, 32, None, None, 32, None, None, 32, 0, None, None, 64, 1, None, 0, None) == 0
    assert lib.spx_quant_rows_i8(0, 32, 1, None, 32, None, 32, None, None) == 0
    assert spx.launch_count() == before


def test_binding_refuses_layouts_and_host_tensors():
    r = spx.Route(4, 2, 3, torch.zeros(4, dtype=torch.int32), torch.zeros(8, dtype=torch.int32),
                  torch.zeros(8, dtype=torch.int32))
    X = torch.zeros(4, 16)
    off = torch.zeros(4, dtype=torch.int32)
    W = torch.zeros(3, 8, 16, dtype=torch.bfloat16)
    A = torch.zeros(8, 16, dtype=torch.bfloat16)
    for call in (lambda: spx.spx_route_build(torch.zeros(4, 2), 3),
                 lambda: spx.spx_route_build(torch.zeros(2, 4, dtype=torch.int32).t(), 3),
                 lambda: spx.spx_route_gather(r, X),                         # a host tensor
                 lambda: spx.spx_route_gather(r, torch.zeros(16, 4).t()),
                 lambda: spx.spx_route_gather(r, torch.zeros(5, 16)),
                 lambda: spx.spx_route_combine(r, torch.zeros(7, 16)),
                 lambda: spx.spx_route_combine(r, torch.zeros(8, 16), torch.zeros(8, dtype=torch.float64)),
                 lambda: spx.spx_route_combine_grad(r, X, torch.zeros(8, 15)),
                 lambda: spx.spx_gemm_grouped(off, A, W, layout="nn"),
                 lambda: spx.spx_gemm_grouped(off, A, W.transpose(1, 2)),
                 lambda: spx.spx_gemm_grouped(off, A[:, :8], W),
                 lambda: spx.spx_gemm_grouped(off.long(), A, W),
                 lambda: spx.spx_gemm_grouped(off, A, W, C=torch.zeros(8, 9, dtype=torch.bfloat16)),
                 lambda: spx.spx_gemm_grouped_wgrad(off, A[:5], A),
                 lambda: spx.spx_gemm_grouped_wgrad(off, A, A, dW=torch.zeros(2, 16, 16, dtype=torch.bfloat16)),
                 lambda: spx.spx_quant_rows_i8(A, torch.zeros(8, 15, dtype=torch.int8)),
                 lambda: spx.spx_gemm_i8(A, torch.zeros(8), W.to(torch.int8), torch.zeros(3, 8), offsets=off),
                 lambda: spx.spx_gemm_i8(A.to(torch.int8), torch.zeros(7), W.to(torch.int8), torch.zeros(3, 8), offsets=off)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        spx._type(torch.zeros(2, dtype=torch.float64))


def test_gemm_i8_scratch_bytes():
    lib = spx._lib()
    assert lib.spx_gemm_i8_scratch_bytes(8, 0, 64, 64, 0) == 0
    assert lib.spx_gemm_i8_scratch_bytes(8, 8 * 128, 64, 64, 1) == 0       # wide rows, few an expert
    assert lib.spx_gemm_i8_scratch_bytes(8, 8 * 128, 64, 64, 0) == 2 * 64 * (8 * 128 + 8 * 64)
    assert lib.spx_gemm_i8_scratch_bytes(8, 8 * 128 + 1, 64, 57, 1) == (2 * 64 * (8 * 128 + 1) + 255) // 256 * 256 + 2 * 64 * 8 * 64
    assert lib.spx_gemm_i8_scratch_bytes(2048, 1 << 20, 1 << 14, 1 << 14, 1) > 1 << 40  # past 32 bits
