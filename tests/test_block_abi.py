"""Refusals of the norm, gated-product and embedding calls (no GPU): a rejected argument gives the documented status and
launches nothing; the binding refuses operands whose layout it would have to copy."""
import ctypes

import pytest
import torch

from csr_bsr_spmv_gb300 import spx

P = ctypes.c_void_p(4096)   # never dereferenced: every call here is refused on the host
ODD = ctypes.c_void_p(4097)
BIG = 2 ** 31 - 1
NAN = float("nan")


def refused(name, args, change, status):
    a = list(args)
    for i, v in change.items():
        a[i] = v
    lib = spx._lib()
    before = spx.launch_count()
    rc = getattr(lib, name)(*a)
    assert spx.STATUS[rc] == status, (name, a, spx.STATUS.get(rc, rc))
    assert spx.launch_count() == before


ARG, RANGE, ALIGN, UNSUP = "SPX_ERR_ARG", "SPX_ERR_INDEX_RANGE", "SPX_ERR_ALIGN", "SPX_ERR_UNSUPPORTED"


@pytest.mark.parametrize("change,status", [
    ({0: -1}, ARG), ({1: 0}, ARG), ({1: 32769}, UNSUP), ({0: BIG}, RANGE), ({2: 3}, ARG), ({3: None}, ARG), ({4: 63}, ARG),
    ({6: 63}, ARG), ({8: 2}, ARG), ({9: -1.0}, ARG), ({9: NAN}, ARG), ({11: 63}, ARG), ({12: None}, ARG), ({13: 63}, ARG),
    ({3: ODD}, ALIGN), ({5: ODD}, ALIGN), ({7: ODD}, ALIGN), ({10: ODD}, ALIGN), ({14: ODD}, ALIGN)])
@pytest.mark.parametrize("name", ["spx_rms_norm", "spx_rms_norm_i8"])
def test_rms_norm_refuses(name, change, status):
    refused(name, [10, 64, 1, P, 64, P, 64, P, 1, 1e-6, P, 64, P, 64, P, None], change, status)


def test_rms_norm_refuses_its_outputs():
    refused("spx_rms_norm", [10, 64, 1, P, 64, P, 64, P, 1, 1e-6, P, 64, ODD, 64, P, None], {}, ALIGN)
    refused("spx_rms_norm_i8", [10, 64, 1, P, 64, P, 64, P, 1, 1e-6, P, 64, P, 64, None, None], {}, ARG)


@pytest.mark.parametrize("change,status", [
    ({0: -1}, ARG), ({1: 0}, ARG), ({1: 32769}, UNSUP), ({0: BIG}, RANGE), ({2: 3}, ARG), ({3: None}, ARG), ({4: 63}, ARG),
    ({5: None}, ARG), ({6: 63}, ARG), ({7: None}, ARG), ({9: 2}, ARG), ({11: 63}, ARG), ({12: None}, ARG), ({13: 63}, ARG),
    ({0: 10000, 15: None}, ARG), ({0: 10000, 16: 64}, ARG), ({3: ODD}, ALIGN), ({5: ODD}, ALIGN), ({7: ODD}, ALIGN),
    ({8: ODD}, ALIGN), ({10: ODD}, ALIGN), ({12: ODD}, ALIGN), ({14: ODD}, ALIGN), ({0: 10000, 15: ODD}, ALIGN)])
def test_rms_norm_grad_refuses(change, status):
    refused("spx_rms_norm_grad", [10, 64, 1, P, 64, P, 64, P, P, 1, P, 64, P, 64, P, P, 1 << 30, None], change, status)


def test_rms_norm_grad_scratch_bytes():
    need = spx._lib().spx_rms_norm_grad_scratch_bytes
    assert need(1, 4096) == need(0, 64) == need(-1, 64) == need(64, 0) == need(64, 32769) == 0
    assert 0 < need(100000, 4096) <= 456 * 4096 * 4
    assert 0 < need(BIG - (1 << 23), 32768) <= 456 * 32768 * 4


@pytest.mark.parametrize("change,status", [
    ({0: 0}, ARG), ({0: 2049}, UNSUP), ({1: -1}, ARG), ({2: -1}, ARG), ({3: -1}, ARG), ({2: 1 << 30}, RANGE), ({4: None}, ARG),
    ({5: None}, ARG), ({6: 31}, ARG), ({7: None}, ARG), ({8: 31}, ARG), ({9: -1}, ARG), ({10: 3}, ARG), ({11: 0}, ARG),
    ({11: 3}, ARG), ({13: 127}, ARG), ({14: None}, ARG), ({15: 63}, ARG), ({16: 2}, ARG), ({4: ODD}, ALIGN), ({5: ODD}, ALIGN),
    ({7: ODD}, ALIGN), ({12: ODD}, ALIGN), ({14: ODD}, ALIGN)])
def test_gated_refuses(change, status):
    refused("spx_gemm_grouped_gated", [4, 100, 64, 32, P, P, 32, P, 32, 4096, 0, 1, P, 128, P, 64, 1, None], change, status)


@pytest.mark.parametrize("change,status", [
    ({0: 0}, ARG), ({0: 2049}, UNSUP), ({1: -1}, ARG), ({2: -1}, ARG), ({3: -1}, ARG), ({2: 1 << 30}, RANGE), ({4: None}, ARG),
    ({5: None}, ARG), ({6: 31}, ARG), ({7: None}, ARG), ({8: 63}, ARG), ({9: -1}, ARG), ({10: 2}, ARG), ({10: 0, 8: 31}, ARG),
    ({11: -1}, ARG), ({12: 0}, ARG), ({13: None}, ARG), ({14: 127}, ARG), ({15: None}, ARG), ({16: 127}, ARG), ({18: 63}, ARG),
    ({4: ODD}, ALIGN), ({5: ODD}, ALIGN), ({7: ODD}, ALIGN), ({13: ODD}, ALIGN), ({15: ODD}, ALIGN), ({17: ODD}, ALIGN)])
def test_gated_grad_refuses(change, status):
    refused("spx_gemm_grouped_gated_grad", [4, 100, 64, 32, P, P, 32, P, 64, 2048, 1, 0, 1, P, 128, P, 128, P, 64, None], change,
            status)


@pytest.mark.parametrize("change,status", [
    ({0: -1}, ARG), ({1: -1}, ARG), ({2: -1}, ARG), ({0: BIG}, RANGE), ({3: 3}, ARG), ({4: None}, ARG), ({5: 2}, ARG),
    ({6: None}, ARG), ({7: 63}, ARG), ({9: None}, ARG), ({10: 63}, ARG), ({4: ODD}, ALIGN), ({6: ODD}, ALIGN), ({9: ODD}, ALIGN)])
def test_embed_refuses(change, status):
    refused("spx_embed", [10, 64, 1000, 1, P, 8, P, 64, 1.0, P, 64, None], change, status)


@pytest.mark.parametrize("change,status", [
    ({0: -1}, ARG), ({1: -1}, ARG), ({2: -1}, ARG), ({2: BIG}, RANGE), ({1: 1 << 24}, UNSUP), ({3: 3}, ARG), ({4: None}, ARG), ({5: 2}, ARG),
    ({8: None}, ARG), ({9: 63}, ARG), ({10: None}, ARG), ({11: 63}, ARG), ({12: 2}, ARG), ({14: None}, ARG), ({15: 100}, ARG),
    ({4: ODD}, ALIGN), ({8: ODD}, ALIGN), ({10: ODD}, ALIGN), ({14: ODD}, ALIGN)])
def test_embed_grad_refuses(change, status):
    refused("spx_embed_grad", [10, 64, 1000, 1, P, 8, -1, 1.0, P, 64, P, 64, 1, 0, P, 1 << 30, None], change, status)


def test_embed_grad_scratch_bytes():
    need = spx._lib().spx_embed_grad_scratch_bytes
    assert need(-1, 4) == need(4, -1) == need(BIG, 4) == need(4, BIG) == 0
    assert need(0, 64) > 0 and need(16384, 2048) >= 2 * 4 * 16384
    assert need(1 << 30, 8192) > 1 << 33


def test_sizes_of_zero_launch_nothing():
    lib = spx._lib()
    before = spx.launch_count()
    assert lib.spx_rms_norm(0, 64, 1, None, 64, None, 0, None, 1, 1e-6, None, 0, None, 64, None, None) == 0
    assert lib.spx_rms_norm_i8(0, 64, 1, None, 64, None, 0, None, 1, 1e-6, None, 0, None, 64, None, None) == 0
    assert lib.spx_rms_norm_grad(0, 64, 1, None, 64, None, 64, None, None, 1, None, 0, None, 64, None, None, 0, None) == 0
    assert lib.spx_gemm_grouped_gated(4, 0, 64, 32, None, None, 32, None, 32, 0, 0, 1, None, 0, None, 64, 1, None) == -1
    assert lib.spx_gemm_grouped_gated(1, 0, 64, 32, None, None, 32, None, 32, 0, 0, 1, None, 0, None, 64, 1, None) == 0
    assert lib.spx_gemm_grouped_gated_grad(1, 5, 0, 32, None, None, 32, None, 0, 0, 1, 0, 1, None, 0, None, 0, None, 0, None) == 0
    assert lib.spx_embed(0, 64, 10, 1, None, 8, None, 64, 1.0, None, 64, None) == 0
    assert lib.spx_embed_grad(0, 64, 10, 1, None, 8, -1, 1.0, None, 64, None, 64, 1, 1, None, 0, None) == 0
    assert spx.launch_count() == before


def test_binding_refuses_layouts_and_host_tensors():
    X, w = torch.zeros(4, 16), torch.zeros(16)
    A, W = torch.zeros(8, 16, dtype=torch.bfloat16), torch.zeros(3, 8, 16, dtype=torch.bfloat16)
    off, ids = torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.int64)
    H = torch.zeros(8, 8, dtype=torch.bfloat16)
    for call in (lambda: spx.spx_rms_norm(X, w),                                 # host tensors
                 lambda: spx.spx_rms_norm(torch.zeros(16, 4).t(), w),
                 lambda: spx.spx_rms_norm(torch.zeros(16), w),
                 lambda: spx.spx_rms_norm_i8(X, w.double()),
                 lambda: spx.spx_rms_norm_grad(X, X, torch.zeros(4), w),
                 lambda: spx.spx_gemm_grouped_gated(off, A, W),
                 lambda: spx.spx_gemm_grouped_gated(off, A, W, act="relu"),
                 lambda: spx.spx_gemm_grouped_gated(None, A, W),
                 lambda: spx.spx_gemm_grouped_gated_grad(off, A, W, H, layout="nn"),
                 lambda: spx.spx_embed(ids.float(), X),
                 lambda: spx.spx_embed(ids, X),
                 lambda: spx.spx_embed_grad(ids, X[:3], 10),
                 lambda: spx.spx_embed_grad(ids, X, 10, accumulate=True)):
        with pytest.raises(ValueError):
            call()
