"""A call that CUDA refuses on the host -- here on a stream whose capture another call has ended -- gives SPX_ERR_CUDA, and
nothing of it is left for the next call, which is in order and says so."""
import ctypes

import pytest
import torch

from block_util import BF16, normal, offsets_of, whole
from csr_bsr_spmv_gb300 import spx

pytestmark = pytest.mark.gpu
RELAXED = 2


@pytest.fixture
def broken():
    """A stream on which a capture was begun and broken: every launch on it is refused until the capture is ended."""
    torch.cuda.init()
    rt = ctypes.CDLL(f"libcudart.so.{torch.version.cuda.split('.')[0]}")
    stream = torch.cuda.Stream()
    handle = ctypes.c_void_p(stream.cuda_stream)
    torch.cuda.synchronize()
    assert rt.cudaStreamBeginCapture(handle, RELAXED) == 0
    assert rt.cudaStreamSynchronize(handle) != 0
    rt.cudaGetLastError()
    yield stream
    graph = ctypes.c_void_p()
    assert rt.cudaStreamEndCapture(handle, ctypes.byref(graph)) != 0 and not graph
    rt.cudaGetLastError()


def calls():
    """name: (call with a stream, what it writes)"""
    X, ids = whole(1, 40, 64, dtype=BF16), torch.arange(40, device="cuda") % 7
    Y, dX, dW = torch.empty_like(X), torch.empty_like(X), torch.zeros(7, 64, dtype=BF16, device="cuda")
    rstd, C, C2 = torch.ones(40, device="cuda"), torch.empty(40, 32, dtype=BF16, device="cuda"), torch.empty(40, 16, dtype=BF16, device="cuda")
    W, off, W2 = normal(2, 1, 32, 64, dtype=BF16), offsets_of([40]), normal(3, 1, 32, 64, dtype=BF16)
    scratch = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    return {
        "norm": (lambda s: spx.spx_rms_norm(X, Y=Y, stream=s), Y),
        "norm_grad": (lambda s: spx.spx_rms_norm_grad(X, X, rstd, dX=dX, dweight=False, stream=s), dX),
        "embed": (lambda s: spx.spx_embed(ids, X[:7], Y=Y, stream=s), Y),
        "embed_grad": (lambda s: spx.spx_embed_grad(ids, X, 7, dW=dW, stream=s, scratch=scratch), dW),
        "product": (lambda s: spx.spx_gemm_grouped(off, X, W, C=C, stream=s), C),
        "gated": (lambda s: spx.spx_gemm_grouped_gated(off, X, W2, C=C2, stream=s), C2),
    }


@pytest.mark.parametrize("after", ["norm", "norm_grad", "embed", "embed_grad", "product", "gated"])
@pytest.mark.parametrize("name", ["norm", "norm_grad", "embed", "embed_grad", "product", "gated"])
def test_the_next_call_is_not_refused(broken, name, after):
    ops = calls()
    ops[after][0](None)
    want = ops[after][1].clone()
    ops[after][1].fill_(5)
    with pytest.raises(spx.SpxError, match="SPX_ERR_CUDA"):
        ops[name][0](broken)
    ops[after][0](None)
    assert torch.equal(ops[after][1], want)


def test_a_refused_wait_for_device_errors_leaves_nothing(broken):
    ops = calls()
    lib = spx._lib()
    assert lib.spx_last_device_error(broken.cuda_stream) != 0
    ops["norm"][0](None)
    assert spx.spx_last_device_error() == 0
