"""The table's gradient of the longest rows it takes: the grid of every launch stays within its limits at each width of a piece."""
import pytest
import torch

from block_util import BF16, F16, F32, whole
from csr_bsr_spmv_gb300 import spx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,dtype,out", [(8388480, BF16, F32), (8388481, F16, F16), (16776958, BF16, F32), (16776959, BF16, F32), (16776960, F16, F32)])
def test_gradient_of_the_longest_rows(H, dtype, out):
    """One id goes on over a chunk's end (1024 sorted tokens at these lengths).  The sums are whole numbers up to 3 * 513, exact
    in fp32; fp16 holds every whole number to 2048."""
    T = 1027
    ids = torch.ones(T, dtype=torch.int32, device="cuda")
    ids[5], ids[701] = 0, 2
    times = torch.arange(T, device="cuda") % 2
    base = whole(1, H, dtype=dtype)
    dY = times.to(dtype)[:, None] * base
    want = torch.stack([base.float() * int(times[ids == v].sum()) for v in range(3)])
    got = spx.spx_embed_grad(ids, dY, 3, dtype=out)
    assert torch.equal(got.float(), want)
    assert spx.spx_embed_grad(ids, dY, 3, dW=got, accumulate=True) is got
    assert torch.equal(got.float(), (2 * want).to(out).float())
