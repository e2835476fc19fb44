"""Rows of a table by token id and the table's gradient on the GPU.

The lookup is one fp32 product rounded once, compared bit for bit with torch's.  The gradient's sums of whole numbers
are exact below 2^24 and compared bit for bit after the same rounding; of other values, a sum of n terms in fp32 is off
by at most n u of the sum of their magnitudes, u = 2^-24, and the factor's product by one more."""
import numpy as np
import pytest
import torch

from block_util import BF16, F16, F32, U, between, close, gen, normal, padded, whole
from csr_bsr_spmv_gb300 import spx

pytestmark = pytest.mark.gpu


def ids_of(T, V, seed, kind="zipf", dtype=torch.int64):
    g = gen(seed)
    if kind == "same":
        return torch.full((T,), V // 2, device="cuda").to(dtype)
    if kind == "even":
        return torch.randint(0, V, (T,), device="cuda", generator=g).to(dtype)
    x = (torch.rand(T, device="cuda", generator=g, dtype=torch.float64).clamp(min=1e-9) ** -1.0).long() - 1  # heavy head
    x = torch.randperm(V, device="cuda", generator=g)[x.clamp(max=V - 1)]
    x[torch.rand(T, device="cuda", generator=g) < 0.05] = -1
    x[torch.rand(T, device="cuda", generator=g) < 0.05] = V
    return x.to(dtype)


def grad64(ids, dY, V, scale, padding=None):
    ok = (ids >= 0) & (ids < V)
    if padding is not None:
        ok &= ids != padding
    at = ids[ok].long()
    out = torch.zeros(V, dY.shape[1], dtype=torch.float64, device="cuda")
    near = torch.zeros_like(out)
    out.index_add_(0, at, dY.double()[ok])
    near.index_add_(0, at, dY.double()[ok].abs())
    n = torch.bincount(at, minlength=V).double()[:, None]
    return out * scale, near * abs(scale) * (n + 1) * U


@pytest.mark.parametrize("T,V,H", [(1, 1, 1), (1, 1000, 4096), (7, 50, 130), (300, 20000, 1002), (5, 9, 4097), (4099, 300, 72),
                                   (2, 77, 40000), (2000, 501, 512)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_lookup_is_the_scaled_row(T, V, H, dtype):
    W = normal(T, V, H, dtype=dtype)
    for id_type in (torch.int32, torch.int64):
        ids = ids_of(T, V, H, dtype=id_type)
        ok = ((ids >= 0) & (ids < V))[:, None]
        for scale in (1.0, 7.3):
            want = torch.where(ok, W[ids.long().clamp(0, V - 1)].float() * scale, 0.0).to(dtype)
            assert torch.equal(spx.spx_embed(ids, W, scale), want)


@pytest.mark.parametrize("T,V,H", [(1, 1, 1), (1, 5000, 4096), (31, 3, 130), (33, 40, 72), (64, 2, 264), (300, 20000, 1002),
                                   (3001, 501, 1031), (5000, 30000, 24), (20000, 100, 40), (140000, 70000, 8), (3000, 1300000, 2)])
@pytest.mark.parametrize("kind", ["zipf", "even", "same"])
@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, BF16), (BF16, F32), (F16, F16)])
def test_gradient_sums_by_id(T, V, H, kind, dtype, out):
    ids = ids_of(T, V, T + H, kind)
    dY = whole(V, T, H, dtype=dtype)
    want = grad64(ids, dY, V, 0.5)[0]
    got = spx.spx_embed_grad(ids, dY, V, 0.5, dtype=out)
    assert torch.equal(got, want.float().to(out))
    base = whole(3, V, H, dtype=out)
    acc = base.clone()
    assert spx.spx_embed_grad(ids.int(), dY, V, 0.5, dW=acc, accumulate=True) is acc
    assert torch.equal(acc, (want + base.double()).float().to(out))


@pytest.mark.parametrize("H", [32, 64, 256, 258, 512, 700, 1024, 2048, 4097])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradient_of_one_id_among_others(H, dtype):
    """An id of hundreds of chunks between ids of one token, rows from one warp's width to several blocks'."""
    T, V = 9001, 5000
    ids = torch.where(torch.arange(T, device="cuda") % 7 == 3, ids_of(T, V, H, "even"), 2500)
    dY = whole(H, T, H, dtype=dtype)
    assert torch.equal(spx.spx_embed_grad(ids, dY, V, dtype=F32), grad64(ids, dY, V, 1.0)[0].float())


@pytest.mark.parametrize("T,V,H", [(3000, 200, 136), (16384, 5000, 264)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradient_of_any_values_is_the_same_every_time(T, V, H, dtype):
    ids, dY = ids_of(T, V, 5), normal(6, T, H, dtype=dtype)
    got = spx.spx_embed_grad(ids, dY, V, 3.7, padding=1, dtype=F32)
    ref, err = grad64(ids, dY, V, 3.7, 1)
    close(got, ref, err)
    assert not got[1].any()
    for _ in range(3):
        assert torch.equal(spx.spx_embed_grad(ids, dY, V, 3.7, padding=1, dtype=F32), got)


@pytest.mark.parametrize("pad", [1, 2, 4, 8])
@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, BF16), (F16, F32)])
@pytest.mark.parametrize("H", [64, 70])
def test_pitches_and_bases_of_any_alignment(pad, dtype, out, H):
    T, V = 500, 90
    ids = ids_of(T, V, 1)
    W, dY = padded(whole(1, V, H, dtype=dtype), pad), padded(whole(2, T, H, dtype=dtype), pad)
    Y, dW = padded(torch.zeros(T, H, dtype=dtype, device="cuda"), pad), padded(torch.zeros(V, H, dtype=out, device="cuda"), pad)
    edges = [between(Y, pad), between(dW, pad)]
    spx.spx_embed(ids, W, 2.0, Y=Y)
    assert torch.equal(Y, spx.spx_embed(ids, W.contiguous(), 2.0))
    want = grad64(ids, dY, V, 2.0)[0]
    spx.spx_embed_grad(ids, dY, V, 2.0, dW=dW)
    assert torch.equal(dW, want.float().to(out))
    spx.spx_embed_grad(ids, dY, V, 2.0, dW=dW, accumulate=True)
    assert torch.equal(dW, (2 * want).float().to(out))
    for t, e in zip((Y, dW), edges):
        assert torch.equal(between(t, pad).nan_to_num(5), e.nan_to_num(5))


def test_ids_of_any_shape_and_of_far_values():
    W = normal(1, 100, 16)
    ids = torch.tensor([[3, -1, 99], [100, 1 << 40, -(1 << 40)]], device="cuda")
    Y = spx.spx_embed(ids, W)
    assert torch.equal(Y[0], W[3]) and torch.equal(Y[2], W[99]) and not Y[[1, 3, 4, 5]].any()
    dW = spx.spx_embed_grad(ids, torch.ones(6, 16, device="cuda"), 100)
    assert dW.sum() == 32 and torch.equal(dW[3], torch.ones(16, device="cuda"))


def test_no_tokens_and_all_dropped():
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert spx.spx_embed(none, normal(1, 5, 8)).shape == (0, 8)
    dW = torch.full((5, 8), 3.0, device="cuda")
    spx.spx_embed_grad(none, torch.empty(0, 8, device="cuda"), 5, dW=dW, accumulate=True)
    assert (dW == 3).all()
    assert not spx.spx_embed_grad(none, torch.empty(0, 8, device="cuda"), 5).any()
    ids = torch.full((700,), -1, device="cuda")
    assert not spx.spx_embed_grad(ids, normal(2, 700, 8), 5, dW=dW).any()
    assert not spx.spx_embed_grad(torch.full((700,), 4, device="cuda"), normal(2, 700, 8), 5, padding=4, dW=dW).any()


def test_infinities_stay_with_their_ids():
    """A NaN or infinity reaches its own id's row alone, though ids share a block's chunk of tokens."""
    T, V, H = 400, 50, 24
    ids = ids_of(T, V, 3, "even")
    dY = whole(4, T, H)
    t = int((ids == ids[7]).nonzero()[-1])
    dY[t, 5] = float("nan")
    got = spx.spx_embed_grad(ids, dY, V)
    bad = got.isnan()
    assert bad[ids[7], 5] and int(bad.sum()) == 1


def test_offsets_past_32_bits():
    V, H = (1 << 31) // 4096 + 9, 4096
    W = torch.zeros(V, H, dtype=BF16, device="cuda")
    W[-1] = 2
    ids = torch.tensor([V - 1, 0, V - 1], device="cuda")
    Y = spx.spx_embed(ids, W)
    assert (Y[0] == 2).all() and not Y[1].any()
    dW = spx.spx_embed_grad(ids, Y, V, dW=W.fill_(1))
    assert (dW[-1] == 4).all() and not dW[:-1].any()


@pytest.mark.parametrize("T,V", [(40, 1000), (5000, 3000)])
def test_streams_and_graphs(T, V):
    H = 136
    ids, W, dY = ids_of(T, V, 1), whole(2, V, H, dtype=BF16), whole(3, T, H, dtype=BF16)

    def run():
        return [spx.spx_embed(ids, W, 2.0), spx.spx_embed_grad(ids, dY, V, 2.0)]

    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [spx.spx_embed(ids, W, 2.0, stream=side), spx.spx_embed_grad(ids, dY, V, 2.0, stream=side)]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
        graphs.append((g, out))
    for seed in (10, 20):
        ids.copy_(ids_of(T, V, seed))
        dY.copy_(whole(seed, T, H, dtype=BF16))
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for a, *rest in zip(run(), *(out for _, out in graphs)):
            assert all(torch.equal(a, b) for b in rest)
